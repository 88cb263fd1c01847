"""Plain decode attention over keys and queries that hold NaN or an infinity:
a row whose softmax has no value is NaN on every kernel (stream-K whole and
cut, forced splits, SIMT, fp8), and no other row is touched.

Tolerances: tests/attention64.py (the SIMT kernel, which does not round its
probabilities, is within them too).
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu

# dtype, Hq, Hkv, D, block size, lengths; blocks per split (0: stream-K, or the SIMT kernel's choice)
CASES = [
    ("bf16", 8, 2, 128, 16, [5000, 300, 17, 1], 0),            # cut many times over
    ("f16", 14, 2, 64, 32, [40 + i for i in range(300)], 0),   # mostly whole
    ("bf16", 32, 8, 128, 16, [700, 64, 2500], 8),              # forced splits, tensor cores
    ("f16", 8, 2, 80, 16, [900, 33, 5], 0),                    # SIMT
    ("f16", 8, 2, 80, 16, [900, 33, 5], 4),
]
IDS = [f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-{c[6]}" for c in CASES]


def batch(case, seed):
    *shape, lens, bps = case
    t = Batch(*shape, [(0, [n]) for n in lens], seed=seed)
    t.q[..., 0] = t.q[..., 0].abs() + 0.5

    def run():
        pk.device_error()
        pk.paged_decode_attention(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, max(lens), blocks_per_split=bps)
        assert pk.device_error() == 0
    seqs = range(0, len(lens), max(1, len(lens) // 20))
    return t, run, seqs


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_a_key_of_no_number(case, value):
    """Plus infinity times a positive query gives NaN, minus weighs nothing."""
    t, run, seqs = batch(case, 111)
    pos = t.lens[0] // 2
    t.kc[int(t.tables[0, pos // t.bs]), pos % t.bs, 0, 0] = value
    run()
    check_batch(t, seqs=seqs)
    assert bool(torch.isnan(t.out[0, 0]).all()) == (value != float("-inf"))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_a_query_of_no_number(case):
    t, run, seqs = batch(case, 112)
    for b in (0, len(t.lens) - 1):
        t.q[b, t.hq - 1, 5] = float("nan")
    run()
    check_batch(t, seqs=sorted(set(seqs) | {len(t.lens) - 1}))
    assert bool(torch.isnan(t.out[0, t.hq - 1]).all())


def test_fp8_queries_of_no_number():
    """The fp8 kernel: the NaN row is NaN, the others are as they were."""
    B, hq, hkv, d, bs = 3, 8, 2, 128, 16
    t = Batch("bf16", hq, hkv, d, bs, [(0, [n]) for n in (5000, 300, 17)], seed=113)
    kc, vc = (torch.zeros(t.nb, bs, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(t.nb, hkv, bs, device="cuda") for _ in range(2))
    n = t.nb * bs
    pk.reshape_and_cache_fp8(t.kc.nan_to_num(0).view(n, hkv, d), t.vc.nan_to_num(0).view(n, hkv, d), kc, vc, ks, vs,
                             torch.arange(n, dtype=torch.int32, device="cuda"))
    outs = []
    for bad in (False, True):
        if bad:
            t.q[0, 3, 7] = float("nan")
            t.q[2, 0, 0] = float("nan")
        out = torch.empty_like(t.q)
        pk.paged_decode_attention_fp8(out, t.q, kc, vc, ks, vs, t.tables, t.seq_lens, t.scale, 5000)
        outs.append(out)
    nan = torch.zeros(B, hq, dtype=torch.bool, device="cuda")
    nan[0, 3] = nan[2, 0] = True
    assert bool(torch.isnan(outs[1][nan]).all()) and torch.equal(outs[0][~nan], outs[1][~nan])
