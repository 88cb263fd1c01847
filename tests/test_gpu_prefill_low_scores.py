"""Chunked prefill of rows all of whose scores lie far below (or above) zero,
from their first key tile on or after tiles that weigh nothing, on both
prefill kernels (tcgen05: block size 16 and more; mma.sync: 8).

Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import attention64, check_rows
from tests.helpers import TORCH

pytestmark = pytest.mark.gpu

SEQS = [(0, 1), (0, 70), (40, 200), (300, 33), (127, 2), (500, 1)]   # history, chunk


def prefill(dtype, hq, hkv, d, bs, nats, seed, nothing=0):
    """Queries about 1 in every dim, keys about -c: scores around -nats; the
    first `nothing` keys of each sequence score -inf."""
    dev, dt = torch.device("cuda"), TORCH[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    scale = d ** -0.5
    lens = [c + n for c, n in SEQS]
    blocks = [-(-L // bs) for L in lens]
    nb = sum(blocks)
    place = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    tables = torch.full((len(SEQS), max(blocks)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(blocks):
        tables[b, :n] = place[at:at + n]
        at += n
    c = nats / (d * scale)
    kc = (torch.randn(nb, bs, hkv, d, generator=g, device=dev) - c).to(dt)
    vc = torch.randn(nb, bs, hkv, d, generator=g, device=dev).to(dt)
    T = sum(n for _, n in SEQS)
    q = (1 + 0.25 * torch.randn(T, hq, d, generator=g, device=dev)).to(dt)
    if nothing:
        q[..., 0] = q[..., 0].abs() + 0.5
        for b, L in enumerate(lens):
            pos = torch.arange(min(nothing, SEQS[b][0]), device=dev)
            kc[tables[b, pos // bs].long(), pos % bs, :, 0] = float("-inf")
    out = torch.full_like(q, float("nan"))
    qsl = torch.tensor([0] + [n for _, n in SEQS]).cumsum(0).to(torch.int32).to(dev)
    pk.device_error()
    pk.paged_prefill_attention(out, q, kc, vc, tables, torch.tensor(lens, dtype=torch.int32, device=dev), qsl, scale,
                               max(n for _, n in SEQS))
    assert pk.device_error() == 0
    at = 0
    for b, (ctx, n) in enumerate(SEQS):
        L = ctx + n
        k = kc[tables[b, :blocks[b]].long()].reshape(-1, hkv, d)[:L]
        v = vc[tables[b, :blocks[b]].long()].reshape(-1, hkv, d)[:L]
        seen = torch.arange(L, device=dev) <= torch.arange(ctx, L, device=dev)[:, None]
        for h in range(hq):
            kvh = h // (hq // hkv)
            o, tol = attention64(q[at:at + n, h], k[:, kvh], v[:, kvh], scale, dtype, seen)
            check_rows(out[at:at + n, h], o, tol, (b, h))
        at += n


@pytest.mark.parametrize("nats", [100, 300, -300])
@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 14, 2, 64, 32), ("bf16", 4, 4, 64, 128),
                                   ("f16", 4, 1, 128, 64), ("bf16", 8, 2, 128, 8)], ids=str)
def test_prefill_with_low_scores(shape, nats):
    prefill(*shape, nats, seed=81)


@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 4, 2, 64, 32)], ids=str)
def test_prefill_whose_first_tiles_weigh_nothing(shape):
    prefill(*shape, 300, seed=82, nothing=256)
