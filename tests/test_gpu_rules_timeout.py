"""The tcgen05 prefill under score rules when a bounded wait runs out: CTA 0
never loads one of its K tiles nor any after it, the launch ends (after a few
seconds) with KV_ERR_DEVICE_TIMEOUT, what it had in flight has ended with it,
no row holds anything but its result or what it held, and later calls are
right."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from paged_kv_cache_128_gb300 import kernels
from tests.helpers import TORCH

pytestmark = pytest.mark.gpu

KV_ERR_DEVICE_TIMEOUT = 10


@pytest.fixture(autouse=True)
def default_controls():
    kernels.debug_reset()
    yield
    kernels.debug_reset()


@pytest.mark.parametrize("dtype, d, skip, rules", [
    ("bf16", 128, 0, {}), ("bf16", 128, 3, dict(softcap=20.0)), ("f16", 64, 0, dict(window=300)), ("f16", 64, 30, {}),
    ("bf16", 64, 9, dict(window=64)),
])
def test_a_wait_that_runs_out(dtype, d, skip, rules):
    dev, dt, bs, hq, hkv, n, seqs = torch.device("cuda"), TORCH[dtype], 16, 8, 2, 1000, 40
    g = torch.Generator(device="cuda").manual_seed(95)
    per = -(-n // bs)
    kc = torch.randn(seqs * per, bs, hkv, d, generator=g, device=dev).to(dt)
    vc = torch.randn(seqs * per, bs, hkv, d, generator=g, device=dev).to(dt)
    q = torch.randn(seqs * n, hq, d, generator=g, device=dev).to(dt)
    tables = torch.arange(seqs * per, dtype=torch.int32, device=dev).view(seqs, per)
    lens = torch.full((seqs,), n, dtype=torch.int32, device=dev)
    qsl = torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device=dev)
    out = torch.zeros_like(q)

    def run():
        pk.paged_prefill_attention_rules(out, q, kc, vc, tables, lens, qsl, d ** -0.5, n, **rules)

    run()
    want = out.clone()
    pk.device_error()
    kernels.debug_set(kernels.DEBUG_SKIP_TILE, skip)
    out.zero_()
    run()
    assert pk.device_error() == KV_ERR_DEVICE_TIMEOUT
    # CTA 0's items from the one with the lost tile on are not written; all else is whole
    lost = (out != want).flatten(2).any(2)
    assert bool(lost.any()) and not bool(out[lost].any())
    assert int(lost.sum()) <= lost.numel() / 100
    kernels.debug_reset()
    for _ in range(3):
        out.zero_()
        run()
        assert torch.equal(out, want)
    assert pk.device_error() == 0
