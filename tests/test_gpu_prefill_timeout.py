"""The tcgen05 prefill when a bounded wait runs out: CTA 0 never loads one of
its K tiles, the launch ends (after a second or two) with
KV_ERR_DEVICE_TIMEOUT, what it had in flight has ended with it, the other
CTAs' rows are right, and so are later calls."""

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


@pytest.mark.parametrize("dtype, d, skip", [("bf16", 128, 0), ("bf16", 128, 3), ("f16", 64, 0), ("f16", 64, 5)])
def test_a_wait_that_runs_out(dtype, d, skip):
    dev, dt, bs, hq, hkv, n, seqs = torch.device("cuda"), TORCH[dtype], 16, 8, 2, 1000, 3
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
        pk.paged_prefill_attention(out, q, kc, vc, tables, lens, qsl, d ** -0.5, n)

    run()
    want = out.clone()
    pk.device_error()
    kernels.debug_set(kernels.DEBUG_SKIP_TILE, skip)
    out.zero_()
    run()
    assert pk.device_error() == KV_ERR_DEVICE_TIMEOUT
    # CTA 0: the first head group's last row tile of the first sequence; nothing of it is written
    assert torch.equal(out[n:], want[n:]) and torch.equal(out[:n, 4:], want[:n, 4:])
    lost = (out[:n, :4] != want[:n, :4]).flatten(1).any(1)
    assert bool(lost.any()) and not bool(out[:n][lost][:, :4].any())
    kernels.debug_reset()
    for _ in range(3):
        out.zero_()
        run()
        assert torch.equal(out, want)
    assert pk.device_error() == 0
