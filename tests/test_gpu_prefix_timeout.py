"""The shared-prefix kernel when a bounded wait runs out: one copy of the
prefix line is never made, the launch ends (after a second or two) with
KV_ERR_DEVICE_TIMEOUT, what it had in flight has ended with it, and later
calls on the same workspace are right."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from paged_kv_cache_128_gb300 import kernels
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu

KV_ERR_DEVICE_TIMEOUT = 10

# case; numbers of copies that the prefix line's first share has: K of the first tile, K of the second, V of the first ..
CASES = [
    (("bf16", 32, 8, 128, 16, [(4096, [300, 17, 64] * 20)]), [0, 1, 2, 9]),  # part of a long unit
    (("f16", 14, 2, 64, 32, [(128, [40] * 30)] * 40), [0, 3, 7]),            # several units
]


@pytest.fixture(autouse=True)
def default_controls():
    kernels.debug_reset()
    yield
    kernels.debug_reset()


@pytest.mark.parametrize("case, skip", [(c, k) for c, skips in CASES for k in skips],
                         ids=lambda x: str(x) if isinstance(x, int) else f"{x[0]}-{x[1]}x{x[2]}x{x[3]}")
def test_a_wait_that_runs_out(case, skip):
    t = Batch(*case, seed=91)
    ws = pk.shared_prefix_workspace(len(t.lens), t.hq, t.hkv, t.d, t.bs, max(t.lens), t.q.dtype, "cuda")
    t.run(workspace=ws)
    want = t.out.clone()
    pk.device_error()
    kernels.debug_set(kernels.DEBUG_SKIP_TILE, skip)
    t.run(workspace=ws)
    assert pk.device_error() == KV_ERR_DEVICE_TIMEOUT
    kernels.debug_reset()
    for _ in range(3):
        t.out.fill_(float("nan"))
        t.run(workspace=ws)
        assert torch.equal(t.out, want)
    assert pk.device_error() == 0
    if skip == 0:
        t.check()
