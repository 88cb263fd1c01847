"""fp16 probabilities far below their row's largest: weights down to 2^-24 of
it count, whatever the level of the row's scores.

Every tile of 16 keys holds one key of the row's largest score and 15 whose
weight is 2^-17.5 of it; the first's value is 0, the others' 1000, so that the
result is the small weights' sum.  Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu

LN2 = 0.6931471805599453


@pytest.mark.parametrize("top", [-7.9, -3.0, 0.0, 5.0, 13.0, -40.0])
@pytest.mark.parametrize("case", [("f16", 8, 2, 128, 16, [(640, [1, 33, 0])]),
                                  ("f16", 14, 2, 64, 32, [(320, [2, 0, 70] * 12)] * 3)], ids=["128", "64"])
def test_shared_prefix_keeps_small_weights(case, top):
    """top: the largest score, in powers of two."""
    t = Batch(*case, seed=71)
    t.scale = 1.0
    t.q.zero_()
    t.q[..., 0] = 1.0
    used = ~torch.isnan(t.kc[..., 0])
    score = torch.full((t.bs,), (top - 17.5) * LN2, device="cuda")
    score[::16] = top * LN2
    value = torch.full((t.bs,), 1000.0, device="cuda")
    value[::16] = 0
    k, v = torch.zeros_like(t.kc), torch.zeros_like(t.vc)
    k[..., 0] = score[None, :, None].half()
    v[:] = value[None, :, None, None].half()
    t.kc[used], t.vc[used] = k[used], v[used]
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)
    assert float(t.out[0].float().mean()) > 0.05       # 15 of 16 keys, 1000 2^-17.5 each: about 0.08
