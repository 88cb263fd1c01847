"""Rows all of whose scores lie far below zero (a key offset against the
query's direction): the reference of the running softmax moves down by
more than float32's exponents hold, on the row's first tile or later.

Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu


def low_scores(t, nats, seed):
    """Queries about 1 in every dim, keys about -c: scores around -nats."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = nats / (t.d * t.scale)
    t.q.copy_(1 + 0.25 * torch.randn(t.q.shape, generator=g, device="cuda"))
    used = ~torch.isnan(t.kc)
    k = (torch.randn(t.kc.shape, generator=g, device="cuda") - c).to(t.kc.dtype)
    t.kc[used] = k[used]


DECODE = [
    ("bf16", 8, 2, 128, 16, [(100, [9, 1, 40]), (64, [0, 0])]),
    ("f16", 14, 2, 64, 16, [(1000, [5, 0, 300] * 9)]),
    ("bf16", 32, 8, 128, 32, [(256, [1 + i % 7 for i in range(100)])]),   # whole units
    ("f16", 6, 2, 128, 32, [(6000, [1500, 0, 40])]),                      # units cut many times over
]


@pytest.mark.parametrize("nats", [100, 300, -300])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}")
def test_shared_prefix_with_low_scores(case, nats):
    t = Batch(*case, seed=51)
    low_scores(t, nats, 52)
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_shared_prefix_whose_first_tiles_weigh_nothing(dtype):
    """Scores of -inf over the prefix's first two tiles, then around -300:
    the reference first moves with O already begun."""
    t = Batch(dtype, 8, 2, 128, 16, [(260, [1, 0, 30])], seed=53)
    low_scores(t, 300, 54)
    t.q[..., 0] = t.q[..., 0].abs() + 0.5
    t.kc[t.tables[0, :8].long(), :, :, 0] = float("-inf")
    t.run()
    check_batch(t)
