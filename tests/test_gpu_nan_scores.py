"""Keys, values and queries that hold NaN or an infinity: a row whose softmax
has no value is NaN, wherever its keys are cut into pieces, and no other row
is touched.

Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu

CASES = [
    ("bf16", 8, 2, 128, 16, [(100, [9, 1, 40]), (64, [0, 0])]),
    ("f16", 14, 2, 64, 16, [(200, [5, 0, 300] * 9)]),
    ("bf16", 32, 8, 128, 32, [(256, [1 + i % 7 for i in range(100)])]),   # whole units
    ("f16", 6, 2, 128, 32, [(6000, [1500, 0, 40])]),                      # units cut many times over
    ("bf16", 8, 2, 128, 16, [(0, [3000, 5])]),                            # nothing shared
]


def slot(t, b, pos):
    return int(t.tables[b, pos // t.bs]), pos % t.bs


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}")
def test_a_key_of_no_number(case, value):
    """In the prefix (or the long sequence's middle), one kv head: with
    infinities of scores' sign, plus gives NaN, minus weighs nothing."""
    t = Batch(*case, seed=61)
    t.q[..., 0] = t.q[..., 0].abs() + 0.5
    blk, off = slot(t, 0, t.lens[0] // 2)
    t.kc[blk, off, 0, 0] = value
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)
    assert bool(torch.isnan(t.out[0, 0]).all()) == (value != float("-inf"))


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}")
def test_a_key_of_no_number_in_a_rest(case):
    t = Batch(*case, seed=62)
    b = max(range(len(t.lens)), key=lambda i: t.lens[i])
    blk, off = slot(t, b, t.lens[b] - 1)
    t.kc[blk, off, t.hkv - 1, 3] = float("nan")
    t.run()
    check_batch(t)
    assert bool(torch.isnan(t.out[b, t.hq - 1]).all()) and not bool(torch.isnan(t.out[b, 0]).any())


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}")
def test_a_query_of_no_number_and_values_of_none(case):
    """A NaN query row: every piece of the row is NaN, no other row is.  A NaN
    in a value: that dim of the rows that read it."""
    t = Batch(*case, seed=63)
    t.q[1, 2, 5] = float("nan")
    blk, off = slot(t, 0, t.lens[0] // 2)
    t.vc[blk, off, 0, 7] = float("nan")
    t.run()
    check_batch(t)
    assert bool(torch.isnan(t.out[1, 2]).all())


def test_a_prefix_of_no_numbers():
    t = Batch("bf16", 8, 2, 128, 16, [(320, [9, 0, 40])], seed=64)
    t.kc[t.tables[0, :20].long(), :, 0] = float("nan")
    t.run()
    check_batch(t)
