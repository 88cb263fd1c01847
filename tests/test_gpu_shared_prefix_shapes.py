"""Shared-prefix attention where the row tiles' shape is unusual: query groups
whose rows do not fill a tile of 128, over several row tiles, and the sizes
that are not the kernel's (more than 16 query heads per kv head, more than
4096 sequences), which are the plain call bit for bit.

Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix, n", [(300, 21), (3000, 9), (64, 40)])
@pytest.mark.parametrize("hq, hkv, d", [(30, 2, 128), (15, 1, 64), (32, 2, 128), (48, 3, 64), (26, 2, 128), (9, 1, 64),
                                        (10, 2, 128), (3, 3, 64)])
def test_groups_that_do_not_fill_their_row_tiles(hq, hkv, d, prefix, n):
    """G 15, 15, 16, 16, 13, 9, 5, 1: 8, 8, 8, 8, 9, 14, 25 and 128 sequences a tile."""
    t = Batch("bf16" if hq % 2 == 0 else "f16", hq, hkv, d, 16, [(prefix, [i * 7 % 50 for i in range(n)])], seed=101)
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t, seqs=sorted({0, 1, 7, 8, n // 2, n - 1} & set(range(n))))


@pytest.mark.parametrize("case", [("f16", 128, 1, 64, 16, [(80, [9, 70, 1])]), ("bf16", 34, 2, 128, 16, [(200, [5, 6])]),
                                  ("bf16", 4, 1, 128, 16, [(64, [1 + i % 3 for i in range(4100)])])],
                         ids=["G128", "G17", "4100 sequences"])
def test_sizes_past_the_kernels_are_the_plain_call(case):
    t = Batch(*case, seed=102)
    t.run()
    want = torch.empty_like(t.out)
    pk.paged_decode_attention(want, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, max(t.lens))
    assert torch.equal(t.out, want) and pk.device_error() == 0
