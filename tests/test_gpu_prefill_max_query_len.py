"""Prefill with a max_query_len of no limit: the largest int32, and sizes
within a row tile of it."""

import pytest

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 65])
@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 6, 6, 64, 32), ("bf16", 8, 2, 64, 8)], ids=str)
@pytest.mark.parametrize("rules", [False, True])
def test_no_limit(shape, most, rules):
    t = PagedBatch(*shape, [430, 37, 5000, 260], [130, 37, 3, 0], seed=12)
    args = (t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, most)
    pk.device_error()
    if rules:
        pk.paged_prefill_attention_rules(t.out, *args, window=90)
    else:
        pk.paged_prefill_attention(t.out, *args)
    assert pk.device_error() == 0
    t.check(window=90 if rules else 0)
