"""Prefill under score rules: a row whose key_end lies far below zero sees
nothing, whatever the other rows of its tile see."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap, sloped", [(0.0, False), (8.0, False), (0.0, True), (8.0, True)])
@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 4, 4, 64, 32), ("f16", 16, 2, 128, 128),
                                   ("bf16", 8, 2, 64, 8)], ids=str)
def test_ends_far_below_zero(shape, cap, sloped):
    t = PagedBatch(*shape, [430, 260], [130, 260], seed=12)
    rows = sum(t.chunks)
    pos = torch.cat([torch.arange(L - n, L) for L, n in zip(t.lens, t.chunks)])
    end = pos + 1
    far = torch.tensor([-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 64, -2 ** 31 + 128, -2 ** 31 + 200, -2 ** 31 + 2 ** 20, -1, 0])
    none = torch.arange(3, rows, 5)
    end[none] = far[torch.arange(len(none)) % len(far)]
    end = end.to(torch.int32).cuda()
    slopes = torch.exp2(-8.0 * torch.arange(1, t.hq + 1, device="cuda") / t.hq) if sloped else None
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 260, key_end=end,
                                     softcap=cap, slopes=slopes)
    assert pk.device_error() == 0
    assert not t.out[none.cuda()].any()
    t.check(cap=cap, slopes=slopes, end=end)
