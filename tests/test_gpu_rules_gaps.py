"""Prefill under score rules where the intervals of a tile's rows leave keys
between them that no row sees: NaN and infinity in the keys and values there
reach no row."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 8, 2, 128, 16), ("f16", 4, 4, 64, 32), ("f16", 16, 2, 128, 128), ("bf16", 3, 1, 64, 64),
          ("bf16", 8, 2, 64, 8), ("f16", 6, 2, 128, 5)]


def _poison(t, b, lo, hi):
    """K and V of sequence b's keys that none of the intervals [lo, hi) holds; how many there are."""
    L = t.lens[b]
    seen = torch.zeros(L, dtype=torch.bool)
    for x, y in zip(lo.tolist(), hi.tolist()):
        seen[max(x, 0):max(min(y, L), 0)] = True
    p = torch.nonzero(~seen)[:, 0].cuda()
    blk, off = t.tables[b].long()[p // t.bs], p % t.bs
    t.kc[blk, off] = float("nan")
    t.vc[blk, off] = torch.where(p % 2 == 0, float("nan"), float("inf"))[:, None, None].to(t.vc.dtype)
    return len(p)


@pytest.mark.parametrize("cap, sloped", [(0.0, False), (9.0, False), (0.0, True)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_nan_between_intervals(shape, cap, sloped):
    """Intervals of neighbouring rows far from each other, over several key tiles; every kind of gap: within a block,
    over whole blocks and whole tiles, at the ends; rows that see nothing among them."""
    t = PagedBatch(*shape, [700, 600], [300, 70], seed=17)
    g = torch.Generator().manual_seed(5)
    begin = torch.zeros(370, dtype=torch.int64)
    end = torch.zeros(370, dtype=torch.int64)
    spots = torch.tensor([[3, 10], [100, 110], [127, 129], [290, 291], [300, 390], [505, 511], [512, 600]])
    pick = torch.randint(0, len(spots), (300,), generator=g)
    begin[:300], end[:300] = spots[pick].T
    end[40:50] = 0                                       # nothing
    begin[200:300], end[200:300] = 650, 655              # later tiles: one stretch alone
    begin[300:], end[300:] = 64, 65                      # the other sequence: two keys
    begin[369], end[369] = 599, 600
    assert _poison(t, 0, begin[:300], end[:300]) > 400
    assert _poison(t, 1, begin[300:], end[300:]) == 598
    begin, end = begin.to(torch.int32).cuda(), end.to(torch.int32).cuda()
    slopes = torch.exp2(-8.0 * torch.arange(1, t.hq + 1, device="cuda") / t.hq) if sloped else None
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 300, key_begin=begin,
                                     key_end=end, softcap=cap, slopes=slopes)
    assert pk.device_error() == 0
    assert bool(torch.isfinite(t.out).all())
    t.check(cap=cap, slopes=slopes, begin=begin, end=end)


@pytest.mark.parametrize("shape", [("bf16", 32, 8, 128, 16), ("f16", 8, 1, 128, 32), ("bf16", 14, 2, 64, 16)], ids=str)
def test_nan_between_intervals_of_a_cut_call(shape):
    """A window and ends below the rows' own positions, over a history long enough for the keys to be cut in pieces."""
    window = 5000
    t = PagedBatch(*shape, [20040], [40], seed=3)
    pos = torch.arange(20000, 20040)
    end = torch.full((40,), 15020)
    end[39] = 20040
    lo = pos - window + 1
    end[:20] = lo[:20] + 3
    assert _poison(t, 0, lo, end) > 15000 + 15
    end = end.to(torch.int32).cuda()
    ws = pk.prefill_rules_workspace(40, 1, t.hq, t.hkv, t.d, t.bs, t.tables.shape[1], 40, "cuda", window)
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 40, window=window,
                                     key_end=end, workspace=ws)
    assert pk.device_error() == 0
    assert int(ws[:4].view(torch.int32)[0]) > 1          # it was cut
    assert bool(torch.isfinite(t.out).all())
    t.check(window=window, end=end)
