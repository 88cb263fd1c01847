"""Decode attention under score rules against float64 (tests/rules64.py).

Caps, slopes, windows and first keys, alone and together, on every kernel
(stream-K in 16 bits and fp8, split, SIMT); one token to thousands; windows
that begin and end anywhere in a tile; sequences that see nothing; freed
blocks; infinities and NaN in keys that are not seen; capture and replay."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu

LENS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 65, 100, 129, 500, 1000, 0, 2049]
SHAPES = [  # dtype, Hq, Hkv, D, bs: stream-K, then SIMT and the split kernel
    ("bf16", 32, 8, 128, 16), ("f16", 28, 4, 128, 32), ("f16", 14, 2, 64, 16), ("bf16", 16, 16, 64, 32),
    ("bf16", 16, 1, 128, 16), ("f16", 16, 8, 256, 16), ("bf16", 8, 1, 256, 32),
    ("f32", 8, 2, 64, 16), ("f32", 6, 3, 20, 5), ("bf16", 20, 1, 128, 16), ("f16", 9, 3, 96, 7), ("bf16", 16, 1, 256, 16),
]
RULES = [  # cap, slopes, window
    (0.0, False, 0), (30.0, False, 0), (0.0, True, 0), (0.0, False, 1), (5.0, True, 33), (0.0, False, 64), (1.5, True, 700),
]


def _slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)


def _run(t, **rules):
    pk.device_error()
    if t.fp8:
        got = pk.paged_decode_attention_rules_fp8(t.out, t.q, t.kc, t.vc, t.cache["ks"], t.cache["vs"], t.tables, t.seq_lens,
                                                  t.scale, max(max(t.lens), 1), **rules)
    else:
        got = pk.paged_decode_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, max(max(t.lens), 1),
                                              **rules)
    assert got is t.out and pk.device_error() == 0


@pytest.mark.parametrize("rules", RULES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decode_under_rules(shape, rules):
    dtype, hq, hkv, d, bs = shape
    cap, sloped, window = rules
    t = PagedBatch(dtype, hq, hkv, d, bs, LENS, seed=hq + d + window)
    slopes = _slopes(hq) if sloped else None
    _run(t, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window)


@pytest.mark.parametrize("rules", RULES, ids=str)
@pytest.mark.parametrize("shape", [("bf16", 28, 4, 128, 16), ("f16", 32, 8, 128, 32), ("bf16", 16, 1, 128, 16),
                                   ("f16", 16, 1, 128, 32)], ids=str)
def test_fp8_decode_under_rules(shape, rules):
    dtype, hq, hkv, d, bs = shape
    cap, sloped, window = rules
    t = PagedBatch(dtype, hq, hkv, d, bs, LENS, seed=hq + bs, fp8=True)
    slopes = _slopes(hq) if sloped else None
    _run(t, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 40])
def test_first_keys(fp8, window):
    """key_begin of every kind: negative, inside, the last key, at and past the end (nothing seen)."""
    lens = [5, 70, 70, 70, 70, 333, 333, 64, 1, 1]
    begin = torch.tensor([-7, 0, 13, 69, 70, 200, 2 ** 31 - 1, 32, 0, 1], dtype=torch.int32, device="cuda")
    t = PagedBatch("bf16", 8, 2, 128, 16, lens, seed=3, fp8=fp8)
    _run(t, key_begin=begin, window=window)
    t.check(begin=begin, window=window)
    for b in (4, 6, 9):
        assert not t.out[b].any()


@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16, False), ("bf16", 8, 2, 128, 32, False), ("f16", 8, 2, 64, 16, False),
                                   ("bf16", 8, 2, 128, 16, True), ("bf16", 8, 2, 128, 32, True), ("f32", 4, 2, 64, 8, False),
                                   ("f16", 32, 1, 64, 16, False)], ids=str)
def test_freed_blocks_are_not_looked_up(shape):
    """Blocks that end before the window hold NaN and their table entries are -1 or wild, as after their release; the
    slots of the window's first block before it hold NaN too."""
    dtype, hq, hkv, d, bs, fp8 = shape
    lens = [700, 64, 65, 90, 301, 41]
    window = 50
    t = PagedBatch(dtype, hq, hkv, d, bs, lens, seed=9, fp8=fp8)
    for b, n in enumerate(lens):
        lo = max(0, n - window)
        blk = int(t.tables[b, lo // bs])
        if fp8:
            for name in ("k", "v"):
                t.cache[name][blk, :lo % bs] = 0x7F
                t.cache[name + "s"][blk, :, :lo % bs] = float("nan")
        else:
            t.kc[blk, :lo % bs] = float("nan")
            t.vc[blk, :lo % bs] = float("inf")
        t.tables[b, :lo // bs] = torch.tensor([-1, 2 ** 30, -2 ** 31, t.nb])[torch.arange(lo // bs) % 4].to(torch.int32).cuda()
    _run(t, window=window)
    assert bool(torch.isfinite(t.out).all())
    t.check(window=window)


@pytest.mark.parametrize("dtype,hq,d", [("bf16", 8, 128), ("f16", 8, 64), ("f32", 8, 64)])
def test_infinite_and_nan_keys(dtype, hq, d):
    """A seen key of NaN reaches its rows, one of +inf is capped to the cap, one of -inf to minus it; unseen: nothing."""
    lens = [100, 100, 100, 100]
    t = PagedBatch(dtype, hq, 2, d, 16, lens, seed=5)
    t.q.abs_()                                                  # so that an infinite key's score is that infinity
    slot = {b: (int(t.tables[b, 5]), 3) for b in range(4)}      # position 83
    for b, x in enumerate((float("nan"), float("inf"), float("-inf"), float("nan"))):
        t.kc[slot[b]] = x
    begin = torch.tensor([0, 0, 0, 84], dtype=torch.int32, device="cuda")
    _run(t, softcap=10.0, key_begin=begin)
    t.check(cap=10.0, begin=begin)
    assert bool(torch.isnan(t.out[0]).all()) and bool(torch.isfinite(t.out[1:]).all())


@pytest.mark.parametrize("cap", [1e-3, 0.5, 1e4, 1e12])
def test_caps_of_any_size(cap):
    """A small cap flattens the weights, a huge one leaves the scores as they are (not lost to the cap's size)."""
    t = PagedBatch("f32", 8, 2, 64, 16, [300, 77], seed=11)
    _run(t, softcap=cap)
    t.check(cap=cap)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_slopes_of_either_sign_over_a_long_cache(sign):
    t = PagedBatch("bf16", 8, 2, 64, 32, [20000, 3], seed=12)
    slopes = _slopes(8) * sign
    _run(t, slopes=slopes)
    t.check(slopes=slopes)


def test_no_rules_is_the_plain_call():
    t = PagedBatch("bf16", 28, 4, 128, 16, [700, 64, 1, 0, 999], seed=2)
    _run(t)
    t.check()
    # (not to the bit: few units are cut into fewer pieces, whose float32 sums are joined in another order)
    plain = torch.empty_like(t.out)
    pk.paged_decode_attention(plain, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, 999)
    t.check(out=plain)


def test_more_sequences_than_the_stream_kernel_takes():
    """4100 sequences: the split kernel."""
    lens = [(7 * i) % 90 for i in range(4100)]
    t = PagedBatch("bf16", 4, 2, 64, 16, lens, seed=1)
    slopes = _slopes(4)
    _run(t, softcap=3.0, slopes=slopes, window=37)
    t.check(cap=3.0, slopes=slopes, window=37, seqs=range(0, 4100, 41))
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert not t.out[empty].any()


def test_a_few_sequences_split_over_their_windows():
    """Few long sequences with a window: SIMT and split partials start at the window, not at the first block."""
    for dtype, hq, hkv, d in (("f32", 4, 2, 64), ("bf16", 16, 1, 256)):
        t = PagedBatch(dtype, hq, hkv, d, 16, [9000, 5000], seed=8)
        for window in (0, 3000, 17):
            _run(t, window=window)
            t.check(window=window)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed_on_another_stream(fp8):
    """One captured call replayed after the lengths and first keys changed in place; the workspace is the caller's."""
    t = PagedBatch("bf16", 32, 8, 128, 16, [3000, 70, 513], seed=6, fp8=fp8)
    begin = torch.zeros(3, dtype=torch.int32, device="cuda")
    plan = pk.decode_plan(3, 32, 8, 128, 16, 3000, torch.bfloat16)
    ws = pk.alloc_workspace(plan, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _run(t, softcap=20.0, window=100, key_begin=begin, workspace=ws, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            kw = dict(softcap=20.0, window=100, key_begin=begin, workspace=ws)
            if fp8:
                pk.paged_decode_attention_rules_fp8(t.out, t.q, t.kc, t.vc, t.cache["ks"], t.cache["vs"], t.tables,
                                                    t.seq_lens, t.scale, 3000, **kw)
            else:
                pk.paged_decode_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, 3000, **kw)
    for lens, first in (([3000, 70, 513], [0, 0, 0]), ([2900, 33, 1], [2850, 40, 0]), ([17, 70, 500], [3, 69, 460])):
        t.lens = lens
        t.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        begin.copy_(torch.tensor(first, dtype=torch.int32))
        t.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        t.check(cap=20.0, window=100, begin=begin)
    assert pk.device_error() == 0


def test_same_call_same_bits():
    t = PagedBatch("f16", 28, 4, 128, 32, [4000, 100, 2222], seed=4)
    slopes = _slopes(28)
    _run(t, softcap=30.0, slopes=slopes, window=2000)
    first = t.out.clone()
    for _ in range(10):
        _run(t, softcap=30.0, slopes=slopes, window=2000)
        assert torch.equal(first, t.out)
