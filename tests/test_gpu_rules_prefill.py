"""Chunked-prefill attention under score rules against float64
(tests/rules64.py): caps, slopes, windows, documents and spans seen both ways,
alone and together, in every head layout and block size; rows that see
nothing; freed blocks; infinities and NaN in keys that no row sees."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu

SEQS = [(0, 1), (0, 5), (0, 17), (13, 7), (100, 1), (0, 130), (300, 130), (31, 33), (5, 0), (127, 129), (700, 65)]
SHAPES = [  # dtype, Hq, Hkv, D, bs
    ("bf16", 8, 2, 128, 16), ("f16", 28, 4, 128, 32), ("bf16", 16, 16, 64, 16), ("f16", 14, 2, 64, 64),
    ("bf16", 8, 1, 128, 128), ("bf16", 3, 1, 64, 32), ("f16", 12, 2, 128, 16), ("bf16", 8, 2, 64, 8), ("f16", 6, 2, 128, 5),
]
RULES = [  # cap, slopes, window
    (0.0, False, 0), (20.0, False, 0), (0.0, True, 0), (0.0, False, 1), (5.0, True, 33), (0.0, False, 150), (1.5, True, 400),
]


def _slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)


def _batch(dtype, hq, hkv, d, bs, seqs, seed, **over):
    return PagedBatch(dtype, hq, hkv, d, bs, [a + n for a, n in seqs], [n for _, n in seqs], seed=seed, **over)


def _run(t, begin=None, end=None, **rules):
    """As the wrapper would, which cuts the keys of few rows into pieces, and without pieces (an empty workspace)."""
    pk.device_error()
    args = (t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, max(max(t.chunks), 1))
    got = pk.paged_prefill_attention_rules(t.out, *args, key_begin=begin, key_end=end, **rules)
    t.uncut = torch.full_like(t.out, float("nan"))
    pk.paged_prefill_attention_rules(t.uncut, *args, key_begin=begin, key_end=end, **rules,
                                     workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert got is t.out and pk.device_error() == 0


def _positions(t):
    return torch.cat([torch.arange(L - n, L) for L, n in zip(t.lens, t.chunks)]).cuda()


@pytest.mark.parametrize("rules", RULES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prefill_under_rules(shape, rules):
    cap, sloped, window = rules
    t = _batch(*shape, SEQS, seed=shape[1] + shape[4] + window)
    slopes = _slopes(t.hq) if sloped else None
    _run(t, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window)


def _spans(t, seed, ahead):
    """Stretches of 1 to 90 tokens over each chunk: key_end their end (ahead) or key_begin their start."""
    g = torch.Generator().manual_seed(seed)
    pos = _positions(t).cpu()
    begin, end = torch.zeros_like(pos), pos + 1
    for r0, n in zip(t.row0, t.chunks):
        at = 0
        while at < n:
            size = min(n - at, int(torch.randint(1, 90, (1,), generator=g)))
            rows = slice(r0 + at, r0 + at + size)
            if ahead and int(torch.randint(0, 2, (1,), generator=g)):
                end[rows] = pos[r0 + at] + size
            elif not ahead:
                begin[rows] = pos[r0 + at]
            at += size
    return begin.to(torch.int32).cuda(), end.to(torch.int32).cuda()


@pytest.mark.parametrize("rules", [(0.0, False, 0), (8.0, True, 0), (0.0, True, 50)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_images_and_documents(shape, rules):
    cap, sloped, window = rules
    t = _batch(*shape, SEQS, seed=shape[1] + 7)
    slopes = _slopes(t.hq) if sloped else None
    _, end = _spans(t, 1, True)
    _run(t, end=end, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window, end=end)
    begin, _ = _spans(t, 2, False)
    _run(t, begin=begin, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window, begin=begin)
    _run(t, begin=begin, end=end, softcap=cap, slopes=slopes, window=window)
    t.check(cap=cap, slopes=slopes, window=window, begin=begin, end=end)


@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 4, 4, 64, 32), ("bf16", 4, 2, 128, 6)], ids=str)
def test_intervals_of_every_kind(shape):
    """Whole sequences seen by every row (a prefix), single keys, ends past the sequence and before its start, and rows
    -- whole tiles of them too -- that see nothing: zeros."""
    seqs = [(0, 150), (90, 40), (200, 300), (10, 3)]
    t = _batch(*shape, seqs, seed=4)
    g = torch.Generator().manual_seed(9)
    L = torch.repeat_interleave(torch.tensor(t.lens), torch.tensor(t.chunks))
    rows = sum(t.chunks)
    begin = (torch.rand(rows, generator=g) * (L + 20)).long() - 10
    end = begin + (torch.rand(rows, generator=g) * L).long() - 5
    begin[:100], end[:100] = -3, 2 ** 31 - 1               # the whole sequence
    begin[100:130] = 149                                   # a single key
    end[100:130] = 150
    end[190:330] = begin[190:330]                          # nothing, over whole tiles
    begin[-1], end[-1] = -2 ** 31, -2 ** 31
    begin, end = begin.to(torch.int32).cuda(), end.to(torch.int32).cuda()
    for cap, slopes in ((0.0, None), (4.0, _slopes(t.hq))):
        t.out.fill_(float("nan"))
        _run(t, begin=begin, end=end, softcap=cap, slopes=slopes)
        t.check(cap=cap, slopes=slopes, begin=begin, end=end)
        assert not t.out[190:330].any()


@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 8, 2, 64, 64), ("bf16", 4, 2, 128, 128),
                                   ("bf16", 4, 2, 64, 8)], ids=str)
def test_freed_blocks_are_not_looked_up(shape):
    """Blocks that end before the first key any row sees are gone from the table; slots of the first block before that
    key hold NaN and infinity.  All rows of a chunk begin at one key, so that key holds for every tile."""
    bs = shape[4]
    t = _batch(*shape, [(300, 40), (130, 70), (64, 64), (1000, 200)], seed=3)
    first = [290, 100, 63, 801]
    begin = torch.cat([torch.full((n,), f, dtype=torch.int32) for f, n in zip(first, t.chunks)]).cuda()
    for b, lo in enumerate(first):
        blk = int(t.tables[b, lo // bs])
        t.kc[blk, :lo % bs] = float("nan")
        t.vc[blk, :lo % bs] = float("inf")
        t.tables[b, :lo // bs] = torch.tensor([-1, 2 ** 30, t.nb])[torch.arange(lo // bs) % 3].to(torch.int32).cuda()
    _run(t, begin=begin, softcap=9.0)
    assert bool(torch.isfinite(t.out).all())
    t.check(begin=begin, cap=9.0)


@pytest.mark.parametrize("dtype,d,bs", [("bf16", 128, 16), ("f16", 64, 32), ("bf16", 64, 8)])
def test_nan_and_infinite_keys(dtype, d, bs):
    """An unseen key of NaN or infinity takes no part; a seen one of +inf scores the cap, NaN reaches its rows."""
    t = _batch(dtype, 4, 2, d, bs, [(0, 200)], seed=8)
    t.q.abs_()
    for p, x in ((20, float("nan")), (60, float("inf")), (100, float("-inf")), (150, float("inf"))):
        t.kc[int(t.tables[0, p // bs]), p % bs] = x
    pos = _positions(t)
    begin = torch.where(pos > 40, 21, 0).to(torch.int32)   # the NaN is seen by rows 20 to 40
    _run(t, begin=begin, softcap=6.0)
    t.check(begin=begin, cap=6.0)
    assert bool(torch.isnan(t.out[20:41]).all()) and bool(torch.isfinite(t.out[41:]).all())


@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 8, 8, 64, 32), ("f16", 4, 2, 128, 5)], ids=str)
@pytest.mark.parametrize("size", [1e-6, 1.0, 400.0])
def test_scores_of_any_size(shape, size):
    """Scores near zero, and far beyond the cap and below zero; slopes of both signs."""
    t = _batch(*shape, [(400, 150), (0, 260)], seed=2, q_spread=size)
    for sign in (1.0, -1.0):
        slopes = _slopes(t.hq) * sign
        _run(t, slopes=slopes)
        t.check(slopes=slopes)
    _run(t, softcap=25.0)
    t.check(cap=25.0)
    t.q.abs_()
    t.kc[...] = torch.where(torch.isnan(t.kc), t.kc, -t.kc.abs())   # every score far below zero
    _run(t, window=200)
    t.check(window=200)


@pytest.mark.parametrize("cap", [1e-3, 0.7, 1e4, 1e12])
def test_caps_of_any_size(cap):
    t = _batch("f16", 8, 2, 128, 16, [(100, 140)], seed=6)
    _run(t, softcap=cap)
    t.check(cap=cap)


def test_rows_behind_the_last_sequence_stay():
    t = _batch("bf16", 8, 2, 128, 16, [(50, 20), (0, 130)], seed=5)
    rows = sum(t.chunks)
    q = torch.cat([t.q, t.q[:40]])
    out = torch.full((rows + 40, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pk.paged_prefill_attention_rules(out, q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 130, window=64)
    assert pk.device_error() == 0
    t.check(out=out[:rows], window=64)
    assert bool((out[rows:] == 7.0).all())


def test_one_token_chunks_are_decode():
    t = _batch("bf16", 28, 4, 128, 16, [(n - 1, 1) for n in (1, 16, 129, 700)], seed=1)
    slopes = _slopes(28)
    _run(t, softcap=12.0, slopes=slopes, window=90)
    t.check(cap=12.0, slopes=slopes, window=90)
    out = torch.empty_like(t.out)
    pk.paged_decode_attention_rules(out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, 700, softcap=12.0, slopes=slopes,
                                    window=90)
    t.check(out=out, cap=12.0, slopes=slopes, window=90)


def test_captured_and_replayed():
    """A captured call replayed after its intervals and lengths changed in place."""
    t = _batch("bf16", 8, 2, 128, 16, [(200, 100), (0, 300)], seed=7)
    pos = _positions(t)
    end = (pos + 1).to(torch.int32)
    kw = dict(key_end=end, softcap=15.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 300, **kw)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for shift in (1, 30, -10):
        end.copy_((pos + shift).to(torch.int32))
        t.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        t.check(out=t.out, cap=15.0, end=end)
    assert pk.device_error() == 0


def test_bad_lengths_are_recorded():
    """A table too short for its sequence and chunks past q: recorded, and the rows that could be read are no fault."""
    t = _batch("bf16", 8, 2, 128, 16, [(0, 40), (10, 20)], seed=1)
    lens = t.seq_lens.clone()
    lens[1] = 10 ** 6
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, lens, t.start, t.scale, 40, window=8)
    assert pk.device_error() == 8
    start = t.start.clone()
    start[2] = 1000
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, start, t.scale, 40, window=8)
    assert pk.device_error() == 8
    assert pk.device_error() == 0


def test_many_sequences_of_every_size():
    """A mixed step: 150 sequences, most of one token, some of none, a few chunks among them."""
    g = torch.Generator().manual_seed(3)
    seqs = []
    for i in range(150):
        hist = int(torch.randint(0, 400, (1,), generator=g))
        seqs.append((hist + 1, 0) if i % 7 == 3 else (hist, 300 + i) if i in (31, 32, 90) else (hist, 1 + (i % 5 == 0) * 9))
    t = _batch("bf16", 8, 2, 128, 16, seqs, seed=10)
    t.out.fill_(float("nan"))
    slopes = _slopes(8)
    _run(t, softcap=15.0, slopes=slopes, window=250)
    t.check(cap=15.0, slopes=slopes, window=250)


def test_same_call_same_bits_and_two_streams_at_once():
    a = _batch("bf16", 8, 2, 128, 16, [(900, 300), (0, 500)], seed=1)
    b = _batch("f16", 12, 4, 64, 32, [(100, 800), (50, 77)], seed=2)
    calls = [(a, dict(softcap=20.0, window=300)), (b, dict(slopes=_slopes(12)))]
    for t, kw in calls:
        _run(t, **kw)
    want = [t.out.clone() for t, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for t, _ in calls:
            t.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for (t, kw), s in zip(calls, streams):
            pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, max(t.chunks),
                                             stream=s, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(t.out, w) for (t, _), w in zip(calls, want))
    assert pk.device_error() == 0


@pytest.mark.parametrize("bs", [16, 8])
def test_chunks_longer_than_max_query_len_are_recorded(bs):
    t = _batch("bf16", 8, 2, 128, bs, [(0, 300), (20, 50)], seed=3)
    t.out.fill_(7.0)
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 64, window=90)
    assert pk.device_error() == 8
    t.check(window=90, seqs=[1])
    assert bool((t.out[200:300] == 7.0).all())            # past the reach: as they were


@pytest.mark.parametrize("shape", [("bf16", 32, 8, 128, 16), ("f16", 8, 1, 128, 32), ("bf16", 14, 2, 64, 16)], ids=str)
@pytest.mark.parametrize("window", [0, 5000])
def test_few_rows_over_many_keys(shape, window):
    """A short chunk after a long history: the keys are cut into pieces.  Rows that see all of them, only the newest or
    none; a workspace of the caller's that held NaN."""
    seqs = [(20000, 40), (9000, 3), (5, 1)]
    t = _batch(*shape, seqs, seed=6)
    slopes = _slopes(t.hq)
    _run(t, softcap=30.0, slopes=slopes, window=window)
    t.check(cap=30.0, slopes=slopes, window=window)
    end = (_positions(t) + 1).to(torch.int32)
    end[10:20] = 37                                        # among the oldest keys: most pieces hold no key of theirs
    end[20:23] = 0
    end[40] = 9003
    args = (t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 40)
    ws = pk.prefill_rules_workspace(44, 3, t.hq, t.hkv, t.d, t.bs, t.tables.shape[1], 40, "cuda", window)
    assert ws is not None
    ws.fill_(0xFF)
    pk.paged_prefill_attention_rules(t.out, *args, window=window, key_end=end, workspace=ws)
    assert int(ws[:4].view(torch.int32)[0]) > 1            # it was cut
    t.check(out=t.out, window=window, end=end)
    assert not t.out[20:23].any() and pk.device_error() == 0
    with pytest.raises(pk.KVError) as e:
        pk.paged_prefill_attention_rules(t.out, *args, window=window, key_end=end, workspace=ws[:-16])
    assert e.value.code == "WORKSPACE"
    assert pk.prefill_rules_workspace(44, 3, t.hq, t.hkv, t.d, t.bs, t.tables.shape[1], 40, "cuda", window, True) is None
