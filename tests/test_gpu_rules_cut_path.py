"""Prefill under score rules whose keys are cut into pieces: NaN and infinite
scores in some pieces, replays of a captured call, and small fp16 weights, on
the whole path as well."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import attention64, check_rows
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu

LN2 = 0.6931471805599453


def _cut_workspace(t, most):
    return pk.prefill_rules_workspace(sum(t.chunks), len(t.lens), t.hq, t.hkv, t.d, t.bs, t.tables.shape[1], most, "cuda")


def _pieces(ws):
    return int(ws[:4].view(torch.int32)[0])


@pytest.mark.parametrize("dtype, d, bs", [("bf16", 128, 16), ("f16", 64, 32)])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_nan_and_infinite_scores_reach_their_rows(dtype, d, bs, cap):
    """Keys of NaN, -inf and, under a cap, +inf far apart, so that they lie in different pieces; rows that end before
    the NaN do not have it."""
    t = PagedBatch(dtype, 8, 2, d, bs, [20040], [40], seed=8)
    t.q.copy_(t.q.abs() + 0.125)
    for p, x in ((3000, float("-inf")), (9000, float("inf") if cap else float("-inf")), (12000, float("nan"))):
        t.kc[int(t.tables[0, p // bs]), p % bs] = x
    end = torch.arange(20001, 20041, dtype=torch.int32, device="cuda")
    end[:25] = 11999
    end[30] = 3001
    ws = _cut_workspace(t, 40)
    ws.fill_(0xFF)
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 40, softcap=cap,
                                     key_end=end, workspace=ws)
    assert pk.device_error() == 0 and _pieces(ws) > 1
    t.check(cap=cap, end=end)
    nan = torch.isnan(t.out).all(-1).all(-1)
    assert bool(nan[31:].all()) and bool(nan[25:30].all()) and not bool(nan[:25].any()) and not bool(nan[30])


def test_a_cut_call_captured_and_replayed():
    t = PagedBatch("bf16", 8, 2, 128, 16, [12040, 9002], [40, 2], seed=7)
    end = torch.cat([torch.arange(12001, 12041), torch.arange(9001, 9003)]).to(torch.int32).cuda()
    first = end.clone()
    ws = _cut_workspace(t, 40)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 40,
                                                    softcap=15.0, key_end=end, workspace=ws)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    pk.device_error()
    for shift in (0, -30, -5000):
        end.copy_(first + shift)
        ws.fill_(0xFF)
        t.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert _pieces(ws) > 1
        t.check(cap=15.0, end=end)
    assert pk.device_error() == 0


@pytest.mark.parametrize("top", [-7.9, 0.0, 7.0, -40.0])
@pytest.mark.parametrize("d, bs", [(64, 16), (128, 64), (64, 8)])
@pytest.mark.parametrize("ctx", [220, 6060])
def test_small_weights_count(d, bs, top, ctx):
    """Every 16 keys hold one of the largest score and value 0 and 15 of value 1000 whose weight is 2^-17.5 of it."""
    dev = torch.device("cuda")
    hq, hkv, n = 4, 2, 100
    L = n + ctx
    nb = -(-L // bs)
    pos = torch.arange(nb * bs, device=dev)
    k = torch.zeros(nb * bs, hkv, d, device=dev)
    k[..., 0] = torch.where(pos % 16 == 0, top * LN2, (top - 17.5) * LN2)[:, None]
    v = torch.where(pos % 16 == 0, 0.0, 1000.0)[:, None, None].expand(-1, hkv, d)
    kc, vc = k.half().view(nb, bs, hkv, d), v.half().contiguous().view(nb, bs, hkv, d)
    tables = torch.arange(nb, dtype=torch.int32, device=dev).view(1, nb)
    q = torch.zeros(n, hq, d, dtype=torch.float16, device=dev)
    q[..., 0] = 1
    out = torch.full_like(q, float("nan"))
    ws = pk.prefill_rules_workspace(n, 1, hq, hkv, d, bs, nb, n, dev)
    pk.device_error()
    pk.paged_prefill_attention_rules(out, q, kc, vc, tables, torch.tensor([L], dtype=torch.int32, device=dev),
                                     torch.tensor([0, n], dtype=torch.int32, device=dev), 1.0, n, workspace=ws)
    assert pk.device_error() == 0
    if ctx > 5000 and bs >= 16:
        assert _pieces(ws) > 1
    seen = torch.arange(L, device=dev) <= torch.arange(ctx, L, device=dev)[:, None]
    for h in range(hq):
        o, tol = attention64(q[:, h], kc.view(-1, hkv, d)[:L, h // 2], vc.view(-1, hkv, d)[:L, h // 2], 1.0, "f16", seen)
        check_rows(out[:, h], o, tol, h)
