"""Rotary embedding with several axes and the cache write, against the
definition: to the bit the float32 oracle's result for a token's own row of
angles, made up pair by pair from its axes' table rows."""

import numpy as np
import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from oracle.fp8_cache import float_to_e4m3_array
from oracle.rope import rotate32
from tests.helpers import sentinel_tensor
from tests.test_gpu_rope_and_cache import CASES, FP8_CASES, MAXPOS, _bits, _case, _dev

pytestmark = pytest.mark.gpu


def _axes(kind, half, seed):
    """(axes, axis of each pair)"""
    rng = np.random.default_rng(seed)
    if kind == "sections":
        side = half * 3 // 8
        return 3, bytes([0] * (half - 2 * side) + [1] * side + [2] * side)
    if kind == "turns":
        return 3, bytes(i % 3 for i in range(half))
    if kind == "four":
        return 4, bytes(rng.integers(0, 4, half).astype(np.uint8))
    if kind == "last":                    # axes that no pair has
        return 4, bytes([3] * half)
    return 1, bytes(half)


def _positions(n, axes, seed):
    pos = np.random.default_rng(seed).integers(0, MAXPOS, (axes, n)).astype(np.int32)
    if n:
        pos[:, 0], pos[-1, 0] = 0, MAXPOS - 1
    return pos


def _rows(table, pos, pair_axes):
    """Each token's own row of cosines and sines."""
    half = len(pair_axes)
    rows = np.empty((pos.shape[1], 2 * half), np.float32)
    for i, a in enumerate(pair_axes):
        rows[:, i], rows[:, half + i] = table[pos[a], i], table[pos[a], half + i]
    return rows


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["sections", "turns", "four", "last", "one"])
@pytest.mark.parametrize("case", [c for c in CASES if c[5] <= 512], ids=lambda c: "-".join(map(str, c)))
def test_axes_are_the_definition(case, kind, interleaved):
    dtype, n, hq, hkv, d, rot, bs, pads, lead = case
    c = _case(dtype, n, hq, hkv, d, rot, bs, pads, seed=n + d + rot, lead=lead)
    axes, pair_axes = _axes(kind, rot // 2, n)
    pos = _positions(n, axes, n + 1)
    dev = torch.device("cuda")
    kc, vc = (sentinel_tensor((c["nb"], bs, hkv, d), dtype, dev) for _ in range(2))
    q_out = sentinel_tensor((n, hq, d), dtype, dev)
    want_k, want_v, want_q = kc.cpu().clone(), vc.cpu().clone(), q_out.cpu().clone()
    pk.device_error()
    got = pk.rope_and_cache_axes(q_out, c["q"], c["k"], c["v"], _dev(pos), pair_axes, _dev(c["table"]), kc, vc,
                                 _dev(c["slots"]), interleaved=interleaved)
    assert got is q_out and pk.device_error() == 0
    real = c["slots"] >= 0
    rows = _rows(c["table"], pos, pair_axes)
    at = torch.from_numpy(c["slots"][real]).long()
    want_q[real] = torch.from_numpy(rotate32(c["q_cpu"].float().numpy(), rows, interleaved)).to(c["dt"])[real]
    want_k.flatten(0, 1)[at] = torch.from_numpy(rotate32(c["k_cpu"].float().numpy(), rows, interleaved)).to(c["dt"])[real]
    want_v.flatten(0, 1)[at] = c["v_cpu"][real]
    for name, a, b in (("q", q_out, want_q), ("k", kc, want_k), ("v", vc, want_v)):
        assert np.array_equal(_bits(a), _bits(b)), name


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["sections", "turns", "four"])
@pytest.mark.parametrize("case", FP8_CASES, ids=lambda c: "-".join(map(str, c)))
def test_axes_fp8_are_the_definition(case, kind, interleaved):
    dtype, n, hq, hkv, d, rot, bs, pads, lead = case
    c = _case(dtype, n, hq, hkv, d, rot, bs, pads, seed=n + d, lead=lead)
    axes, pair_axes = _axes(kind, rot // 2, n)
    pos = _positions(n, axes, n + 1)
    dev = torch.device("cuda")
    kc, vc = (torch.full((c["nb"], bs, hkv, d), 0x7F, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.full((c["nb"], hkv, bs), -1.0, device=dev) for _ in range(2))
    q_out = torch.zeros(n, hq, d, dtype=c["dt"], device=dev)
    pk.device_error()
    pk.rope_and_cache_axes_fp8(q_out, c["q"], c["k"], c["v"], _dev(pos), pair_axes, _dev(c["table"]), kc, vc, ks, vs,
                               _dev(c["slots"]), interleaved=interleaved)
    assert pk.device_error() == 0
    real = np.nonzero(c["slots"] >= 0)[0]
    rows = _rows(c["table"], pos, pair_axes)
    rq = torch.from_numpy(rotate32(c["q_cpu"].float().numpy(), rows, interleaved)).to(c["dt"])
    assert np.array_equal(_bits(q_out[real]), _bits(rq[real]))
    blk, off = c["slots"][real] // bs, c["slots"][real] % bs
    for codes, scales, x in ((kc, ks, rotate32(c["k_cpu"].float().numpy(), rows, interleaved)),
                             (vc, vs, c["v_cpu"].float().numpy())):
        x = x[real]
        amax = np.abs(x).max(-1)
        scale = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
        want = np.full((c["nb"], bs, hkv, d), 0x7F, np.uint8)
        want[blk, off] = float_to_e4m3_array(x / scale[..., None])
        want_s = np.full((c["nb"], hkv, bs), -1.0, np.float32)
        want_s[blk, :, off] = scale
        assert np.array_equal(codes.cpu().numpy(), want)
        assert np.array_equal(scales.cpu().numpy(), want_s)


def test_equal_positions_are_the_single_axis_call():
    c = _case("bf16", 300, 28, 4, 128, 128, 16, 11, seed=3)
    dev = torch.device("cuda")
    caches = [torch.zeros(c["nb"], 16, 4, 128, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    pos, rest = _dev(c["pos"]), (_dev(c["table"]),)
    a, b = (torch.zeros(300, 28, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pk.rope_and_cache(a, c["q"], c["k"], c["v"], pos, *rest, caches[0], caches[1], _dev(c["slots"]))
    pk.rope_and_cache_axes(b, c["q"], c["k"], c["v"], pos.repeat(3, 1), _axes("turns", 64, 0)[1], *rest, caches[2], caches[3],
                           _dev(c["slots"]))
    assert torch.equal(a, b) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("d,hkv", [(128, 2), (72, 1)])
@pytest.mark.parametrize("axis", [0, 2])
@pytest.mark.parametrize("value", [-1, MAXPOS])
def test_a_position_out_of_range_skips_its_token(axis, value, d, hkv):
    c = _case("f16", 6, 4, hkv, d, 16, 16, 0, seed=5)
    pos = _positions(6, 3, 1)
    pos[axis, 2] = value
    dev = torch.device("cuda")
    kc = torch.zeros(c["nb"], 16, hkv, d, dtype=torch.float16, device=dev)
    vc, q_out = torch.zeros_like(kc), torch.zeros(6, 4, d, dtype=torch.float16, device=dev)
    pk.device_error()
    pk.rope_and_cache_axes(q_out, c["q"], c["k"], c["v"], _dev(pos), bytes([0] * 8), _dev(c["table"]), kc, vc,
                           _dev(c["slots"]))
    assert pk.device_error() == 8
    rows = torch.arange(6) != 2
    assert not q_out[2].any() and q_out[rows].any(-1).all()
    assert int(vc.flatten(0, 1).any(-1).any(-1).sum()) == 5 == int(kc.flatten(0, 1).any(-1).any(-1).sum())


def test_axes_in_place_without_queries_and_replayed():
    c = _case("bf16", 40, 8, 2, 128, 128, 16, 4, seed=3, fused=False)
    dev = torch.device("cuda")
    pair_axes = _axes("sections", 64, 0)[1]
    pos = _dev(_positions(40, 3, 5))
    rest = (pos, pair_axes, _dev(c["table"]))
    caches = [torch.zeros(c["nb"], 16, 2, 128, dtype=torch.bfloat16, device=dev) for _ in range(8)]
    slots = _dev(c["slots"])
    out = torch.zeros_like(c["q"])
    pk.rope_and_cache_axes(out, c["q"], c["k"], c["v"], *rest, caches[0], caches[1], slots)
    q = c["q"].clone()
    assert pk.rope_and_cache_axes(q, q, c["k"], c["v"], *rest, caches[2], caches[3], slots) is q
    assert pk.rope_and_cache_axes(None, None, c["k"], c["v"], *rest, caches[4], caches[5], slots) is None
    again = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.rope_and_cache_axes(again, c["q"], c["k"], c["v"], *rest, caches[6], caches[7], slots)
    graph.replay()
    pad = torch.from_numpy(c["slots"] < 0).cuda()
    assert torch.equal(out, again)
    out[pad] = c["q"][pad]
    assert torch.equal(q, out)
    for i in (2, 4, 6):
        assert torch.equal(caches[0], caches[i]) and torch.equal(caches[1], caches[i + 1])
    assert pk.device_error() == 0


def test_axes_wrapper_refusals():
    c = _case("f16", 4, 4, 2, 64, 64, 16, 0, seed=2)
    dev = torch.device("cuda")
    kc = torch.zeros(c["nb"], 16, 2, 64, dtype=torch.float16, device=dev)
    pos = _dev(_positions(4, 3, 1))
    good = dict(q_out=torch.empty(4, 4, 64, dtype=torch.float16, device=dev), q=c["q"], k=c["k"], v=c["v"], positions=pos,
                pair_axes=bytes(i % 3 for i in range(32)), cos_sin=_dev(c["table"]), k_cache=kc,
                v_cache=torch.zeros_like(kc), slot_mapping=_dev(c["slots"]))
    pk.rope_and_cache_axes(**good)
    bad = dict(positions=[pos[0], pos[:, :3], pos.long(), pos.cpu(), pos.T.contiguous().T, pos[:0], pos.repeat(2, 1)],
               pair_axes=[bytes(31), bytes(33), bytes([3] * 32), [0] * 32, None], k=[c["k"].float()], q_out=[None],
               k_cache=[kc.bfloat16()])
    for name, values in bad.items():
        for x in values:
            with pytest.raises(pk.KVError) as e:
                pk.rope_and_cache_axes(**{**good, name: x})
            assert e.value.code == "INVALID_ARG", name
