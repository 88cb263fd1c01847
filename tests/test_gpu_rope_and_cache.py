"""Rotary embedding with the cache write against the definition.

The result is defined to the bit (float32 products and sums, one rounding),
so q_out and the whole caches must equal the float32 oracle's bits; the
float64 formula bounds it too, with the roundings counted.  Cases: fp32,
fp16, bf16; both pairings; partial rotation; head sizes and alignments that
take the vector kernel and those that take the other; padded tokens; strided
q, k, v of one fused tensor; one token; none.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from oracle.fp8_cache import float_to_e4m3_array
from oracle.rope import angle_table, rotate32, rotate64
from tests.helpers import TORCH, sentinel_tensor

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest subnormal
MAXPOS = 4000


def _bits(t):
    return t.detach().cpu().contiguous().view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()]).numpy()


def _case(dtype, n, hq, hkv, d, rot, bs, pads, seed, lead=0, fused=True):
    """Inputs on the GPU and what the definition gives, as torch CPU tensors.
    lead: elements before q in the fused tensor (shifts its alignment)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = TORCH[dtype]
    nb = (n + bs - 1) // bs + 3
    width = (hq + 2 * hkv) * d + lead
    qkv = (torch.randn(max(n, 1), width, generator=g) * 2).to(dt)[:n]
    qkv_dev = qkv.cuda()

    def part(t, first, heads):
        return t[:, lead + first * d:lead + (first + heads) * d].unflatten(1, (heads, d))

    if not fused:
        q, k, v = (part(qkv_dev, a, b).contiguous() for a, b in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    else:
        q, k, v = (part(qkv_dev, a, b) for a, b in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    slots = rng.permutation(nb * bs)[:n].astype(np.int32)
    slots[rng.permutation(n)[:pads]] = -1
    pos = rng.integers(0, MAXPOS, n).astype(np.int32)
    if n:
        pos[0] = MAXPOS - 1
    table = angle_table(MAXPOS, rot)
    return dict(q=q, k=k, v=v, q_cpu=part(qkv, 0, hq), k_cpu=part(qkv, hq, hkv), v_cpu=part(qkv, hq + hkv, hkv),
                slots=slots, pos=pos, table=table, nb=nb, dt=dt)


def _dev(a):
    return torch.from_numpy(a).cuda()


CASES = [  # dtype, tokens, Hq, Hkv, D, rot, bs, pads, lead
    ("bf16", 1, 32, 8, 128, 128, 32, 0, 0),
    ("bf16", 37, 32, 8, 128, 128, 16, 5, 0),
    ("f16", 200, 14, 2, 64, 64, 16, 13, 0),
    ("f16", 65, 14, 2, 64, 32, 16, 0, 0),
    ("f32", 33, 4, 2, 128, 96, 8, 3, 0),
    ("f32", 5, 2, 1, 8, 8, 4, 1, 0),          # head_dim 8: the kernel for any size
    ("bf16", 29, 3, 1, 80, 80, 16, 2, 0),     # five lanes a head
    ("bf16", 31, 5, 5, 96, 64, 16, 0, 0),
    ("f16", 23, 6, 3, 72, 20, 5, 2, 0),       # rot 20, head_dim 72, blocks of 5
    ("bf16", 19, 8, 2, 128, 128, 16, 1, 1),   # rows one element off every 16-byte boundary
    ("f16", 17, 8, 2, 128, 2, 16, 0, 0),      # a single pair
    ("bf16", 9, 4, 2, 256, 256, 32, 0, 0),
    ("bf16", 1500, 32, 8, 128, 128, 16, 70, 0),  # one CTA walks a token's heads
    ("f32", 1300, 28, 4, 64, 64, 16, 0, 0),
    ("bf16", 3, 200, 8, 64, 64, 16, 0, 0),    # several rounds of heads side by side
    ("bf16", 1400, 200, 8, 64, 64, 16, 0, 0),  # and one after another
    ("f16", 4, 2, 1, 2048, 2048, 2, 0, 0),
    ("f16", 4, 2, 1, 2064, 16, 2, 0, 0),
    ("bf16", 0, 4, 2, 64, 64, 16, 0, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_and_cache_is_the_definition(case, interleaved):
    dtype, n, hq, hkv, d, rot, bs, pads, lead = case
    c = _case(dtype, n, hq, hkv, d, rot, bs, pads, seed=n + d + rot, lead=lead)
    dev = torch.device("cuda")
    kc, vc = (sentinel_tensor((c["nb"], bs, hkv, d), dtype, dev) for _ in range(2))
    want_k, want_v = kc.cpu().clone(), vc.cpu().clone()
    q_out = sentinel_tensor((n, hq, d), dtype, dev)
    want_q = q_out.cpu().clone()
    pk.device_error()
    got = pk.rope_and_cache(q_out, c["q"], c["k"], c["v"], _dev(c["pos"]), _dev(c["table"]), kc, vc, _dev(c["slots"]),
                            interleaved=interleaved)
    assert got is q_out and pk.device_error() == 0
    real = c["slots"] >= 0
    rows = c["table"][c["pos"]]
    rq = rotate32(c["q_cpu"].float().numpy(), rows, interleaved)
    rk = rotate32(c["k_cpu"].float().numpy(), rows, interleaved)
    want_q[real] = torch.from_numpy(rq).to(c["dt"])[real]
    at = torch.from_numpy(c["slots"][real]).long()
    want_k.flatten(0, 1)[at] = torch.from_numpy(rk).to(c["dt"])[real]
    want_v.flatten(0, 1)[at] = c["v_cpu"][real]
    for name, a, b in (("q", q_out, want_q), ("k", kc, want_k), ("v", vc, want_v)):
        assert np.array_equal(_bits(a), _bits(b)), name
    # the formula in 64 bits: two products and a sum in float32, each off by half a step of at most
    # |a c| + |b s| <= 2 max|x| (three of them, and the float32 tables are the inputs), then the output's rounding
    if real.any():
        for x, out in ((c["q_cpu"], q_out.cpu()[real]), (c["k_cpu"], kc.cpu().flatten(0, 1)[at])):
            ref = rotate64(x.double().numpy(), rows, interleaved)[real]
            err = np.abs(out.double().numpy() - ref)
            big = 2 * float(x.abs().max())
            step = HALF_STEP[dtype] if dtype != "f32" else 0.0
            assert np.all(err <= 3 * 2.0 ** -24 * big + step * (np.abs(ref) + 3 * 2.0 ** -24 * big) + TINY[dtype])


def test_rope_in_place_and_without_queries():
    c = _case("bf16", 40, 8, 2, 128, 128, 16, 4, seed=3, fused=False)
    dev = torch.device("cuda")

    def caches():
        return [torch.zeros(c["nb"], 16, 2, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]

    rest = (_dev(c["pos"]), _dev(c["table"]))
    k1, v1 = caches()
    out = torch.zeros_like(c["q"])
    pk.rope_and_cache(out, c["q"], c["k"], c["v"], *rest, k1, v1, _dev(c["slots"]))
    k2, v2 = caches()
    q = c["q"].clone()
    assert pk.rope_and_cache(q, q, c["k"], c["v"], *rest, k2, v2, _dev(c["slots"])) is q
    pad = torch.from_numpy(c["slots"] < 0).cuda()
    out[pad] = c["q"][pad]                       # in place a padded token keeps its query
    assert torch.equal(q, out) and torch.equal(k1, k2) and torch.equal(v1, v2)
    k3, v3 = caches()
    assert pk.rope_and_cache(None, None, c["k"], c["v"], *rest, k3, v3, _dev(c["slots"])) is None
    assert torch.equal(k1, k3) and torch.equal(v1, v3)
    assert pk.device_error() == 0


@pytest.mark.parametrize("d,hkv", [(128, 2), (72, 1)])
@pytest.mark.parametrize("field,value", [("pos", -1), ("pos", MAXPOS), ("slots", -2), ("slots", 10 ** 6)])
def test_rope_out_of_range_is_recorded_and_skipped(field, value, d, hkv):
    c = _case("f16", 6, 4, hkv, d, 16, 16, 0, seed=5)
    c[field][2] = value
    dev = torch.device("cuda")
    kc = torch.zeros(c["nb"], 16, hkv, d, dtype=torch.float16, device=dev)
    vc, q_out = torch.zeros_like(kc), torch.zeros(6, 4, d, dtype=torch.float16, device=dev)
    pk.device_error()
    pk.rope_and_cache(q_out, c["q"], c["k"], c["v"], _dev(c["pos"]), _dev(c["table"]), kc, vc, _dev(c["slots"]))
    assert pk.device_error() == 8
    assert pk.device_error() == 0
    rows = torch.arange(6) != 2
    assert not q_out[2].any() and q_out[rows].any(-1).all()
    assert int(vc.flatten(0, 1).any(-1).any(-1).sum()) == 5 == int(kc.flatten(0, 1).any(-1).any(-1).sum())


FP8_CASES = [  # dtype, tokens, Hq, Hkv, D, rot, bs, pads, lead
    ("bf16", 1, 32, 8, 128, 128, 32, 0, 0),
    ("f16", 50, 14, 2, 64, 64, 16, 7, 0),
    ("bf16", 43, 28, 4, 128, 64, 16, 3, 0),
    ("f16", 21, 8, 3, 256, 256, 16, 0, 0),
    ("bf16", 1400, 32, 8, 128, 128, 32, 60, 0),
    ("bf16", 27, 8, 2, 128, 128, 16, 2, 1),
    ("f16", 27, 5, 1, 64, 10, 16, 2, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", FP8_CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_and_cache_fp8_is_the_definition(case, interleaved):
    dtype, n, hq, hkv, d, rot, bs, pads, lead = case
    c = _case(dtype, n, hq, hkv, d, rot, bs, pads, seed=n + d, lead=lead)
    c["k"][n // 2, 0] = 0                        # a row of zeros has scale 1
    c["k_cpu"][n // 2, 0] = 0
    dev = torch.device("cuda")
    kc, vc = (torch.full((c["nb"], bs, hkv, d), 0x7F, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.full((c["nb"], hkv, bs), -1.0, device=dev) for _ in range(2))
    q_out = torch.zeros(n, hq, d, dtype=c["dt"], device=dev)
    pk.device_error()
    pk.rope_and_cache_fp8(q_out, c["q"], c["k"], c["v"], _dev(c["pos"]), _dev(c["table"]), kc, vc, ks, vs,
                          _dev(c["slots"]), interleaved=interleaved)
    assert pk.device_error() == 0
    real = np.nonzero(c["slots"] >= 0)[0]
    rows = c["table"][c["pos"]]
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


def test_rope_fp8_then_plain_fp8_write_agree_at_position_zero():
    """At position 0 nothing turns: the fp8 write's own codes and scales."""
    c = _case("bf16", 33, 8, 2, 128, 128, 16, 2, seed=9)
    dev = torch.device("cuda")
    pos = torch.zeros(33, dtype=torch.int32, device=dev)

    def pool():
        return [torch.zeros(c["nb"], 16, 2, 128, dtype=torch.uint8, device=dev) for _ in range(2)] + \
            [torch.zeros(c["nb"], 2, 16, device=dev) for _ in range(2)]

    a, b = pool(), pool()
    q_out = torch.empty_like(c["q"].contiguous())
    pk.rope_and_cache_fp8(q_out, c["q"], c["k"], c["v"], pos, _dev(c["table"]), *a, _dev(c["slots"]))
    pk.reshape_and_cache_fp8(c["k"], c["v"], *b, _dev(c["slots"]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rope_captured_replayed_and_on_another_stream():
    c = _case("bf16", 64, 32, 8, 128, 128, 32, 0, seed=11)
    dev = torch.device("cuda")
    kc = torch.zeros(c["nb"], 32, 8, 128, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    q_out = torch.zeros(64, 32, 128, dtype=torch.bfloat16, device=dev)
    pos, table, slots = _dev(c["pos"]), _dev(c["table"]), _dev(c["slots"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pk.rope_and_cache(q_out, c["q"], c["k"], c["v"], pos, table, kc, vc, slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (q_out, kc, vc)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.rope_and_cache(q_out, c["q"], c["k"], c["v"], pos, table, kc, vc, slots)
    for t in (q_out, kc, vc):
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((q_out, kc, vc), want))
    # new positions in the captured buffers are what the next replay reads
    pos.copy_(torch.flip(pos, (0,)))
    graph.replay()
    rows = c["table"][c["pos"][::-1]]
    ref = torch.from_numpy(rotate32(c["q_cpu"].float().numpy(), rows, False)).bfloat16()
    assert torch.equal(q_out.cpu(), ref)


def test_rope_wrapper_refusals():
    c = _case("f16", 4, 4, 2, 64, 64, 16, 0, seed=2)
    dev = torch.device("cuda")
    kc = torch.zeros(c["nb"], 16, 2, 64, dtype=torch.float16, device=dev)
    good = dict(q_out=torch.empty(4, 4, 64, dtype=torch.float16, device=dev), q=c["q"], k=c["k"], v=c["v"],
                positions=_dev(c["pos"]), cos_sin=_dev(c["table"]), k_cache=kc, v_cache=torch.zeros_like(kc),
                slot_mapping=_dev(c["slots"]))
    pk.rope_and_cache(**good)
    bad = dict(q_out=[None, good["q_out"][:3], good["q_out"].float(), good["q_out"].cpu()], q=[c["q"][:, :, :32]],
               k=[c["k"].cpu(), c["k"].float(), c["k"][:3]], v=[c["v"][:, :1]],
               positions=[good["positions"].long(), good["positions"][:3]],
               cos_sin=[good["cos_sin"].half(), good["cos_sin"][0], good["cos_sin"][:, :63].contiguous(),
                        torch.zeros(8, 66, device=dev)],
               k_cache=[kc.bfloat16(), kc[:, :, :, :32], kc[:1]], slot_mapping=[good["slot_mapping"].long()])
    for name, values in bad.items():
        for x in values:
            with pytest.raises(pk.KVError) as e:
                pk.rope_and_cache(**{**good, name: x})
            assert e.value.code == "INVALID_ARG", name


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 2), (6, 1, 1), (1, 1, 1)])
def test_rope_one_token_or_one_head_of_a_transposed_tensor(n, hq, hkv):
    """[heads, tokens, D] transposed: dense rows whose other stride (of a
    single token, of a single head) is not that of a dense [N, H, D]."""
    c = _case("bf16", n, hq, hkv, 64, 64, 16, 0, seed=5)
    dev = torch.device("cuda")

    def turned(t):
        t = t.transpose(0, 1).clone(memory_format=torch.contiguous_format)
        if t.shape[0] == 1:  # a single head: one of a larger tensor, its own stride 2 N D
            t = torch.cat([t, t], 1)[:, :n]
        return t.transpose(0, 1)

    rest = (_dev(c["pos"]), _dev(c["table"]))
    caches = [torch.zeros(c["nb"], 16, hkv, 64, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    q, k, v = (turned(c[x]) for x in "qkv")
    assert q.stride()[:2] != (hq * 64, 64) and k.stride()[:2] != (hkv * 64, 64)
    a = pk.rope_and_cache(torch.zeros_like(c["q"].contiguous()), c["q"].contiguous(), c["k"].contiguous(),
                          c["v"].contiguous(), *rest, caches[0], caches[1], _dev(c["slots"]))
    b = pk.rope_and_cache(torch.zeros_like(q), q, k, v, *rest, caches[2], caches[3], _dev(c["slots"]))
    assert torch.equal(a, b) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert pk.device_error() == 0
