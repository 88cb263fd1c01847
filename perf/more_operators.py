"""Cases for attention under score rules -- scores capped by a tanh, a bias
that falls with the distance, sliding windows, documents and image spans --
over a paged cache, and for rotary positions with several axes written into
one.

Four operators, each with its plain form in elementary torch operations:

* ``axes`` -- ``rope_and_cache_axes``: the rotary embedding of a step's
  queries and keys, each pair of values by its own axis' position (time,
  height, width), the queries into a buffer, the keys and values into the
  paged cache; ``axes_fp8`` into E4M3 codes and scales;
* ``prefill`` -- ``paged_prefill_attention_rules``: each sequence's chunk
  (its last tokens) over its keys through the block table;
* ``decode`` -- ``paged_decode_attention_rules``: one query token per sequence;
* ``decode_fp8`` -- ``paged_decode_attention_rules_fp8``: the same over E4M3
  codes with one float32 scale per (token, kv head).

A query at position i gives key j the score t(scale q.k) - slope |i - j| with
t(s) = cap tanh(s / cap), and sees the keys of its interval: from the start of
its window or document up to itself, or to the end of its image span.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


def listed():
    return [
        # eight sequences of an image-text model decoding: one token each
        {"name": "axes_decode_8", "op": "axes", "dtype": "bf16", "tokens": 8, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "order": "sections", "interleaved": False, "bs": 32, "pads": 0},
        # the prompt of a few large images
        {"name": "axes_prefill_8192", "op": "axes", "dtype": "bf16", "tokens": 8192, "hq": 28, "hkv": 4, "d": 128,
         "rot": 128, "order": "sections", "interleaved": False, "bs": 16, "pads": 0},
        # a mixed step into an fp8 cache, the axes in turn over the pairs, some padding
        {"name": "axes_fp8_2501", "op": "axes_fp8", "dtype": "bf16", "tokens": 2501, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "order": "turns", "interleaved": False, "bs": 32, "pads": 117},
        # eight chats' next chunks in a layer with a window and capped scores
        {"name": "prefill_cap_window_8x512", "op": "prefill", "dtype": "bf16", "seqs": 8, "chunk": 512,
         "history": 2048, "hq": 32, "hkv": 8, "d": 128, "bs": 32, "cap": 30.0, "slopes": False, "window": 1024,
         "mask": "causal"},
        # a small model with a distance bias in the place of positions, ragged chunks
        {"name": "prefill_slopes_5x300", "op": "prefill", "dtype": "f16", "seqs": 5, "chunk": 300, "history": 1000,
         "hq": 16, "hkv": 16, "d": 64, "bs": 16, "cap": 0.0, "slopes": True, "window": 0, "mask": "causal"},
        # prompts with images, whose tokens see their whole image
        {"name": "prefill_images_3x2500", "op": "prefill", "dtype": "bf16", "seqs": 3, "chunk": 2500, "history": 0,
         "hq": 32, "hkv": 8, "d": 128, "bs": 16, "cap": 50.0, "slopes": False, "window": 0, "mask": "images"},
        # a chunk of a long document in a layer with a window
        {"name": "prefill_window_8192", "op": "prefill", "dtype": "bf16", "seqs": 1, "chunk": 8192, "history": 24576,
         "hq": 28, "hkv": 4, "d": 128, "bs": 16, "cap": 0.0, "slopes": False, "window": 4096, "mask": "causal"},
        # four short sequences of a small model: latency counts
        {"name": "decode_slopes_4x512", "op": "decode", "dtype": "f16", "seqs": 4, "length": 512, "hq": 14, "hkv": 2,
         "d": 64, "bs": 16, "cap": 0.0, "slopes": True, "window": 0, "begins": 0},
        # 64 long conversations in a layer with a window and capped scores
        {"name": "decode_cap_window_64", "op": "decode", "dtype": "bf16", "seqs": 64, "length": 16384, "hq": 32,
         "hkv": 8, "d": 128, "bs": 32, "cap": 30.0, "slopes": False, "window": 4096, "begins": 0},
        # a layer that sees everything, heads of 256, capped scores
        {"name": "decode_cap_d256_32", "op": "decode", "dtype": "bf16", "seqs": 32, "length": 8192, "hq": 16, "hkv": 8,
         "d": 256, "bs": 16, "cap": 50.0, "slopes": False, "window": 0, "begins": 0},
        # keys from the start of the token's own stretch of 8192 positions on, fp8 cache
        {"name": "decode_fp8_stretch_121", "op": "decode_fp8", "dtype": "bf16", "seqs": 121, "length": 20000, "hq": 28,
         "hkv": 4, "d": 128, "bs": 16, "cap": 0.0, "slopes": False, "window": 0, "begins": 8192},
        # long contexts under a distance bias, fp8 cache
        {"name": "decode_fp8_slopes_9", "op": "decode_fp8", "dtype": "f16", "seqs": 9, "length": 40000, "hq": 32,
         "hkv": 8, "d": 128, "bs": 32, "cap": 0.0, "slopes": True, "window": 0, "begins": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 8, 128), (28, 4, 128), (14, 2, 64), (16, 16, 64), (8, 1, 128), (16, 2, 128)])
    op = rng.choice(["axes", "axes_fp8", "prefill", "prefill", "decode", "decode", "decode_fp8"])
    dtype, bs = rng.choice(["bf16", "bf16", "f16"]), rng.choice([16, 32])
    if op in ("axes", "axes_fp8"):
        tokens = _log_int(rng, 1, 8192)
        return {"op": op, "dtype": dtype, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "order": rng.choice(["sections", "turns"]),
                "interleaved": rng.random() < 0.3, "bs": bs, "pads": rng.randint(0, tokens // 8)}
    rules = {"cap": rng.choice([0.0, 20.0, 30.0, 50.0]), "slopes": rng.random() < 0.4,
             "window": rng.choice([0, 0, _log_int(rng, 1, 8192)])}
    if op == "prefill":
        seqs = _log_int(rng, 1, 32)
        chunk = _log_int(rng, 1, 6000 // seqs)
        history = rng.choice([0, _log_int(rng, 1, min(16384, 10000000 // (seqs * chunk)))])
        return {"op": op, "dtype": dtype, "seqs": seqs, "chunk": chunk, "history": history, "hq": hq, "hkv": hkv,
                "d": d, "bs": bs, **rules, "mask": rng.choice(["causal", "causal", "images", "documents"])}
    if op == "decode" and rng.random() < 0.25:
        hq, hkv, d = rng.choice([(16, 8, 256), (8, 1, 256)])
    if op == "decode_fp8":
        hq, hkv, d = rng.choice([(32, 8, 128), (28, 4, 128), (8, 1, 128), (16, 16, 128)])
    seqs = _log_int(rng, 1, 256)
    return {"op": op, "dtype": dtype, "seqs": seqs, "length": _log_int(rng, 1, 262144 // seqs if seqs > 8 else 32768),
            "hq": hq, "hkv": hkv, "d": d, "bs": bs, **rules, "begins": rng.choice([0, 0, 0, 2048])}


def _spread(n, most, g):
    """n lengths from a quarter of `most` up to it, one of them the longest."""
    x = (most * (0.25 + 0.75 * torch.rand(n, generator=g))).long().clamp(min=1)
    x[int(torch.randint(0, n, (1,), generator=g))] = most
    return x


def _sizes(case):
    """Lengths, chunks, and each query's interval of keys (first, one past the last, by position); by the case alone."""
    n = case["seqs"]
    if case["op"] != "prefill":
        g = torch.Generator().manual_seed(n * 1000003 + case["length"])
        lens = _spread(n, case["length"], g)
        chunks, pos = torch.ones(n).long(), lens - 1
    else:
        g = torch.Generator().manual_seed(n * 1000003 + case["chunk"] * 101 + case["history"])
        chunks = _spread(n, case["chunk"], g)
        old = _spread(n, case["history"], g) if case["history"] else torch.zeros(n).long()
        lens = chunks + old
        pos = torch.cat([torch.arange(int(o), int(l)) for o, l in zip(old, lens)])
    begin, end = torch.zeros_like(pos), pos + 1
    if case.get("begins"):
        begin = pos // case["begins"] * case["begins"]
    if case.get("mask") in ("images", "documents"):
        row = 0
        for c in chunks.tolist():
            at = 0
            while at < c:
                size = min(c - at, int(torch.randint(20, 900, (1,), generator=g)))
                if case["mask"] == "documents":
                    begin[row + at:row + at + size] = pos[row + at]
                elif int(torch.randint(0, 2, (1,), generator=g)):
                    end[row + at:row + at + size] = pos[row + at] + size
                at += size
            row += c
    lo = torch.maximum(begin, pos - case["window"] + 1) if case["window"] else begin
    return lens, chunks, pos, begin, end, lo.clamp(min=0)


def _axis_of_pair(case):
    """The axis (time 0, height 1, width 2) of each of the rot / 2 pairs."""
    half = case["rot"] // 2
    if case["order"] == "turns":
        return [i % 3 for i in range(half)]
    side = half * 3 // 8
    return [0] * (half - 2 * side) + [1] * side + [2] * side


FAR = 16384  # rows of the angle table


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] in ("axes", "axes_fp8"):
        n, rot = case["tokens"], case["rot"]
        nb = (n + n // 4) // bs + 2
        # the projection's output, queries, keys and values side by side; keys with the offsets per channel they have
        qkv = randn(n, hq + 2 * hkv, d)
        qkv[:, hq:hq + hkv] += 2 * randn(1, hkv, d)
        qkv = qkv.to(dt)
        slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n].to(torch.int32)
        if case["pads"]:
            slots[torch.randperm(n, generator=g, device=DEV)[:case["pads"]]] = -1
        # an image's tokens share a time and have a row and a column of their own
        positions = torch.randint(0, FAR - 256, (1, n), generator=g, device=DEV)
        positions = (positions + torch.randint(0, 256, (3, n), generator=g, device=DEV)).to(torch.int32)
        angle = torch.arange(FAR, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        axes = _axis_of_pair(case)
        fp8 = case["op"] == "axes_fp8"
        state = {"op": case["op"], "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
                 "q_out": torch.zeros(n, hq, d, dtype=dt, device=DEV), "positions": positions, "pair_axes": bytes(axes),
                 "axes": torch.tensor(axes, device=DEV), "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
                 "slots": slots, "interleaved": case["interleaved"],
                 "k_cache": torch.zeros(nb, bs, hkv, d, dtype=torch.uint8 if fp8 else dt, device=DEV),
                 "v_cache": torch.zeros(nb, bs, hkv, d, dtype=torch.uint8 if fp8 else dt, device=DEV)}
        if fp8:
            state["k_scales"] = torch.zeros(nb, hkv, bs, device=DEV)
            state["v_scales"] = torch.zeros(nb, hkv, bs, device=DEV)
        return state

    lens, chunks, pos, begin, end, lo = _sizes(case)
    B = case["seqs"]
    nblk = (lens + bs - 1) // bs
    most = int(nblk.max()) + 3
    takes = torch.arange(most) < nblk[:, None]
    nb = int(takes.sum()) + 5
    place = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    fresh = torch.cumsum(takes.reshape(-1).long(), 0).reshape(B, most) - 1
    table = torch.where(takes.to(DEV), place[fresh.clamp(min=0).to(DEV)], -1).to(torch.int32).contiguous()
    rows = pos.numel()
    state = {"op": case["op"], "q": (3 * randn(rows, hq, d)).to(dt), "out": torch.zeros(rows, hq, d, dtype=dt, device=DEV),
             "tables": table, "lens": lens.to(torch.int32).to(DEV), "cap": case["cap"], "window": case["window"],
             "scale": d ** -0.5, "longest": int(lens.max()), "pos": pos.to(DEV), "lo": lo.to(DEV), "end": end.to(DEV),
             "slopes": torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) if case["slopes"] else None,
             "key_begin": None, "key_end": None, "host_lens": lens.tolist(), "host_chunks": chunks.tolist(),
             "first": [int(x.min()) for x in lo.split(chunks.tolist())], "most": int((lens - lo).max()) if rows == B else 0}
    if case.get("begins") or case.get("mask") == "documents":
        state["key_begin"] = begin.to(torch.int32).to(DEV)
    if case.get("mask") == "images":
        state["key_end"] = end.to(torch.int32).to(DEV)
    if case["op"] == "prefill":
        state["start"] = torch.cat([torch.zeros(1).long(), chunks.cumsum(0)]).to(torch.int32).to(DEV)
        state["longest_chunk"] = int(chunks.max())
    if case["op"] == "decode_fp8":
        for name in ("k", "v"):
            x = randn(nb, bs, hkv, d)
            scale = x.abs().amax(-1) / 448.0
            state[name + "_cache"] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            state[name + "_scales"] = scale.transpose(1, 2).contiguous()
    else:
        state["k_cache"], state["v_cache"] = randn(nb, bs, hkv, d).to(dt), randn(nb, bs, hkv, d).to(dt)
    return state


def run(s):
    return _axes(s) if s["op"] in ("axes", "axes_fp8") else _prefill(s) if s["op"] == "prefill" else _decode(s)


def _rotate(x, s):
    """x [N, H, D] in float32, its first `rot` values of each head rotated, each pair by its axis' position."""
    half = s["cos_sin"].shape[1] // 2
    pair = torch.arange(half, device=DEV)
    at = s["positions"].long()[s["axes"]].T                     # [N, half]: the position of each pair's axis
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, pair + half][:, None]
    x = x.float()
    rest = x[..., 2 * half:]
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _quantise(x):
    """E4M3 codes (as bytes) and the scale of each row of x: amax / 448, 1 for a row of zeros."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _axes(s):
    fp8 = s["op"] == "axes_fp8"
    if own:
        import paged_kv_cache_128_gb300 as pk
        if fp8:
            pk.rope_and_cache_axes_fp8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["pair_axes"], s["cos_sin"],
                                       s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["slots"],
                                       interleaved=s["interleaved"])
        else:
            pk.rope_and_cache_axes(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["pair_axes"], s["cos_sin"],
                                   s["k_cache"], s["v_cache"], s["slots"], interleaved=s["interleaved"])
    else:
        real = s["slots"] >= 0
        at, dt, bs = s["slots"][real].long(), s["q"].dtype, s["k_cache"].shape[1]
        s["q_out"][real] = _rotate(s["q"], s)[real].to(dt)
        k, v = _rotate(s["k"], s)[real], s["v"][real]
        if fp8:
            k, ks = _quantise(k)
            v, vs = _quantise(v.float())
            s["k_scales"][at // bs, :, at % bs] = ks
            s["v_scales"][at // bs, :, at % bs] = vs
        s["k_cache"].flatten(0, 1)[at] = k.to(s["k_cache"].dtype)
        s["v_cache"].flatten(0, 1)[at] = v
    if fp8:
        return [s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn),
                s["k_scales"], s["v_scales"]]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _weigh(w, s, near, seen):
    """Scores w [Hkv or B Hkv, rows of G heads, keys] into softmax weights, in place: the cap, the bias by `near`
    (slope times distance, or None), the keys of each row's interval."""
    if s["cap"]:
        w = w.div_(s["cap"]).tanh_().mul_(s["cap"])
    if near is not None:
        w = w.sub_(near)
    w = w.masked_fill_(~seen, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return w.div_(w.sum(-1, keepdim=True).clamp(min=1e-30))


def _prefill(s):
    if own:
        import paged_kv_cache_128_gb300 as pk
        return pk.paged_prefill_attention_rules(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["start"], s["scale"],
            s["longest_chunk"], softcap=s["cap"], slopes=s["slopes"], window=s["window"], key_begin=s["key_begin"],
            key_end=s["key_end"])
    hq, d = s["q"].shape[1:]
    bs, hkv = s["k_cache"].shape[1:3]
    G, row = hq // hkv, 0
    for b, (n, L, first) in enumerate(zip(s["host_chunks"], s["host_lens"], s["first"])):
        j = torch.arange(first, L, device=DEV)
        slot = s["tables"][b].long()[j // bs] * bs + j % bs
        k = s["k_cache"].flatten(0, 1)[slot].float().permute(1, 2, 0)            # [Hkv, D, keys]
        v = s["v_cache"].flatten(0, 1)[slot].float().transpose(0, 1)
        rows = slice(row, row + n)
        row += n
        q = (s["q"][rows].float() * s["scale"]).view(n, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * n, d)
        seen = (j >= s["lo"][rows, None]) & (j < s["end"][rows, None])           # [n, keys]
        near = None
        if s["slopes"] is not None:
            far = (s["pos"][rows, None] - j).abs().float()
            near = s["slopes"].view(hkv, G, 1, 1) * far
        w = (q @ k).view(hkv, G, n, -1)
        w = _weigh(w, s, near, seen).view(hkv, G * n, -1)
        s["out"][rows] = (w @ v).view(hkv, G, n, d).permute(2, 0, 1, 3).reshape(n, hq, d).to(s["out"].dtype)
    return s["out"]


def _decode(s):
    B, hq, d = s["q"].shape
    bs, hkv = s["k_cache"].shape[1:3]
    fp8 = s["op"] == "decode_fp8"
    if own:
        import paged_kv_cache_128_gb300 as pk
        if "workspace" not in s:  # kept between calls, as a serving loop keeps it
            plan = pk.decode_plan(B, hq, hkv, d, bs, s["longest"], s["q"].dtype)
            s["workspace"] = pk.alloc_workspace(plan, s["q"].device)
        rules = {"softcap": s["cap"], "slopes": s["slopes"], "window": s["window"], "key_begin": s["key_begin"],
                 "workspace": s["workspace"]}
        if fp8:
            return pk.paged_decode_attention_rules_fp8(
                s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"], s["lens"],
                s["scale"], s["longest"], **rules)
        return pk.paged_decode_attention_rules(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                               s["scale"], s["longest"], **rules)
    # the keys of each sequence's interval, from its first one on
    j = s["lo"][:, None] + torch.arange(s["most"], device=DEV)
    seen = j <= s["pos"][:, None]
    at = j.clamp(max=s["tables"].shape[1] * bs - 1)
    slot = s["tables"].long().gather(1, at // bs).clamp(min=0) * bs + at % bs
    kv = []
    for name in ("k", "v"):
        x = s[name + "_cache"].flatten(0, 1)
        if fp8:
            x = x.view(torch.float8_e4m3fn)[slot].float() * s[name + "_scales"].transpose(1, 2).flatten(0, 1)[slot][..., None]
        else:
            x = x[slot].float()
        kv.append(x.transpose(1, 2))                                             # [B, Hkv, keys, D]
    k, v = kv
    q = (s["q"].float() * s["scale"]).view(B, hkv, hq // hkv, d)
    near = None
    if s["slopes"] is not None:
        near = s["slopes"].view(hkv, -1, 1) * (s["pos"][:, None] - j).abs().float()[:, None, None]
    w = _weigh(q @ k.transpose(-1, -2), s, near, seen[:, None, None])
    s["out"].copy_((w @ v).view(B, hq, d))
    return s["out"]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("axes", "axes_fp8"):
        n = case["tokens"] - case["pads"]
        kept = hkv * (d + 4) if case["op"] == "axes_fp8" else hkv * d * 2
        rows = min(3 * n, FAR)                         # rows of the angle table that can be asked for
        moved = n * (4 * hq * d + 4 * hkv * d + 2 * kept) + rows * case["rot"] * 4 // (3 if 3 * n <= FAR else 1)
        return {"bytes": moved + 12 * n + 4 * case["tokens"], "flops": 3 * n * (hq + hkv) * case["rot"]}
    lens, chunks, pos, begin, end, lo = _sizes(case)
    pairs = int((end - lo).sum())
    # keys that some query of the sequence sees
    first = torch.stack([x.min() for x in lo.split(chunks.tolist())])
    keys = int((lens - first).sum())
    per_key = 2 * hkv * (d + 4) if case["op"] == "decode_fp8" else 4 * hkv * d
    return {"bytes": keys * per_key + 4 * pos.numel() * hq * d + 4 * keys // case["bs"], "flops": pairs * hq * d * 4}


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if case["op"] in ("axes", "axes_fp8"):
        half = case["rot"] // 2
        # the angles are those of the float32 table, which is an input
        cos, sin = torch.zeros(2, case["tokens"], 1, half, dtype=torch.float64, device=DEV)
        for i, axis in enumerate(_axis_of_pair(case)):
            rows = s["cos_sin"].double()[s["positions"][axis].long()]
            cos[:, 0, i], sin[:, 0, i] = rows[:, i], rows[:, half + i]
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)

        def turn(x):
            y = x.double().clone()
            z = torch.complex(y[..., a], y[..., b]) * torch.complex(cos, sin)
            y[..., a], y[..., b] = z.real, z.imag
            return y

        real = torch.nonzero(s["slots"] >= 0)[:, 0]
        blk, off = s["slots"][real].long() // bs, s["slots"][real].long() % bs
        q_out = s["q_out"].double()
        q_out[real] = turn(s["q"])[real]
        outs, scales = [q_out], []
        for x in (turn(s["k"])[real], s["v"].double()[real]):
            c = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV)
            if case["op"] == "axes_fp8":
                amax = x.abs().amax(-1)
                scale = torch.where(amax > 0, amax / 448.0, 1.0)
                x = x / scale[..., None]
                # E4M3: three bits after the leading one, steps of 2^-9 below 2^-6, nearest, ties to even
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                x = torch.round(x / step) * step
                z = torch.zeros(s["k_scales"].shape, dtype=torch.float64, device=DEV)
                z[blk, :, off] = scale
                scales.append(z)
            c[blk, off] = x
            outs.append(c)
        return outs + scales

    lens, chunks, pos, begin, end, lo = _sizes(case)
    out = torch.zeros(pos.numel(), hq, d, dtype=torch.float64, device=DEV)
    row = 0
    for b in range(case["seqs"]):
        L, n, first = int(lens[b]), int(chunks[b]), s["first"][b]
        blocks = s["tables"][b, :(L + bs - 1) // bs].long()
        k, v = [s[name][blocks].reshape(-1, hkv, d) if case["op"] != "decode_fp8" else
                s[name][blocks].view(torch.float8_e4m3fn).double().reshape(-1, hkv, d)
                for name in ("k_cache", "v_cache")]
        if case["op"] == "decode_fp8":
            k, v = [x * s[name][blocks].double().transpose(1, 2).reshape(-1, hkv, 1)
                    for x, name in ((k, "k_scales"), (v, "v_scales"))]
        key = torch.arange(first, L, device=DEV)
        i = pos[row:row + n].to(DEV)[:, None]
        hidden = (key < lo[row:row + n].to(DEV)[:, None]) | (key >= end[row:row + n].to(DEV)[:, None])
        for h in range(hq):
            kh, vh = k[first:L, h * hkv // hq].double(), v[first:L, h * hkv // hq].double()
            t = s["q"][row:row + n, h].double() @ kh.T * (1.0 / math.sqrt(d))
            if case["cap"]:
                t = case["cap"] * torch.tanh(t / case["cap"])
            if case["slopes"]:
                t = t - s["slopes"][h].double() * (i - key).abs()
            out[row:row + n, h] = torch.softmax(t.masked_fill(hidden, -math.inf), -1) @ vh
        row += n
    return out
