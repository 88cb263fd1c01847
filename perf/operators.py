"""Cases for the position rotation fused with the cache write, and for decode
attention over a prefix that a group of sequences shares.

Three operators, each with its plain form in elementary torch operations:

* ``rope`` -- ``rope_and_cache``: the rotary position embedding of a step's
  queries and keys, the queries into a buffer of their own, the keys and the
  values into the paged cache at their slots;
* ``rope_fp8`` -- ``rope_and_cache_fp8``: the same with the keys and values
  quantised to E4M3 codes and one float32 scale per (token, kv head);
* ``shared`` -- ``paged_decode_attention_shared_prefix``: one query token per
  sequence over the sequence's whole block table, where consecutive sequences
  form groups whose first tokens lie in the same blocks.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # eight sequences decoding: one token each, the smallest call of a serving loop
        {"name": "rope_decode_8", "op": "rope", "dtype": "bf16", "tokens": 8, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "bs": 32, "pads": 0, "far": 8192},
        # a mixed step: 256 decode tokens, a 4096-token prefill chunk and 5 % padding
        {"name": "rope_mixed_4581", "op": "rope", "dtype": "bf16", "tokens": 4581, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "bs": 32, "pads": 229, "far": 8192},
        # a small model's prefill, adjacent pairs rotated, half of each head left as it is
        {"name": "rope_partial_2047", "op": "rope", "dtype": "f16", "tokens": 2047, "hq": 14, "hkv": 2, "d": 64,
         "rot": 32, "interleaved": True, "bs": 16, "pads": 31, "far": 2048},
        # the prefill of a long document in one chunk
        {"name": "rope_prefill_32768", "op": "rope", "dtype": "bf16", "tokens": 32768, "hq": 28, "hkv": 4, "d": 128,
         "rot": 128, "interleaved": False, "bs": 16, "pads": 0, "far": 65536},
        # 64 sequences decoding into an fp8 cache
        {"name": "rope_fp8_decode_64", "op": "rope_fp8", "dtype": "bf16", "tokens": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "bs": 32, "pads": 0, "far": 8192},
        # the mixed step into an fp8 cache
        {"name": "rope_fp8_mixed_4581", "op": "rope_fp8", "dtype": "bf16", "tokens": 4581, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "bs": 32, "pads": 229, "far": 8192},
        # four samples of one prompt just begun on a small model: latency counts
        {"name": "shared_4x512", "op": "shared", "dtype": "f16", "seqs": 4, "groups": 1, "hq": 14, "hkv": 2, "d": 64,
         "bs": 16, "prefix": 517, "suffix": 16},
        # a chat server: every request begins with the same 4096-token system prompt
        {"name": "shared_64x4096", "op": "shared", "dtype": "bf16", "seqs": 64, "groups": 1, "hq": 32, "hkv": 8,
         "d": 128, "bs": 16, "prefix": 4096, "suffix": 1024},
        # several tools' prompts side by side, groups of uneven size, some of them of one sequence
        {"name": "shared_9_groups", "op": "shared", "dtype": "bf16", "seqs": 121, "groups": 9, "hq": 28, "hkv": 4,
         "d": 128, "bs": 32, "prefix": 2500, "suffix": 700},
        # a few questions about one long document: the shared part is nearly all there is to read
        {"name": "shared_7x32768", "op": "shared", "dtype": "bf16", "seqs": 7, "groups": 1, "hq": 32, "hkv": 8,
         "d": 128, "bs": 16, "prefix": 32768, "suffix": 300},
        # many samples of one prompt: more query rows to each key than the memory needs
        {"name": "shared_256x8192", "op": "shared", "dtype": "bf16", "seqs": 256, "groups": 1, "hq": 32, "hkv": 8,
         "d": 128, "bs": 32, "prefix": 8192, "suffix": 512},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 8, 128), (28, 4, 128), (14, 2, 64), (16, 16, 64), (8, 1, 128), (16, 2, 128)])
    op = rng.choice(["rope", "rope_fp8", "shared", "shared"])
    bs = rng.choice([16, 32])
    if op != "shared":
        dtype = rng.choice(["bf16", "f16", "f32"] if op == "rope" else ["bf16", "f16"])
        tokens = _log_int(rng, 1, 8192 if dtype == "f32" else 16384)
        return {"op": op, "dtype": dtype, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.3, "bs": bs,
                "pads": rng.randint(0, tokens // 8), "far": rng.choice([2048, 8192, 65536])}
    seqs = _log_int(rng, 2, 256)
    groups = min(seqs, rng.choice([1, 1, 2, 5, 12]))
    return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "seqs": seqs, "groups": groups, "hq": hq, "hkv": hkv,
            "d": d, "bs": bs, "prefix": _log_int(rng, 32, min(32768 // groups, 8192 * 256 // seqs)),
            "suffix": _log_int(rng, 1, 512)}


def _sizes(case):
    """Group bounds, prefix lengths and sequence lengths of a shared case; they go by the case alone."""
    g = torch.Generator().manual_seed(case["seqs"] * 1000003 + case["prefix"])
    B, NG = case["seqs"], case["groups"]
    cuts = torch.randperm(B - 1, generator=g)[:NG - 1].add(1).sort().values if NG > 1 else torch.zeros(0).long()
    start = torch.cat([torch.zeros(1).long(), cuts, torch.full((1,), B).long()])
    share = torch.ones(NG) if NG == 1 else torch.rand(NG, generator=g) * 1.2 + 0.1
    prefix = (share * case["prefix"]).long().clamp(min=1)
    # suffix lengths: one token to `suffix`, spread over their logarithm as conversations are
    suffix = torch.exp(torch.rand(B, generator=g) * math.log(case["suffix"] + 0.5)).long().clamp(1, case["suffix"])
    return start, prefix, prefix.repeat_interleave(start.diff()) + suffix


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] != "shared":
        n, rot = case["tokens"], case["rot"]
        nb = (n + n // 4) // bs + 2
        # the projection's output, queries, keys and values side by side; keys with the offsets per channel they have
        qkv = randn(n, hq + 2 * hkv, d)
        qkv[:, hq:hq + hkv] += 2 * randn(1, hkv, d)
        qkv = qkv.to(dt)
        slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n].to(torch.int32)
        if case["pads"]:
            slots[torch.randperm(n, generator=g, device=DEV)[:case["pads"]]] = -1
        positions = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        angle = torch.arange(case["far"], device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        state = {"op": case["op"], "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
                 "q_out": torch.zeros(n, hq, d, dtype=dt, device=DEV), "positions": positions,
                 "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(), "slots": slots,
                 "interleaved": case["interleaved"]}
        if case["op"] == "rope":
            state["k_cache"] = torch.zeros(nb, bs, hkv, d, dtype=dt, device=DEV)
            state["v_cache"] = torch.zeros(nb, bs, hkv, d, dtype=dt, device=DEV)
        else:
            state["k_cache"] = torch.zeros(nb, bs, hkv, d, dtype=torch.uint8, device=DEV)
            state["v_cache"] = torch.zeros(nb, bs, hkv, d, dtype=torch.uint8, device=DEV)
            state["k_scales"] = torch.zeros(nb, hkv, bs, device=DEV)
            state["v_scales"] = torch.zeros(nb, hkv, bs, device=DEV)
        return state

    start, prefix, lens = _sizes(case)
    B = case["seqs"]
    group = torch.arange(case["groups"]).repeat_interleave(start.diff())
    whole = (prefix // bs)[group]                      # blocks of the prefix that every sequence of the group shares
    nblk = (lens + bs - 1) // bs
    most = int(nblk.max()) + 3
    j = torch.arange(most)
    # a sequence's first blocks are its group's first sequence's, the rest its own (a prefix's last, partly
    # filled block has been copied on write)
    leads = torch.zeros(B, dtype=torch.bool)
    leads[start[:-1]] = True
    takes = (j < nblk[:, None]) & (leads[:, None] | (j >= whole[:, None]))
    fresh = torch.cumsum(takes.reshape(-1).long(), 0).reshape(B, most) - 1
    nb = int(takes.sum()) + 5
    place = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    table = torch.where(takes, fresh, torch.where(j < whole[:, None], fresh[start[:-1]][group], 0)).to(DEV)
    table = torch.where((j < nblk[:, None]).to(DEV), place[table], -1)
    return {"op": "shared", "q": (1.5 * randn(B, hq, d)).to(dt), "k_cache": randn(nb, bs, hkv, d).to(dt),
            "v_cache": randn(nb, bs, hkv, d).to(dt), "out": torch.zeros(B, hq, d, dtype=dt, device=DEV),
            "tables": table.to(torch.int32).contiguous(), "lens": lens.to(torch.int32).to(DEV),
            "start": start.to(torch.int32).to(DEV), "prefix": prefix.to(torch.int32).to(DEV),
            "group_of": group.to(DEV), "row_of": (torch.arange(B) - start[:-1][group]).to(DEV),
            "largest": int(start.diff().max()), "longest_prefix": int(prefix.max()),
            "longest_rest": int((lens - whole * bs).max()), "longest": int(lens.max()), "scale": d ** -0.5}


def run(s):
    return _rope(s) if s["op"] == "rope" else _rope_fp8(s) if s["op"] == "rope_fp8" else _shared(s)


def _rotate(x, s):
    """x [N, H, D] in float32, its first `rot` values of each head rotated by the token's position."""
    half = s["cos_sin"].shape[1] // 2
    row = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    x = x.float()
    rest = x[..., 2 * half:]
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _rope(s):
    if own:
        import paged_kv_cache_128_gb300 as pk
        pk.rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"],
                          s["slots"], interleaved=s["interleaved"])
    else:
        real = s["slots"] >= 0
        at, dt = s["slots"][real].long(), s["q"].dtype
        s["q_out"][real] = _rotate(s["q"], s)[real].to(dt)
        s["k_cache"].flatten(0, 1)[at] = _rotate(s["k"], s)[real].to(dt)
        s["v_cache"].flatten(0, 1)[at] = s["v"][real]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _quantise(x):
    """E4M3 codes (as bytes) and the scale of each row of x: amax / 448, 1 for a row of zeros."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _rope_fp8(s):
    if own:
        import paged_kv_cache_128_gb300 as pk
        pk.rope_and_cache_fp8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"],
                              s["v_cache"], s["k_scales"], s["v_scales"], s["slots"], interleaved=s["interleaved"])
    else:
        real = s["slots"] >= 0
        at, bs = s["slots"][real].long(), s["k_cache"].shape[1]
        s["q_out"][real] = _rotate(s["q"], s)[real].to(s["q"].dtype)
        k, ks = _quantise(_rotate(s["k"], s)[real])
        v, vs = _quantise(s["v"][real].float())
        s["k_cache"].flatten(0, 1)[at] = k
        s["v_cache"].flatten(0, 1)[at] = v
        s["k_scales"][at // bs, :, at % bs] = ks
        s["v_scales"][at // bs, :, at % bs] = vs
    return [s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn),
            s["k_scales"], s["v_scales"]]


def _shared(s):
    if own:
        import paged_kv_cache_128_gb300 as pk
        B, hq, d = s["q"].shape
        if "workspace" not in s:  # kept between calls, as a serving loop keeps it
            bs, hkv = s["k_cache"].shape[1:3]
            s["workspace"] = pk.shared_prefix_workspace(B, hq, hkv, d, bs, s["longest"], s["q"].dtype, s["q"].device)
        return pk.paged_decode_attention_shared_prefix(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["start"], s["prefix"], s["scale"],
            s["longest"], workspace=s["workspace"])
    B, hq, d = s["q"].shape
    bs, hkv = s["k_cache"].shape[1:3]
    k_rows, v_rows = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)

    def gather(tables, first, count):
        """Keys and values [rows, Hkv, count, D] of `count` positions from `first` [rows] on, through the tables."""
        pos = (first[:, None] + torch.arange(count, device=DEV)).clamp(max=tables.shape[1] * bs - 1)
        slot = tables.gather(1, pos // bs).clamp(min=0) * bs + pos % bs
        return k_rows[slot].float().transpose(1, 2), v_rows[slot].float().transpose(1, 2)

    q = s["q"].float().view(B, hkv, hq // hkv, d) * s["scale"]
    tables, lens, group = s["tables"].long(), s["lens"].long(), s["group_of"]
    NG, most = s["start"].numel() - 1, s["largest"]
    shared = s["prefix"].long() // bs * bs             # tokens of whole blocks
    # the prefix, once for each group: rows (sequence, head) of the group against its keys
    count = max(1, s["longest_prefix"] // bs * bs)
    k, v = gather(tables[s["start"][:-1].long()], torch.zeros(NG, dtype=torch.long, device=DEV), count)
    qg = q.new_zeros(NG, most, *q.shape[1:])
    qg[group, s["row_of"]] = q
    qg = qg.transpose(1, 2).flatten(2, 3)              # [NG, Hkv, most * G, D]
    seen = (torch.arange(count, device=DEV) < shared[:, None])[:, None, None]
    w = (qg @ k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    top1 = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.sub_(top1).exp_()
    parts = [w @ v, w.sum(-1, keepdim=True), top1]
    num1, den1, top1 = [p.view(NG, hkv, most, hq // hkv, -1).transpose(1, 2)[group, s["row_of"]] for p in parts]
    # each sequence's own rest
    count = s["longest_rest"]
    k, v = gather(tables, shared[group], count)
    seen = (torch.arange(count, device=DEV) < (lens - shared[group])[:, None])[:, None, None]
    w = (q @ k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    top2 = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.sub_(top2).exp_()
    num2, den2 = w @ v, w.sum(-1, keepdim=True)
    top = torch.maximum(top1, top2)
    a, b = (top1 - top).exp(), (top2 - top).exp()
    s["out"].copy_(((num1 * a + num2 * b) / (den1 * a + den2 * b)).view(B, hq, d))
    return s["out"]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] != "shared":
        n = case["tokens"] - case["pads"]
        kept = hkv * (d + 4) if case["op"] == "rope_fp8" else hkv * d * size
        rows = min(n, case["far"])                     # rows of the angle table that can be asked for
        moved = n * (2 * hq * d * size + 2 * hkv * d * size + 2 * kept) + rows * case["rot"] * 4
        return {"bytes": moved + 4 * n + 4 * case["tokens"], "flops": 3 * n * (hq + hkv) * case["rot"]}
    start, prefix, lens = _sizes(case)
    whole = prefix // case["bs"] * case["bs"]
    tokens = int(whole.sum() + (lens - whole.repeat_interleave(start.diff())).sum())
    return {"bytes": tokens * 2 * hkv * d * size + 2 * case["seqs"] * hq * d * size + 4 * tokens // case["bs"],
            "flops": int(lens.sum()) * hq * d * 4}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared":
        B, hq, d = s["q"].shape
        bs, hkv = s["k_cache"].shape[1:3]
        out = torch.zeros(B, hq, d, dtype=torch.float64, device=DEV)
        for b in range(B):
            L = int(s["lens"][b])
            blocks = s["tables"][b, :(L + bs - 1) // bs].long()
            k = s["k_cache"][blocks].double().reshape(-1, hkv, d)[:L]
            v = s["v_cache"][blocks].double().reshape(-1, hkv, d)[:L]
            q = s["q"][b].double().reshape(hkv, hq // hkv, d)
            p = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) * (1.0 / math.sqrt(d)), -1)
            out[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(hq, d)
        return out
    rot, pos = case["rot"], s["positions"].double()
    # the angles are those of the float32 table, which is an input
    table = s["cos_sin"].double()[pos.long()]
    i = torch.arange(rot // 2, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)

    def turn(x):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    bs = case["bs"]
    real = torch.nonzero(s["slots"] >= 0)[:, 0]
    blk, off = s["slots"][real].long() // bs, s["slots"][real].long() % bs
    q_out = s["q_out"].double()
    q_out[real] = turn(s["q"])[real]
    outs = [q_out]
    rows = [turn(s["k"])[real], s["v"].double()[real]]
    if case["op"] == "rope":
        for name, x in zip(("k_cache", "v_cache"), rows):
            c = s[name].double()
            c[blk, off] = x
            outs.append(c)
        return outs
    scales = []
    for x in rows:
        amax = x.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        y = x / scale[..., None]
        # E4M3: three bits after the leading one, steps of 2^-9 below 2^-6, nearest, ties to even
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        c = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV)
        c[blk, off] = torch.round(y / step) * step
        outs.append(c)
        z = torch.zeros(s["k_scales"].shape, dtype=torch.float64, device=DEV)
        z[blk, :, off] = scale
        scales.append(z)
    return outs + scales
