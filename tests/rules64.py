"""Float64 attention under score rules, with a bound on what a kernel may be
off by, and a paged batch for its tests.

The bound, from the arithmetic, for row weights p_j, result o and values V_j
(u: half a step of the type, 2^-8 bf16, 2^-11 fp16, 2^-24 fp32):

* the probabilities are rounded to the type of the products and summed as
  rounded: u / (1 - u) sum_j p_j |V_j - o|; an fp16 probability below 2^-14 is
  off by up to 2^-25 against the row's largest, which is 1 or more: 2^-25
  max_j p_j sum_{j seen} |V_j - o|;
* key j's score is off by d_j, which moves the result by sum_j p_j d_j
  |V_j - o| (a tenth more for the second order), d_j in units of 2^-23:
  (D + 4) A_j, A_j = |scale| sum_d |q_d k_jd|, for the products and sums in
  float32 (a cap's slope is at most 1, so it does not grow that); 10 |s_j| for the
  scale, the cap (its polynomial and its exponential form are within 7e-7 of
  the score) and the steps after it; 8 |b_j| for the bias b_j; 2 |x| with x the
  row's largest score, from which the others are taken; 2 for exp2;
* float32 sums of the values and the joining of up to 1024 parts:
  1100 2^-23 sum_j p_j |V_j|;
* the output's own rounding: u |o|.

An fp8 cache is multiplied in fp16 whatever the type: the products p_j f_j of
the probabilities with the values' scales f_j are rounded to fp16, 2^-11, with
the floor of 2^-25, and multiply codes V_j / f_j.  The softmax sum is that of
the p_j themselves, not of what the rounding left, so the rounding does not
cancel between the two as it does above: with r_j the relative error of
product j, |r_j| <= 2^-11, the result is sum_j p_j (1 + r_j) V_j / sum_j p_j,
off by up to 2^-11 sum_j p_j |V_j| (a single key, p = 1: 2^-11 |V|, where
|V_j - o| is 0).
"""

import math

import numpy as np
import torch

from tests.helpers import TORCH, sentinel_tensor

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rules64(q, k, v, scale, dtype, pos, lo, hi, cap=0.0, slope=0.0, v_scale=None):
    """q [R, D] rows at positions pos [R] against k, v [L, D]; row r sees keys
    lo[r] <= j < hi[r].  v_scale [L]: the values' scales of an fp8 cache.
    Returns (o, tol) [R, D] in float64."""
    q, k, v = q.double(), k.double(), v.double()
    d, R, L = q.shape[-1], q.shape[0], k.shape[0]
    j = torch.arange(L, device=q.device)
    pos, lo, hi = (torch.as_tensor(x, device=q.device).expand(R)[:, None] for x in (pos, lo, hi))
    seen = (j >= lo) & (j < hi)
    s = q @ k.T * scale
    a = q.abs().nan_to_num(0, 0, 0) @ k.abs().nan_to_num(0, 0, 0).T * abs(scale)
    if cap:
        s = cap * torch.tanh(s / cap)
    bias = slope * (pos - j).abs().double()
    x = (s - bias).masked_fill(~seen, -math.inf)
    p = torch.softmax(x, -1).masked_fill(~seen, 0)
    none = ~seen.any(-1)
    p[none] = 0
    vv = v.nan_to_num(0, 0, 0)
    o = p @ torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
    o[none] = 0
    pf, of = p.nan_to_num(0), o.nan_to_num(0)
    top = x.nan_to_num(0, 0, 0).masked_fill(~seen, -math.inf).amax(-1, keepdim=True).clamp(min=-1e30).abs()
    delta = ((d + 4) * a + 10 * s.nan_to_num(0, 0, 0).abs() + 8 * bias.abs() + 2 * top.nan_to_num(0, 0, 0) + 2) * 2.0 ** -23
    u = U[dtype]
    tol = u * of.abs() + 1100 * 2.0 ** -23 * (pf @ vv.abs()) + 1e-7
    w = 1.1 * pf * delta
    if v_scale is None:
        w = w + u / (1 - u) * pf
    else:
        tol += U["f16"] * (pf @ vv.abs())
    for r0 in range(0, R, 64):  # [64, L, D] at a time
        r = slice(r0, r0 + 64)
        off = (vv[None] - of[r, None]).abs()
        tol[r] += (w[r, :, None] * off).sum(1)
        if v_scale is None and dtype == "f16":
            tol[r] += 2.0 ** -25 * pf[r].amax(-1, keepdim=True) * (seen[r, :, None] * off).sum(1)
    if v_scale is not None:
        codes = (vv.abs() / v_scale.double()[:, None]).nan_to_num(0, 0, 0)
        tol += 2.0 ** -25 * pf.amax(-1, keepdim=True) * (seen.double() @ codes)
    return o, tol


def check_rows(got, o, tol, where=None):
    """got within tol of o; NaN exactly where o is."""
    got = got.double()
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(got), nan), (where, "NaN", int(torch.isnan(got).sum()), int(nan.sum()))
    err = (got - o).abs()[~nan]
    if err.numel():
        ratio = err / tol[~nan]
        assert bool((ratio <= 1).all()), (where, float(err.max()), float(ratio.max()))


class PagedBatch:
    """Sequences of `lens` tokens behind block tables in random order.  Slots
    past a sequence's end and blocks that no sequence owns hold NaN; table
    entries past a row's blocks are -1.  chunks: query rows of each sequence,
    its last ones (one each for decode)."""

    def __init__(self, dtype, hq, hkv, d, bs, lens, chunks=None, seed=0, spread=1.0, q_spread=2.0, fp8=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        dev = torch.device("cuda")
        self.dtype, self.hq, self.hkv, self.d, self.bs, self.lens = dtype, hq, hkv, d, bs, list(lens)
        self.chunks = [1] * len(lens) if chunks is None else list(chunks)
        self.fp8 = fp8
        need = [-(-n // bs) for n in lens]
        self.nb = sum(need) + 2
        place = rng.permutation(self.nb).astype(np.int32)
        tab = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            tab[b, :n] = place[at:at + n]
            at += n
        self.tables = torch.from_numpy(tab).to(dev)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        used = torch.zeros(self.nb, bs, dtype=torch.bool, device=dev)
        for b, n in enumerate(self.lens):
            p = torch.arange(n, device=dev)
            used.view(-1)[self.tables[b].long()[p // bs] * bs + p % bs] = True
        dt = TORCH[dtype]
        shape = (self.nb, bs, hkv, d)
        self.k = torch.randn(shape, generator=g, device=dev) * spread
        self.v = torch.randn(shape, generator=g, device=dev) * spread
        if fp8:
            self.cache = {}
            for name in ("k", "v"):
                x = getattr(self, name)
                sc = x.abs().amax(-1) / 448.0
                codes = (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                codes[~used] = 0x7F                                    # the NaN code
                sc[~used] = float("nan")
                self.cache[name] = codes
                self.cache[name + "s"] = sc.transpose(1, 2).contiguous()
                setattr(self, name, codes.view(torch.float8_e4m3fn).double() * sc.double()[..., None])
            self.kc, self.vc = self.cache["k"], self.cache["v"]
        else:
            self.kc, self.vc = (sentinel_tensor(shape, dtype, dev) for _ in range(2))
            self.kc[used], self.vc[used] = self.k[used].to(dt), self.v[used].to(dt)
        rows = sum(self.chunks)
        self.q = (torch.randn(rows, hq, d, generator=g, device=dev) * q_spread).to(dt)
        self.out = sentinel_tensor((rows, hq, d), dtype, dev)
        self.uncut = None
        self.scale = 1.0 / math.sqrt(d)
        self.row0 = [0] + np.cumsum(self.chunks).tolist()
        self.start = torch.tensor(self.row0, dtype=torch.int32, device=dev)

    def keys(self, b):
        """Logical K and V [L, Hkv, D] of sequence b (and V's scales, fp8); positions whose block is not in the
        table are NaN."""
        n, t = self.lens[b], self.tables[b].long()
        at = t[:-(-n // self.bs)]
        gone = ((at < 0) | (at >= self.nb)).repeat_interleave(self.bs)[:n]
        at = at.clamp(0, self.nb - 1)
        out = []
        for c, x in ((self.kc, self.k), (self.vc, self.v)):
            y = (x if self.fp8 else c)[at].double().reshape(-1, self.hkv, self.d)[:n].clone()
            y[gone] = float("nan")
            out.append(y)
        out.append(self.cache["vs"][at].transpose(1, 2).reshape(-1, self.hkv)[:n] if self.fp8 else None)
        return out

    def check(self, out=None, cap=0.0, slopes=None, window=0, begin=None, end=None, seqs=None):
        """Every sequence's rows against rules64; self.out, and self.uncut if a test has set it, unless `out` is given."""
        outs = [out] if out is not None else [self.out] if self.uncut is None else [self.out, self.uncut]
        G = self.hq // self.hkv
        for b in range(len(self.lens)) if seqs is None else seqs:
            L, n, r0 = self.lens[b], self.chunks[b], self.row0[b]
            if n == 0:
                continue
            rows = slice(r0, r0 + n)
            if L == 0:
                assert not any(x[rows].any() for x in outs), b
                continue
            pos = torch.arange(L - n, L, device="cuda")
            lo = torch.zeros_like(pos) if begin is None else begin[rows].long()
            if window:
                lo = torch.maximum(lo, pos - window + 1)
            hi = pos + 1 if end is None else end[rows].long()
            hi = hi.clamp(max=L)
            k, v, vs = self.keys(b)
            for h in range(self.hq):
                kv = h // G
                o, tol = rules64(self.q[rows, h], k[:, kv], v[:, kv], self.scale, self.dtype, pos, lo.clamp(min=0), hi, cap,
                                 0.0 if slopes is None else float(slopes[h]), None if vs is None else vs[:, kv])
                for i, x in enumerate(outs):
                    check_rows(x[rows, h], o, tol, (i, b, h, L))
