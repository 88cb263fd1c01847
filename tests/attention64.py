"""Float64 attention of rows over their keys, with a bound on what a kernel
that rounds its probabilities to 16 bits may be off by.

The bound, from the arithmetic, for weights p_j and result o: the
probabilities are rounded to the type (u: 2^-8 bf16, 2^-11 fp16, 2^-24 fp32, relative)
and summed as rounded, which moves the result by at most
u sum_j p_j |V_j - o| / (1 - u); an fp16 probability below 2^-14 is rounded
to a step of 2^-24, half of which, 2^-25, is its error against the row's
largest, which is 1 or more: 2^-25 max_j p_j sum_j |V_j - o|; a score is off by
at most (D + 4) 2^-23 A, A = |scale| sum_d |q_d k_d|, plus 2^-22 |s| for
the exponential, and moves the result by twice that times sum_j p_j |V_j|; the float32
sums of the values and the joining of up to 1024 tiles' parts add
1100 2^-23 sum_j p_j |V_j|; the output's own rounding is u |o|.
"""

import torch

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def attention64(q, k, v, scale, dtype, seen=None):
    """q [R, D] rows against k, v [L, D] (any float type); seen [R, L] (bool):
    the keys a row has, all if None.  Returns (o, tol) [R, D] in float64; o
    holds NaN where the definition gives NaN, tol is finite."""
    q, k, v = q.double(), k.double(), v.double()
    u, d = U[dtype], q.shape[-1]
    s = q @ k.T * scale
    # a product with an infinity or NaN is no rounding error's measure
    a = q.abs().nan_to_num(0, 0, 0) @ k.abs().nan_to_num(0, 0, 0).T * abs(scale)
    if seen is not None:
        s = s.masked_fill(~seen, float("-inf"))
        a = a.masked_fill(~seen, 0)
    p = torch.softmax(s, -1)
    o = p @ v
    pf, vf, of = p.nan_to_num(0), v.nan_to_num(0, 0, 0), o.nan_to_num(0)
    off = (vf[None] - of[:, None]).abs()               # [R, L, D]
    spread = (pf[:, :, None] * off).sum(1)
    tol = u / (1 - u) * spread + u * of.abs()
    if dtype == "f16":
        keys = torch.ones_like(s, dtype=torch.bool) if seen is None else seen
        tol = tol + 2.0 ** -25 * pf.amax(-1, keepdim=True) * (keys[:, :, None] * off).sum(1)
    sf = s.abs().nan_to_num(0, 0, 0).amax(-1, keepdim=True)
    err = 2 * ((d + 4) * a.amax(-1, keepdim=True) + 2 * sf) + 1100
    return o, tol + (pf @ vf.abs()) * 2.0 ** -23 * err + 1e-7


def check_rows(got, o, tol, where=None):
    """got within tol of o; NaN exactly where o is."""
    got = got.double()
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(got), nan), (where, "NaN", int(torch.isnan(got).sum()), int(nan.sum()))
    err = (got - o).abs()[~nan]
    assert bool((err <= tol[~nan]).all()), (where, float(err.max()), float((err / tol[~nan]).max()))


def check_batch(t, out=None, seqs=None):
    """Each sequence of a decode batch (tests.test_gpu_shared_prefix.Batch)
    against attention over its own whole table."""
    out = t.out if out is None else out
    G = t.hq // t.hkv
    for b in range(len(t.lens)) if seqs is None else seqs:
        L = t.lens[b]
        if L == 0:
            assert not out[b].any(), b
            continue
        blocks = t.tables[b, :-(-L // t.bs)].long()
        k = t.kc[blocks].reshape(-1, t.hkv, t.d)[:L]
        v = t.vc[blocks].reshape(-1, t.hkv, t.d)[:L]
        for h in range(t.hkv):
            rows = slice(h * G, (h + 1) * G)
            o, tol = attention64(t.q[b, rows], k[:, h], v[:, h], t.scale, t.dtype)
            check_rows(out[b, rows], o, tol, (b, h, L))
