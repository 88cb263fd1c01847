"""The calls of an image-text model with capped, windowed layers run together,
as a server runs them: the prompt's rotation on three axes into the cache,
prefill whose image tokens see their whole image, then decode steps, each
rotating and writing its token first; 16-bit and fp8 caches side by side.
Every step against 64-bit arithmetic on the rotated keys the cache holds."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from oracle.rope import angle_table
from tests.rules64 import check_rows, rules64

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, HALF = 8, 2, 128, 16, 64
PAIR_AXES = bytes([0] * 16 + [1] * 24 + [2] * 24)


class Layer:
    def __init__(self, cap, window, sloped, fp8, nb):
        self.cap, self.window, self.fp8 = cap, window, fp8
        self.slopes = torch.exp2(-torch.arange(1, HQ + 1, device="cuda").float()) if sloped else None
        shape = (nb, BS, HKV, D)
        # whatever was there before: NaN
        if fp8:
            self.kc, self.vc = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.full((nb, HKV, BS), float("nan"), device="cuda") for _ in range(2))
        else:
            self.kc, self.vc = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def write(self, q, k, v, positions, table, slots):
        out = torch.empty_like(q)
        if self.fp8:
            pk.rope_and_cache_axes_fp8(out, q, k, v, positions, PAIR_AXES, table, self.kc, self.vc, self.ks, self.vs, slots)
        else:
            pk.rope_and_cache_axes(out, q, k, v, positions, PAIR_AXES, table, self.kc, self.vc, slots)
        return out

    def keys(self, row, n):
        at = row[:-(-n // BS)].long()
        res = []
        for c, s in ((self.kc, "ks"), (self.vc, "vs")):
            x = c[at]
            if self.fp8:
                x = x.view(torch.float8_e4m3fn).double() * getattr(self, s)[at].double().transpose(1, 2)[..., None]
            res.append(x.reshape(-1, HKV, D)[:n])
        res.append(self.vs[at].transpose(1, 2).reshape(-1, HKV)[:n] if self.fp8 else None)
        return res


@pytest.mark.parametrize("sloped", [False, True])
@pytest.mark.parametrize("cap,window", [(30.0, 0), (0.0, 70), (12.0, 70)])
def test_prompt_and_decode_steps(cap, window, sloped):
    g = torch.Generator(device="cuda").manual_seed(int(cap) + window)
    prompts = [211, 60, 130]                              # tokens; an image of 80 at 30, one of 25 at 10, none
    images = [(30, 80), (10, 25), (0, 0)]
    mgr = pk.KVBlockManager(60, BS, list(range(59, -1, -1)))
    slots = torch.cat([torch.from_numpy(mgr.allocate_for_prefill(s, n)) for s, n in enumerate(prompts)]).cuda()
    table = torch.from_numpy(angle_table(1000, D)).cuda()
    pos, end = [], []
    for n, (at, size) in zip(prompts, images):
        p = torch.arange(n)
        axes = p.repeat(3, 1)
        axes[0, at:at + size] = at                        # an image's tokens share a time and lie on a grid
        axes[1, at:at + size] = at + torch.arange(size) // 9
        axes[2, at:at + size] = at + torch.arange(size) % 9
        e = p + 1
        e[at:at + size] = at + size
        pos.append(axes)
        end.append(e)
    pos, end = torch.cat(pos, 1).to(torch.int32).cuda(), torch.cat(end).to(torch.int32).cuda()
    start = torch.tensor([0, 211, 271, 401], dtype=torch.int32, device="cuda")
    layers = [Layer(cap, window, sloped, fp8, 60) for fp8 in (False, True)]
    scale = D ** -0.5
    pk.device_error()

    def randn(n, h):
        return torch.randn(n, h, D, generator=g, device="cuda").bfloat16()

    def check(layer, got, q, rows, ids, i, hi):
        """rows: each sequence's slice of got and q; i, hi: positions and interval ends."""
        tables, lens = mgr.export(list(range(3)), 20)
        for b in ids:
            k, v, vs = layer.keys(torch.from_numpy(tables[b]).cuda(), int(lens[b]))
            lo = (i[rows[b]] - window + 1).clamp(min=0) if window else torch.zeros_like(i[rows[b]])
            for h in range(HQ):
                slope = 0.0 if layer.slopes is None else float(layer.slopes[h])
                kv = h * HKV // HQ
                o, tol = rules64(q[rows[b], h], k[:, kv], v[:, kv], scale, "bf16", i[rows[b]], lo, hi[rows[b]], cap, slope,
                                 None if vs is None else vs[:, kv])
                check_rows(got[rows[b], h], o, tol, (layer.fp8, b, h))

    q, k, v = randn(401, HQ) * 2, randn(401, HKV), randn(401, HKV)
    tables, lens = (torch.from_numpy(x).cuda() for x in mgr.export([0, 1, 2], 20))
    parts = [slice(0, 211), slice(211, 271), slice(271, 401)]
    i = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    for layer in layers:
        turned = layer.write(q, k, v, pos, table, slots)
        if layer.fp8:
            continue                                      # prefill reads 16-bit caches
        out = torch.full_like(turned, float("nan"))
        pk.paged_prefill_attention_rules(out, turned, layer.kc, layer.vc, tables, lens, start, scale, 211, softcap=cap,
                                         slopes=layer.slopes, window=window, key_end=end)
        check(layer, out, turned, parts, range(3), i, end.long())
    for step in range(20):
        new = [int(mgr.append_slot_for_decode(s)) for s in range(3)]
        slots = torch.tensor(new, dtype=torch.int32, device="cuda")
        tables, lens = (torch.from_numpy(x).cuda() for x in mgr.export([0, 1, 2], 20))
        p = lens - 1
        q, k, v = randn(3, HQ) * 2, randn(3, HKV), randn(3, HKV)
        for layer in layers:
            turned = layer.write(q, k, v, p.repeat(3, 1), table, slots)
            out = torch.full_like(turned, float("nan"))
            args = (tables, lens, scale, 300)
            kw = dict(softcap=cap, slopes=layer.slopes, window=window)
            if layer.fp8:
                pk.paged_decode_attention_rules_fp8(out, turned, layer.kc, layer.vc, layer.ks, layer.vs, *args, **kw)
            else:
                pk.paged_decode_attention_rules(out, turned, layer.kc, layer.vc, *args, **kw)
            check(layer, out, turned, [slice(b, b + 1) for b in range(3)], range(3), p.long(), p.long() + 1)
    assert pk.device_error() == 0
