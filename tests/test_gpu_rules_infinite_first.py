"""Capped attention where the first key tile that a row's walk meets holds one
key of its own alone, with a score of minus infinity: the cap makes it minus
the cap, as anywhere else."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.rules64 import PagedBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [0.5, 6.0, 50.0, 1e38])
@pytest.mark.parametrize("window, sloped", [(1, False), (2, False), (2, True), (9, False)])
@pytest.mark.parametrize("shape", [("bf16", 8, 2, 128, 16), ("f16", 8, 2, 128, 64), ("f16", 4, 4, 64, 32),
                                   ("bf16", 4, 1, 64, 128), ("f16", 8, 2, 64, 8)], ids=str)
def test_a_lone_infinite_key(shape, window, sloped, cap):
    t = PagedBatch(*shape, [390, 129], [390, 60], seed=21)
    t.q.copy_(t.q.abs() + 0.125)                 # so that an infinite key's score is that infinity
    for b, L in enumerate(t.lens):
        for p in (64, 128, 192, 256, 384):       # first keys of tiles and of their halves
            if p < L:
                t.kc[int(t.tables[b, p // t.bs]), p % t.bs] = float("-inf")
                t.kc[int(t.tables[b, (p - 1) // t.bs]), (p - 1) % t.bs] = -4.0   # its score: close to minus the cap
    slopes = torch.exp2(-8.0 * torch.arange(1, t.hq + 1, device="cuda") / t.hq) if sloped else None
    pk.device_error()
    pk.paged_prefill_attention_rules(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.start, t.scale, 390, softcap=cap,
                                     slopes=slopes, window=window)
    assert pk.device_error() == 0
    t.check(cap=cap, slopes=slopes, window=window)
