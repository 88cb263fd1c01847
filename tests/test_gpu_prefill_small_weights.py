"""Chunked prefill in fp16: weights down to 2^-24 of a row's largest count,
whatever the level of the row's scores.

Every 16 keys hold one of the largest score and 15 whose weight is 2^-17.5
of it; the first's value is 0, the others' 1000, so that the result is the
small weights' sum.  Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import attention64, check_rows

pytestmark = pytest.mark.gpu

LN2 = 0.6931471805599453


@pytest.mark.parametrize("top", [-7.9, -3.0, 0.0, 5.0, 7.0, -40.0])
@pytest.mark.parametrize("d, bs", [(64, 16), (128, 64), (64, 8)])
def test_prefill_keeps_small_weights(d, bs, top):
    """top: the largest score, in powers of two."""
    dev = torch.device("cuda")
    hq, hkv, n, ctx = 4, 2, 100, 220
    L = n + ctx
    nb = L // bs
    pos = torch.arange(nb * bs, device=dev)
    k = torch.zeros(nb * bs, hkv, d, device=dev)
    k[..., 0] = torch.where(pos % 16 == 0, top * LN2, (top - 17.5) * LN2)[:, None]
    v = torch.where(pos % 16 == 0, 0.0, 1000.0)[:, None, None].expand(-1, hkv, d)
    kc, vc = k.half().view(nb, bs, hkv, d), v.half().contiguous().view(nb, bs, hkv, d)
    tables = torch.arange(nb, dtype=torch.int32, device=dev).view(1, nb)
    q = torch.zeros(n, hq, d, dtype=torch.float16, device=dev)
    q[..., 0] = 1
    out = torch.full_like(q, float("nan"))
    pk.device_error()
    pk.paged_prefill_attention(out, q, kc, vc, tables, torch.tensor([L], dtype=torch.int32, device=dev),
                               torch.tensor([0, n], dtype=torch.int32, device=dev), 1.0, n)
    assert pk.device_error() == 0
    seen = torch.arange(L, device=dev) <= torch.arange(ctx, L, device=dev)[:, None]
    for h in range(hq):
        o, tol = attention64(q[:, h], kc.view(-1, hkv, d)[:L, h // 2], vc.view(-1, hkv, d)[:L, h // 2], 1.0, "f16", seen)
        check_rows(out[:, h], o, tol, h)
