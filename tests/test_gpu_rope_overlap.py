"""rope_and_cache with q_out beside, over and in the place of q, k and v."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk

pytestmark = pytest.mark.gpu


def _inputs(n=37, hq=4, hkv=2, d=64):
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").bfloat16()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.randn(n, d, generator=g, device="cuda")
    return qkv, pos, table


def _call(q_out, qkv, pos, table, hq=4, hkv=2):
    n, d = qkv.shape[0], qkv.shape[2]
    kc = torch.zeros(n, 1, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pk.rope_and_cache(q_out, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, table, kc, vc, pos)
    return kc, vc


def test_rows_between_and_in_place_of_other_rows():
    """q_out in place of q, and in a free column of a wider buffer that holds q, k and v too."""
    qkv, pos, table = _inputs()
    want_q = torch.empty_like(qkv[:, :4])
    want = _call(want_q, qkv, pos, table)
    wide = torch.zeros(qkv.shape[0], 12, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = qkv
    got = _call(wide[:, 8:], wide[:, :8], pos, table)
    assert torch.equal(wide[:, 8:], want_q) and all(torch.equal(a, b) for a, b in zip(got, want))
    # the same column where q, k and v lie elsewhere with another stride
    got = _call(wide[:, 4:8], qkv, pos, table)
    assert torch.equal(wide[:, 4:8], want_q) and all(torch.equal(a, b) for a, b in zip(got, want))
    inside = qkv.clone()
    got = _call(inside[:, :4], inside, pos, table)
    assert torch.equal(inside[:, :4], want_q) and torch.equal(inside[:, 4:], qkv[:, 4:])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and pk.device_error() == 0


def test_rows_over_other_rows_are_refused():
    qkv, pos, table = _inputs()
    for first in (1, 2, 4):                            # over q and k, over k and v
        with pytest.raises(pk.KVError) as e:
            _call(qkv[:, first:first + 4], qkv, pos, table)
        assert e.value.code == "INVALID_ARG"
    # one token later: rows of tokens that have not been read
    later = torch.cat([qkv, qkv])
    with pytest.raises(pk.KVError):
        _call(later[1:38, :4], later[:37], pos, table)
