"""Refusals of the rotating cache writes: host-side checks, no GPU needed."""

import ctypes

import pytest

import paged_kv_cache_128_gb300 as pk

BUF = (ctypes.c_char * 4096)()
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256


def _args(fp8=False, **over):
    a = dict(q_out=PTR, q=PTR + 512, k=PTR, v=PTR, positions=PTR, cos_sin=PTR, k_cache=PTR, v_cache=PTR)
    if fp8:
        a.update(k_scales=PTR, v_scales=PTR)
    # num_tokens 0: a call that passes every check launches nothing
    a.update(slot_mapping=PTR, num_tokens=0, num_heads=4, num_kv_heads=2, head_dim=64, rot_dim=64, max_positions=16,
             interleaved=0, block_size=16, num_blocks=4, q_out_token_stride=256, q_token_stride=256,
             k_token_stride=128, v_token_stride=128, dtype=2, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


def _call(fp8=False, **over):
    fn = pk.lib().paged_rope_and_cache_fp8 if fp8 else pk.lib().paged_rope_and_cache
    return fn(*_args(fp8, **over))


@pytest.mark.parametrize("fp8", [False, True])
def test_empty_call_passes(fp8):
    assert _call(fp8) == 0
    assert _call(fp8, num_heads=0, q=None, q_out=None) == 0
    assert _call(fp8, q=None, k=None, slot_mapping=None) == 0      # nothing to do: pointers are not looked at


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(num_tokens=-1), dict(num_tokens=2 ** 31), dict(num_heads=-1), dict(num_kv_heads=0), dict(head_dim=0),
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=-2), dict(max_positions=0), dict(block_size=0),
    dict(num_blocks=0), dict(num_blocks=2 ** 31), dict(k_token_stride=127), dict(v_token_stride=0),
    dict(q_token_stride=255), dict(q_out_token_stride=255), dict(dtype=3), dict(dtype=-1),
], ids=str)
def test_bad_sizes_are_refused(fp8, bad):
    assert _call(fp8, **bad) == 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["q_out", "q", "k", "v", "positions", "cos_sin", "k_cache", "v_cache", "slot_mapping"])
def test_missing_or_misaligned_pointers_are_refused(fp8, name):
    assert _call(fp8, num_tokens=1, **{name: None}) == 1
    if name not in ("positions", "slot_mapping") and not (fp8 and name.endswith("cache")):
        assert _call(fp8, num_tokens=1, **{name: PTR + 1}) == 1


def test_more_refusals():
    assert _call(True, num_tokens=1, k_scales=None) == 1
    assert _call(True, dtype=0) == 1                               # fp32 has no fp8 write
    assert _call(True, head_dim=96, rot_dim=96, q_token_stride=999, q_out_token_stride=999, k_token_stride=999,
                 v_token_stride=999) == 1
    assert _call(num_tokens=1, q_out=PTR, q=PTR, q_token_stride=512) == 1   # in place, but not the same rows
