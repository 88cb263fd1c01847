"""Refusals of the calls with score rules and with several axes: host-side
checks, no GPU needed."""

import ctypes

import pytest

import paged_kv_cache_128_gb300 as pk

BUF = (ctypes.c_char * 4096)()
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256

CACHES = dict(out=PTR, q=PTR, k_cache=PTR, v_cache=PTR)
SCALES = dict(k_scales=PTR, v_scales=PTR)
SIZES = dict(num_heads=4, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=4, max_blocks_per_seq=2)
RULES = dict(scale=0.125, softcap=0.0, slopes=None, window=0, key_begin=None)
END = dict(dtype=2, workspace=None, workspace_bytes=0, stream=None)
# no sequence: a call that passes every check launches nothing
CALLS = {
    "paged_decode_attention_rules": {**CACHES, "block_tables": PTR, "seq_lens": PTR, "num_seqs": 0, **SIZES,
                                     "max_seq_len": 32, **RULES, **END},
    "paged_decode_attention_rules_fp8": {**CACHES, **SCALES, "block_tables": PTR, "seq_lens": PTR, "num_seqs": 0, **SIZES,
                                         "max_seq_len": 32, **RULES, **END},
    "paged_prefill_attention_rules": {**CACHES, "block_tables": PTR, "seq_lens": PTR, "query_start_loc": PTR,
                                      "num_query_tokens": 0, "num_seqs": 0, **SIZES, "max_query_len": 8, **RULES,
                                      "key_end": None, **END},
}


def _call(name, **over):
    a = dict(CALLS[name])
    assert set(over) <= set(a)
    a.update(over)
    return getattr(pk.lib(), name)(*a.values())


@pytest.mark.parametrize("name", CALLS)
def test_empty_calls_pass(name):
    assert _call(name) == 0
    assert _call(name, softcap=50.0, slopes=PTR, window=2 ** 31 - 1, key_begin=PTR) == 0
    assert _call(name, q=None, k_cache=None) == 0       # nothing to do: pointers are not looked at


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [
    dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=3e38),
    dict(softcap=1e-42, scale=1.0), dict(window=-1), dict(slopes=PTR + 2), dict(key_begin=PTR + 1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(num_heads=5), dict(num_kv_heads=0), dict(head_dim=0),
    dict(block_size=0), dict(num_blocks=0), dict(num_blocks=2 ** 31), dict(max_blocks_per_seq=0), dict(dtype=3), dict(num_seqs=-1),
], ids=str)
def test_bad_arguments_are_refused(name, bad):
    assert _call(name, **bad) == 1


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("ptr", ["out", "q", "k_cache", "v_cache", "block_tables", "seq_lens"])
def test_missing_or_misaligned_pointers_are_refused(name, ptr):
    more = dict(num_query_tokens=3) if "prefill" in name else {}
    assert _call(name, num_seqs=1, **more, **{ptr: None}) == 1
    if ptr not in ("block_tables", "seq_lens"):
        assert _call(name, num_seqs=1, **more, **{ptr: PTR + 2}) == 1


def test_more_refusals():
    pre, fp8 = "paged_prefill_attention_rules", "paged_decode_attention_rules_fp8"
    assert _call(pre, dtype=0) == 1                                    # prefill is 16-bit
    assert _call(pre, head_dim=256) == 1
    assert _call(pre, key_end=PTR + 2) == 1
    assert _call(pre, num_query_tokens=3, num_seqs=1, query_start_loc=None) == 1
    assert _call(fp8, dtype=0) == 1
    assert _call(fp8, head_dim=64) == 1
    assert _call(fp8, block_size=8) == 1
    assert _call(fp8, num_seqs=1, k_scales=None) == 1


def _axes(fp8=False, **over):
    a = dict(q_out=PTR, q=PTR + 512, k=PTR, v=PTR, positions=PTR, num_axes=3, pair_axes=bytes(32), cos_sin=PTR,
             k_cache=PTR, v_cache=PTR)
    if fp8:
        a.update(SCALES)
    a.update(slot_mapping=PTR, num_tokens=0, num_heads=4, num_kv_heads=2, head_dim=64, rot_dim=64, max_positions=16,
             interleaved=0, block_size=16, num_blocks=4, q_out_token_stride=256, q_token_stride=256,
             k_token_stride=128, v_token_stride=128, dtype=2, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    fn = pk.lib().paged_rope_and_cache_axes_fp8 if fp8 else pk.lib().paged_rope_and_cache_axes
    return fn(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
def test_axes(fp8):
    assert _axes(fp8) == 0
    assert _axes(fp8, num_axes=1) == 0 and _axes(fp8, num_axes=4, pair_axes=bytes([3] * 32)) == 0
    for bad in (dict(num_axes=0), dict(num_axes=5), dict(pair_axes=None), dict(pair_axes=bytes([0] * 31 + [3])),
                dict(num_axes=1, pair_axes=bytes([1] * 32)), dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=66),
                dict(num_tokens=-1), dict(k_token_stride=127), dict(max_positions=0), dict(dtype=7)):
        assert _axes(fp8, **bad) == 1, bad
    assert _axes(head_dim=1024, rot_dim=514, pair_axes=bytes(257), q_out_token_stride=4096, q_token_stride=4096,
                 k_token_stride=2048, v_token_stride=2048) == 1        # more than 256 pairs
    for name in ("positions", "cos_sin", "k", "q_out"):
        assert _axes(fp8, num_tokens=1, **{name: None}) == 1
