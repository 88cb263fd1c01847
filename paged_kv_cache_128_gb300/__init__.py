"""GB300-native paged KV cache: host block manager + sm_103a kernels.

Public API (all work runs in libpagedkv.so; see include/pagedkv.h):

* ``KVBlockManager`` -- host metadata plane (prefill / decode allocation,
  release, export of block tables, seq_lens and slot_mapping).
* ``reshape_and_cache`` -- CUDA cache write by slot_mapping.
* ``paged_decode_attention`` -- CUDA single-query GQA attention through
  block tables, with split-K and a log-sum-exp merge.
* ``rope_and_cache`` / ``rope_and_cache_fp8`` -- rotary embedding of a step's
  queries and keys with the cache write of its keys and values, one launch.
* ``rope_and_cache_axes`` / ``rope_and_cache_axes_fp8`` -- the same for tokens
  with a position on each of several axes (time, height, width).
* ``paged_prefill_attention_rules``, ``paged_decode_attention_rules`` /
  ``paged_decode_attention_rules_fp8`` -- prefill and decode attention with
  capped scores, a distance bias, windows, documents and spans seen both ways.
* ``paged_decode_attention_shared_prefix`` -- decode attention that reads the
  prefix shared by a group of sequences once for the group.
* ``paged_decode_step`` -- the step's cache write and decode attention in
  one launch (stream-K kernel), else the two in stream order.
"""

from ._lib import KVError, LIB_PATH, lib  # noqa: F401
from .block_manager import KVBlockManager, kv_cache_ledger  # noqa: F401


def __getattr__(name):
    # the kernel wrappers need torch; import them on first use
    if name in ("reshape_and_cache", "reshape_and_cache_layers", "paged_decode_attention", "paged_decode_step", "copy_blocks", "decode_plan",
                "device_error", "alloc_workspace", "DecodePlan", "reshape_and_cache_fp8",
                "paged_decode_attention_fp8", "paged_decode_step_fp8", "paged_prefill_attention",
                "rope_and_cache", "rope_and_cache_fp8", "paged_decode_attention_shared_prefix",
                "rope_and_cache_axes", "rope_and_cache_axes_fp8", "paged_prefill_attention_rules",
                "prefill_rules_workspace",
                "paged_decode_attention_rules", "paged_decode_attention_rules_fp8",
                "shared_prefix_workspace"):
        from . import kernels
        value = globals()[name] = getattr(kernels, name)  # found directly from now on
        return value
    raise AttributeError(name)
