"""Torch-facing wrappers of the CUDA entry points in libpagedkv.

Argument marshalling only: shapes, dtypes and device pointers are read off
the tensors and passed to the C ABI; every step of the computation runs in
the library's kernels.  There is no CPU path: CPU tensors are rejected.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from ._lib import DTYPE_BF16, DTYPE_F16, DTYPE_F32, KVError, check, lib

_DTYPES = {torch.float32: DTYPE_F32, torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16}


def dtype_code(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise KVError(1, f"unsupported dtype {dtype}")
    return _DTYPES[dtype]


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the handle alone: building a Stream object costs 3 us a call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _call_workspace(stream: Optional[torch.cuda.Stream], alloc, *args) -> Optional[torch.Tensor]:
    """A workspace for one call, from the memory of the stream that the call
    runs on: another stream's memory may still be in use by earlier work
    there, and may be handed out again there before the call is over."""
    if stream is None:
        return alloc(*args)
    with torch.cuda.stream(stream):
        return alloc(*args)


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise KVError(1, f"{name} must be a CUDA tensor")
    return t


def reshape_and_cache(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write k/v ``[N, Hkv, D]`` (token stride may exceed Hkv*D) into the
    ``[NB, BS, Hkv, D]`` caches at ``slot_mapping[N]`` (int32, -1 = skip)."""
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache"), (slot_mapping, "slot_mapping")):
        _cuda(t, n)
    nb, bs, hkv, d = k_cache.shape
    n = slot_mapping.numel()
    if slot_mapping.dtype != torch.int32 or not slot_mapping.is_contiguous():
        raise KVError(1, "slot_mapping must be contiguous int32")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise KVError(1, "k, v and the caches must share one dtype")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and v_cache.shape == k_cache.shape):
        raise KVError(1, "caches must be contiguous [NB, BS, Hkv, D] of one shape")
    for t in (k, v):
        if t.dim() != 3 or t.shape[0] != n or t.shape[1] != hkv or t.shape[2] != d or t.stride(2) != 1 \
                or t.stride(1) != d:
            raise KVError(1, "k and v must be [N, Hkv, D] with dense heads")
    check(lib().paged_reshape_and_cache(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                        slot_mapping.data_ptr(), n, hkv, d, bs, nb, k.stride(0), v.stride(0),
                                        dtype_code(k_cache.dtype), _stream_ptr(stream)),
          "paged_reshape_and_cache")


def reshape_and_cache_layers(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                             slot_mapping: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write k/v ``[L, N, Hkv, D]`` into L layers' caches ``[L, NB, BS, Hkv,
    D]`` at ``slot_mapping[N]`` (int32, -1 = skip) in one launch: one block
    table and slot mapping serve every layer."""
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache"), (slot_mapping, "slot_mapping")):
        _cuda(t, n)
    if k_cache.dim() != 5 or not (k_cache.is_contiguous() and v_cache.is_contiguous()) \
            or v_cache.shape != k_cache.shape:
        raise KVError(1, "caches must be contiguous [L, NB, BS, Hkv, D] of one shape")
    layers, nb, bs, hkv, d = k_cache.shape
    n = slot_mapping.numel()
    if slot_mapping.dtype != torch.int32 or not slot_mapping.is_contiguous():
        raise KVError(1, "slot_mapping must be contiguous int32")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise KVError(1, "k, v and the caches must share one dtype")
    for t in (k, v):
        if t.dim() != 4 or tuple(t.shape) != (layers, n, hkv, d) or t.stride(3) != 1 or t.stride(2) != d:
            raise KVError(1, "k and v must be [L, N, Hkv, D] with dense heads")
    check(lib().paged_reshape_and_cache_layers(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                               slot_mapping.data_ptr(), n, layers, k.stride(0), v.stride(0),
                                               k_cache.stride(0), hkv, d, bs, nb, k.stride(1), v.stride(1),
                                               dtype_code(k_cache.dtype), _stream_ptr(stream)),
          "paged_reshape_and_cache_layers")


def reshape_and_cache_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          k_scales: torch.Tensor, v_scales: torch.Tensor, slot_mapping: torch.Tensor,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantised cache write: k/v ``[N, Hkv, D]`` (fp16/bf16) to E4M3 codes
    ``[NB, BS, Hkv, D]`` (uint8) with one float32 scale per (token, kv head)
    in ``[NB, Hkv, BS]`` scale arrays, at ``slot_mapping[N]`` (-1 = skip)."""
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_scales, "k_scales"),
                 (v_scales, "v_scales"), (slot_mapping, "slot_mapping")):
        _cuda(t, n)
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_scales.dtype != torch.float32 \
            or v_scales.dtype != torch.float32:
        raise KVError(1, "fp8 caches are uint8 codes with float32 scales")
    nb, bs, hkv, d = k_cache.shape
    if v_cache.shape != k_cache.shape or tuple(k_scales.shape) != (nb, hkv, bs) or v_scales.shape != k_scales.shape:
        raise KVError(1, "caches [NB, BS, Hkv, D], scales [NB, Hkv, BS]")
    if not all(t.is_contiguous() for t in (k_cache, v_cache, k_scales, v_scales, slot_mapping)) \
            or slot_mapping.dtype != torch.int32:
        raise KVError(1, "caches, scales and slot_mapping must be contiguous (slot_mapping int32)")
    n = slot_mapping.numel()
    for t in (k, v):
        if t.dim() != 3 or t.shape[0] != n or t.shape[1] != hkv or t.shape[2] != d or t.stride(2) != 1 \
                or t.stride(1) != d:
            raise KVError(1, "k and v must be [N, Hkv, D] with dense heads")
    check(lib().paged_reshape_and_cache_fp8(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                            k_scales.data_ptr(), v_scales.data_ptr(), slot_mapping.data_ptr(), n, hkv,
                                            d, bs, nb, k.stride(0), v.stride(0), dtype_code(k.dtype),
                                            _stream_ptr(stream)), "paged_reshape_and_cache_fp8")


def _check_device(dev: int, tensors, names: str) -> None:
    """Every tensor on CUDA device ``dev`` (``names``: their names, for the
    refusal)."""
    for i, t in enumerate(tensors):
        if t.get_device() != dev or dev < 0:
            n = names.split()[i]
            raise KVError(1, f"{n} must be a CUDA tensor" if t.get_device() < 0 else
                          f"{n} is on cuda:{t.get_device()}, another tensor on cuda:{dev}")


def _rope_args(q_out, q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, pair_axes=None):
    """Checks shared by the rotating cache writes; the sizes of the call:
    (N, Hq, Hkv, D, rot_dim, max_positions, bs, NB, token strides of q_out, q,
    k and v).  ``pair_axes``: several positions per token, ``[axes, N]``."""
    _check_device(k_cache.get_device(), (k, v, positions, cos_sin, k_cache, v_cache, slot_mapping),
                  "k v positions cos_sin k_cache v_cache slot_mapping")
    shape, dt = k.shape, k.dtype
    cache = k_cache.shape
    if len(cache) != 4 or v_cache.shape != cache or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise KVError(1, "caches must be contiguous [NB, BS, Hkv, D] of one shape")
    nb, bs, hkv, d = cache
    n = slot_mapping.numel()
    if pair_axes is not None:
        if slot_mapping.dtype != torch.int32 or positions.dtype != torch.int32 or positions.dim() != 2 \
                or positions.shape[1] != n or not slot_mapping.is_contiguous() or not positions.is_contiguous():
            raise KVError(1, "slot_mapping [N] and positions [axes, N] must be contiguous int32")
        if not isinstance(pair_axes, bytes) or 2 * len(pair_axes) != cos_sin.shape[-1]:
            raise KVError(1, "pair_axes must be bytes, one axis for each of the rot_dim / 2 pairs")
    elif slot_mapping.dtype != torch.int32 or positions.dtype != torch.int32 or positions.numel() != n \
            or not slot_mapping.is_contiguous() or not positions.is_contiguous():
        raise KVError(1, "slot_mapping and positions must be contiguous int32 of one length")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise KVError(1, "cos_sin must be contiguous float32 [max_positions, rot_dim]")
    if shape != (n, hkv, d) or v.shape != shape or v.dtype != dt:
        raise KVError(1, "k and v must be [N, Hkv, D] of one dtype")
    sk, sv = k.stride(), v.stride()
    if sk[2] != 1 or sv[2] != 1 or (hkv > 1 and (sk[1] != d or sv[1] != d)):
        raise KVError(1, "k and v must have dense heads")
    # one token's or one head's stride is anything (a transposed view's, say)
    sk, sv = (sk[0], sv[0]) if n > 1 else (hkv * d, hkv * d)
    rows, rot = cos_sin.shape
    if q is None:
        if q_out is not None:
            raise KVError(1, "q_out without q")
        return n, 0, hkv, d, rot, rows, bs, nb, 0, 0, sk, sv
    if q_out is None:
        raise KVError(1, "q without q_out")
    _check_device(k_cache.get_device(), (q, q_out), "q q_out")
    qs = q.shape
    if len(qs) != 3 or q_out.shape != qs or qs[0] != n or qs[2] != d or q.dtype != dt or q_out.dtype != dt:
        raise KVError(1, "q and q_out must be [N, Hq, D] of k's dtype")
    sq, so = q.stride(), q_out.stride()
    if sq[2] != 1 or so[2] != 1 or (qs[1] > 1 and (sq[1] != d or so[1] != d)):
        raise KVError(1, "q and q_out must have dense heads")
    so, sq = (so[0], sq[0]) if n > 1 else (qs[1] * d, qs[1] * d)
    return n, qs[1], hkv, d, rot, rows, bs, nb, so, sq, sk, sv


def rope_and_cache(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                   positions: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slot_mapping: torch.Tensor, interleaved: bool = False,
                   stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Rotary embedding and cache write in one launch: ``q_out`` becomes q
    ``[N, Hq, D]`` rotated to ``positions[N]`` (int32), the rotated k and v
    ``[N, Hkv, D]`` go into the ``[NB, BS, Hkv, D]`` caches at
    ``slot_mapping[N]`` (-1 = padded token, skipped whole).  ``cos_sin``
    float32 ``[max_positions, rot_dim]``: cosines, then sines, of each
    position's angles; value pairs ``(i, i + rot_dim / 2)``, or ``(2i, 2i+1)``
    if ``interleaved``.  Token strides are free, ``q_out`` may be ``q``; q and
    q_out ``None``: only k and v."""
    n, hq, hkv, d, rot, rows, bs, nb, so, sq, sk, sv = _rope_args(q_out, q, k, v, positions, cos_sin, k_cache,
                                                                  v_cache, slot_mapping)
    dt = k.dtype
    if k_cache.dtype != dt or v_cache.dtype != dt:
        raise KVError(1, "k, v and the caches must share one dtype")
    if k_cache.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(k_cache.device):
            return rope_and_cache(q_out, q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, interleaved,
                                  stream)
    check(lib().paged_rope_and_cache(q_out.data_ptr() if hq else None, q.data_ptr() if hq else None, k.data_ptr(),
                                     v.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), k_cache.data_ptr(),
                                     v_cache.data_ptr(), slot_mapping.data_ptr(), n, hq, hkv, d, rot, rows,
                                     1 if interleaved else 0, bs, nb, so, sq, sk, sv, dtype_code(dt),
                                     _stream_ptr(stream)), "paged_rope_and_cache")
    return q_out


def rope_and_cache_fp8(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                       positions: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scales: torch.Tensor, v_scales: torch.Tensor, slot_mapping: torch.Tensor,
                       interleaved: bool = False,
                       stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """``rope_and_cache`` into fp8 caches: E4M3 codes ``[NB, BS, Hkv, D]``
    (uint8) and float32 scales ``[NB, Hkv, BS]``, the rotated key quantised
    from float32; q, k, v fp16 or bf16."""
    n, hq, hkv, d, rot, rows, bs, nb, so, sq, sk, sv = _rope_args(q_out, q, k, v, positions, cos_sin, k_cache,
                                                                  v_cache, slot_mapping)
    _check_device(k_cache.get_device(), (k_scales, v_scales), "k_scales v_scales")
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_scales.dtype != torch.float32 \
            or v_scales.dtype != torch.float32:
        raise KVError(1, "fp8 caches are uint8 codes with float32 scales")
    if k_scales.shape != (nb, hkv, bs) or v_scales.shape != (nb, hkv, bs) or not k_scales.is_contiguous() \
            or not v_scales.is_contiguous():
        raise KVError(1, "scales must be contiguous [NB, Hkv, BS]")
    if k_cache.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(k_cache.device):
            return rope_and_cache_fp8(q_out, q, k, v, positions, cos_sin, k_cache, v_cache, k_scales, v_scales,
                                      slot_mapping, interleaved, stream)
    check(lib().paged_rope_and_cache_fp8(q_out.data_ptr() if hq else None, q.data_ptr() if hq else None, k.data_ptr(),
                                         v.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), k_cache.data_ptr(),
                                         v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                         slot_mapping.data_ptr(), n, hq, hkv, d, rot, rows, 1 if interleaved else 0,
                                         bs, nb, so, sq, sk, sv, dtype_code(k.dtype), _stream_ptr(stream)),
          "paged_rope_and_cache_fp8")
    return q_out


def rope_and_cache_axes(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                        positions: torch.Tensor, pair_axes: bytes, cos_sin: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, slot_mapping: torch.Tensor, interleaved: bool = False,
                        stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """``rope_and_cache`` for tokens with a position on each of up to four
    axes (time, height, width): ``positions`` int32 ``[axes, N]``, and pair i
    of a head turns by the angle i of ``positions[pair_axes[i]]``.
    ``pair_axes``: bytes, one axis per pair -- ``bytes([0] * 16 + [1] * 24 +
    [2] * 24)`` for three sections, or the axes in turn."""
    n, hq, hkv, d, rot, rows, bs, nb, so, sq, sk, sv = _rope_args(q_out, q, k, v, positions, cos_sin, k_cache,
                                                                  v_cache, slot_mapping, pair_axes)
    dt = k.dtype
    if k_cache.dtype != dt or v_cache.dtype != dt:
        raise KVError(1, "k, v and the caches must share one dtype")
    if k_cache.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(k_cache.device):
            return rope_and_cache_axes(q_out, q, k, v, positions, pair_axes, cos_sin, k_cache, v_cache, slot_mapping,
                                       interleaved, stream)
    check(lib().paged_rope_and_cache_axes(q_out.data_ptr() if hq else None, q.data_ptr() if hq else None, k.data_ptr(),
                                          v.data_ptr(), positions.data_ptr(), positions.shape[0], pair_axes,
                                          cos_sin.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                          slot_mapping.data_ptr(), n, hq, hkv, d, rot, rows, 1 if interleaved else 0,
                                          bs, nb, so, sq, sk, sv, dtype_code(dt), _stream_ptr(stream)),
          "paged_rope_and_cache_axes")
    return q_out


def rope_and_cache_axes_fp8(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k: torch.Tensor,
                            v: torch.Tensor, positions: torch.Tensor, pair_axes: bytes, cos_sin: torch.Tensor,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                            v_scales: torch.Tensor, slot_mapping: torch.Tensor, interleaved: bool = False,
                            stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """``rope_and_cache_axes`` into fp8 caches, as ``rope_and_cache_fp8`` is
    to ``rope_and_cache``."""
    n, hq, hkv, d, rot, rows, bs, nb, so, sq, sk, sv = _rope_args(q_out, q, k, v, positions, cos_sin, k_cache,
                                                                  v_cache, slot_mapping, pair_axes)
    _check_device(k_cache.get_device(), (k_scales, v_scales), "k_scales v_scales")
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8 or k_scales.dtype != torch.float32 \
            or v_scales.dtype != torch.float32:
        raise KVError(1, "fp8 caches are uint8 codes with float32 scales")
    if k_scales.shape != (nb, hkv, bs) or v_scales.shape != (nb, hkv, bs) or not k_scales.is_contiguous() \
            or not v_scales.is_contiguous():
        raise KVError(1, "scales must be contiguous [NB, Hkv, BS]")
    if k_cache.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(k_cache.device):
            return rope_and_cache_axes_fp8(q_out, q, k, v, positions, pair_axes, cos_sin, k_cache, v_cache, k_scales,
                                           v_scales, slot_mapping, interleaved, stream)
    check(lib().paged_rope_and_cache_axes_fp8(
        q_out.data_ptr() if hq else None, q.data_ptr() if hq else None, k.data_ptr(), v.data_ptr(),
        positions.data_ptr(), positions.shape[0], pair_axes, cos_sin.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), slot_mapping.data_ptr(), n, hq, hkv, d, rot,
        rows, 1 if interleaved else 0, bs, nb, so, sq, sk, sv, dtype_code(k.dtype), _stream_ptr(stream)),
        "paged_rope_and_cache_axes_fp8")
    return q_out


def _rules_args(dev: int, hq: int, rows: int, softcap: float, slopes, window: int, key_begin, key_end=None):
    """Checks of the score rules' tensors; the rules as the C calls take them:
    (softcap, slopes, window, key_begin, key_end), pointers or None."""
    if slopes is not None:
        if slopes.get_device() != dev or slopes.dtype != torch.float32 or slopes.numel() != hq \
                or not slopes.is_contiguous():
            raise KVError(1, "slopes must be contiguous float32 [Hq] on q's device")
        slopes = slopes.data_ptr()
    if key_begin is not None:
        if key_begin.get_device() != dev or key_begin.dtype != torch.int32 or key_begin.numel() != rows \
                or not key_begin.is_contiguous():
            raise KVError(1, "key_begin must be contiguous int32, one per query row, on q's device")
        key_begin = key_begin.data_ptr()
    if key_end is not None:
        if key_end.get_device() != dev or key_end.dtype != torch.int32 or key_end.numel() != rows \
                or not key_end.is_contiguous():
            raise KVError(1, "key_end must be contiguous int32, one per query row, on q's device")
        key_end = key_end.data_ptr()
    if not 0 <= window < 2 ** 31:
        raise KVError(1, "window must be 0 (all) or a number of keys")
    return float(softcap), slopes, window, key_begin, key_end


def _rules_decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, cache_dtype):
    """Checks shared by the two decode calls with rules; (B, Hq, D, NB, bs,
    Hkv, max_blocks)."""
    _check_device(q.get_device(), (q, out, k_cache, v_cache, block_tables, seq_lens),
                  "q out k_cache v_cache block_tables seq_lens")
    shape, cache, dt = q.shape, k_cache.shape, q.dtype
    if len(shape) != 3 or len(cache) != 4:
        raise KVError(1, "q [B, Hq, D], caches [NB, BS, Hkv, D]")
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    if cache[3] != shape[2] or out.shape != shape or v_cache.shape != cache or out.dtype != dt \
            or k_cache.dtype != cache_dtype or v_cache.dtype != cache_dtype:
        raise KVError(1, "shape or dtype mismatch")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or not block_tables.is_contiguous() \
            or not seq_lens.is_contiguous() or block_tables.dim() != 2 or block_tables.shape[0] != shape[0] \
            or seq_lens.numel() != shape[0]:
        raise KVError(1, "block_tables [B, max_blocks] and seq_lens [B] must be contiguous int32")
    return shape[0], shape[1], shape[2], cache[0], cache[1], cache[2], block_tables.shape[1]


def _decode_workspace(workspace, stream, dev, B, hq, hkv, d, bs, max_seq_len, q):
    """(pointer, bytes) of a decode call's workspace and the tensor that holds
    it, allocated on the call's stream if None was given."""
    if workspace is None:
        plan = decode_plan(B, hq, hkv, d, bs, max_seq_len, q.dtype)
        workspace = _call_workspace(stream, alloc_workspace, plan, q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise KVError(1, "workspace must be contiguous on q's device")
    if workspace is None:
        return None, 0, None
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def paged_decode_attention_rules(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                                 *, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
                                 key_begin: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_decode_attention`` under score rules.  Key j of a sequence of L
    tokens (the query's position is i = L - 1) scores ``s = scale q.k_j``,
    capped to ``softcap * tanh(s / softcap)`` if ``softcap`` > 0, less
    ``slopes[h] * (i - j)`` (float32 ``[Hq]``), and is seen if it is among the
    last ``window`` keys (0: all) and ``j >= key_begin[b]`` (int32 ``[B]``).
    A sequence that sees no key gets zeros.  Blocks that end before the first
    key seen are not looked up.  ``workspace``: as for
    ``paged_decode_attention``."""
    dev = q.get_device()
    B, hq, d, nb, bs, hkv, width = _rules_decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, q.dtype)
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return paged_decode_attention_rules(out, q, k_cache, v_cache, block_tables, seq_lens, scale, max_seq_len,
                                                softcap=softcap, slopes=slopes, window=window, key_begin=key_begin,
                                                workspace=workspace, stream=stream)
    cap, sl, win, begin, _ = _rules_args(dev, hq, B, softcap, slopes, window, key_begin)
    ws_ptr, ws_bytes, workspace = _decode_workspace(workspace, stream, dev, B, hq, hkv, d, bs, max_seq_len, q)
    check(lib().paged_decode_attention_rules(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), B, hq, hkv, d, bs, nb, width, max_seq_len, float(scale), cap, sl, win, begin,
        dtype_code(q.dtype), ws_ptr, ws_bytes, _stream_ptr(stream)), "paged_decode_attention_rules")
    return out


def paged_decode_attention_rules_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                     k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                                     seq_lens: torch.Tensor, scale: float, max_seq_len: int, *, softcap: float = 0.0,
                                     slopes: Optional[torch.Tensor] = None, window: int = 0,
                                     key_begin: Optional[torch.Tensor] = None,
                                     workspace: Optional[torch.Tensor] = None,
                                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_decode_attention_rules`` over fp8 (E4M3) caches with per-token
    scales (``[NB, Hkv, BS]``); q and out fp16/bf16."""
    dev = q.get_device()
    B, hq, d, nb, bs, hkv, width = _rules_decode_args(out, q, k_cache, v_cache, block_tables, seq_lens, torch.uint8)
    _check_device(dev, (k_scales, v_scales), "k_scales v_scales")
    if k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32 or k_scales.shape != (nb, hkv, bs) \
            or v_scales.shape != (nb, hkv, bs) or not k_scales.is_contiguous() or not v_scales.is_contiguous():
        raise KVError(1, "scales must be contiguous float32 [NB, Hkv, BS]")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return paged_decode_attention_rules_fp8(
                out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, scale, max_seq_len,
                softcap=softcap, slopes=slopes, window=window, key_begin=key_begin, workspace=workspace,
                stream=stream)
    cap, sl, win, begin, _ = _rules_args(dev, hq, B, softcap, slopes, window, key_begin)
    ws_ptr, ws_bytes, workspace = _decode_workspace(workspace, stream, dev, B, hq, hkv, d, bs, max_seq_len, q)
    check(lib().paged_decode_attention_rules_fp8(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
        v_scales.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), B, hq, hkv, d, bs, nb, width, max_seq_len,
        float(scale), cap, sl, win, begin, dtype_code(q.dtype), ws_ptr, ws_bytes, _stream_ptr(stream)),
        "paged_decode_attention_rules_fp8")
    return out


def paged_decode_attention_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                               seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                               workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode attention over fp8 (E4M3) caches with per-token scales; q and
    out fp16/bf16 ``[B, Hq, D]``."""
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_scales, "k_scales"),
                 (v_scales, "v_scales"), (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _cuda(t, n)
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or out.shape != q.shape or out.dtype != q.dtype or k_cache.dtype != torch.uint8:
        raise KVError(1, "shape or dtype mismatch")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or block_tables.dim() != 2 \
            or block_tables.shape[0] != B or seq_lens.numel() != B:
        raise KVError(1, "block_tables must be [B, max_blocks] and seq_lens [B], int32")
    if workspace is None:
        plan = decode_plan(B, hq, hkv, d, bs, max_seq_len, q.dtype)
        workspace = _call_workspace(stream, alloc_workspace, plan, q.device)
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    check(lib().paged_decode_attention_fp8(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                           k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
                                           seq_lens.data_ptr(), B, hq, hkv, d, bs, nb, block_tables.shape[1],
                                           max_seq_len, float(scale), dtype_code(q.dtype), ws_ptr, ws_bytes,
                                           _stream_ptr(stream)), "paged_decode_attention_fp8")
    return out


def paged_decode_step_fp8(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          slot_mapping: torch.Tensor, new_token_row: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                          workspace: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The step's quantised cache write and decode attention over fp8
    caches in one call (one launch when the rows are 8-byte aligned)."""
    for t, n in ((out, "out"), (q, "q"), (k, "k"), (v, "v"), (slot_mapping, "slot_mapping"),
                 (new_token_row, "new_token_row"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (k_scales, "k_scales"), (v_scales, "v_scales"), (block_tables, "block_tables"),
                 (seq_lens, "seq_lens")):
        _cuda(t, n)
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    n = slot_mapping.numel()
    if d2 != d or out.shape != q.shape or out.dtype != q.dtype or k_cache.dtype != torch.uint8 \
            or k.dtype != q.dtype or v.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    for t, nm in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (slot_mapping, "slot_mapping"),
                  (new_token_row, "new_token_row")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise KVError(1, f"{nm} must be contiguous int32")
    for t in (k, v):
        if t.dim() != 3 or t.shape[0] != n or t.shape[1] != hkv or t.shape[2] != d or t.stride(2) != 1 \
                or t.stride(1) != d:
            raise KVError(1, "k and v must be [N, Hkv, D] with dense heads")
    if workspace is None:
        plan = decode_plan(B, hq, hkv, d, bs, max_seq_len, q.dtype)
        workspace = _call_workspace(stream, alloc_workspace, plan, q.device)
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    check(lib().paged_decode_step_fp8(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      slot_mapping.data_ptr(), n, k.stride(0), v.stride(0), new_token_row.data_ptr(),
                                      k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                      block_tables.data_ptr(), seq_lens.data_ptr(), B, hq, hkv, d, bs, nb,
                                      block_tables.shape[1], max_seq_len, float(scale), dtype_code(q.dtype), ws_ptr,
                                      ws_bytes, _stream_ptr(stream)), "paged_decode_step_fp8")
    return out


def paged_prefill_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                            scale: float, max_query_len: int,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Chunked prefill: q/out ``[T, Hq, D]``, sequence b's chunk is rows
    ``query_start_loc[b]:query_start_loc[b+1]``, its last positions; each
    chunk token attends causally to its sequence's keys through the table."""
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (block_tables, "block_tables"),
                 (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        _cuda(t, n)
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    nb, bs, hkv, d = k_cache.shape
    T, hq, d2 = q.shape
    B = seq_lens.numel()
    if d2 != d or out.shape != q.shape or out.dtype != q.dtype or k_cache.dtype != q.dtype \
            or v_cache.shape != k_cache.shape or v_cache.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    for t, nm in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start_loc, "query_start_loc")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise KVError(1, f"{nm} must be contiguous int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or query_start_loc.numel() != B + 1:
        raise KVError(1, "block_tables [B, max_blocks], seq_lens [B], query_start_loc [B + 1]")
    check(lib().paged_prefill_attention(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                        block_tables.data_ptr(), seq_lens.data_ptr(), query_start_loc.data_ptr(), T,
                                        B, hq, hkv, d, bs, nb, block_tables.shape[1], max_query_len, float(scale),
                                        dtype_code(q.dtype), _stream_ptr(stream)), "paged_prefill_attention")
    return out


def prefill_rules_workspace(num_tokens: int, num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                            block_size: int, max_blocks: int, max_query_len: int, device, window: int = 0,
                            begins: bool = False) -> Optional[torch.Tensor]:
    """Workspace of ``paged_prefill_attention_rules`` for these sizes (None
    when it needs none); ``max_blocks``: columns of the block table,
    ``begins``: whether the call gives ``key_begin`` (its keys are not cut then)."""
    index = torch.device(device).index
    if index is not None and index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return prefill_rules_workspace(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                           max_blocks, max_query_len, device, window, begins)
    n = ctypes.c_size_t()
    check(lib().paged_prefill_rules_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                   max_blocks, max_query_len, window, 1 if begins else 0,
                                                   ctypes.byref(n)), "paged_prefill_rules_workspace_size")
    return torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None


def paged_prefill_attention_rules(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                                  scale: float, max_query_len: int, *, softcap: float = 0.0,
                                  slopes: Optional[torch.Tensor] = None, window: int = 0,
                                  key_begin: Optional[torch.Tensor] = None, key_end: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_prefill_attention`` under score rules.  Row r of q, at position
    i of a sequence of L tokens, gives key j the score ``s = scale q.k_j``,
    capped to ``softcap * tanh(s / softcap)`` if ``softcap`` > 0, less
    ``slopes[h] * |i - j|`` (float32 ``[Hq]``), and sees it if
    ``lo <= j < hi``: lo the larger of ``i - window + 1`` (``window`` > 0) and
    ``key_begin[r]``, hi the smaller of L and ``key_end[r]`` (int32 ``[T]``,
    positions in the row's sequence), or i + 1 without ``key_end``.  A
    ``key_end`` past the row's own position lets it see ahead (a prefix, an
    image), ``key_begin`` the start of its document.  A row that sees no key
    gets zeros.  Blocks that end before the first key a tile of rows sees are
    not looked up.  ``workspace``: ``prefill_rules_workspace(...)`` of these
    sizes (allocated here if omitted), for calls whose few rows see many keys,
    which are cut into pieces then; an empty tensor: they are not."""
    dev = q.get_device()
    _check_device(dev, (q, out, k_cache, v_cache, block_tables, seq_lens, query_start_loc),
                  "q out k_cache v_cache block_tables seq_lens query_start_loc")
    if q.dim() != 3 or k_cache.dim() != 4:
        raise KVError(1, "q [T, Hq, D], caches [NB, BS, Hkv, D]")
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    nb, bs, hkv, d = k_cache.shape
    T, hq, d2 = q.shape
    B = seq_lens.numel()
    if d2 != d or out.shape != q.shape or out.dtype != q.dtype or k_cache.dtype != q.dtype \
            or v_cache.shape != k_cache.shape or v_cache.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    for t in (block_tables, seq_lens, query_start_loc):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise KVError(1, "block_tables, seq_lens and query_start_loc must be contiguous int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or query_start_loc.numel() != B + 1:
        raise KVError(1, "block_tables [B, max_blocks], seq_lens [B], query_start_loc [B + 1]")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return paged_prefill_attention_rules(out, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc,
                                                 scale, max_query_len, softcap=softcap, slopes=slopes, window=window,
                                                 key_begin=key_begin, key_end=key_end, workspace=workspace,
                                                 stream=stream)
    cap, sl, win, begin, end = _rules_args(dev, hq, T, softcap, slopes, window, key_begin, key_end)
    if workspace is None:
        workspace = _call_workspace(stream, prefill_rules_workspace, T, B, hq, hkv, d, bs, block_tables.shape[1],
                                    max_query_len, q.device, window, begin is not None)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise KVError(1, "workspace must be contiguous on q's device")
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    check(lib().paged_prefill_attention_rules(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), query_start_loc.data_ptr(), T, B, hq, hkv, d, bs, nb, block_tables.shape[1],
        max_query_len, float(scale), cap, sl, win, begin, end, dtype_code(q.dtype), ws_ptr, ws_bytes,
        _stream_ptr(stream)), "paged_prefill_attention_rules")
    return out


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy-on-write copies: block ``dst[i]`` of every layer's K and V cache
    becomes a copy of block ``src[i]`` (int32 device tensors).  Caches are
    ``[NB, BS, Hkv, D]`` or ``[layers, NB, BS, Hkv, D]``, contiguous."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (src, "src"), (dst, "dst")):
        _cuda(t, n)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and k_cache.shape == v_cache.shape
            and k_cache.dtype == v_cache.dtype):
        raise KVError(1, "caches must be contiguous, of one shape and dtype")
    if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.numel() != dst.numel() \
            or not src.is_contiguous() or not dst.is_contiguous():
        raise KVError(1, "src and dst must be contiguous int32 of one length")
    if k_cache.dim() == 4:
        layers, (nb, bs, hkv, d) = 1, k_cache.shape
        stride = 0
    elif k_cache.dim() == 5:
        layers, nb, bs, hkv, d = k_cache.shape
        stride = k_cache.stride(0)
    else:
        raise KVError(1, "caches must be 4-D or 5-D")
    check(lib().paged_copy_blocks(k_cache.data_ptr(), v_cache.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                  src.numel(), layers, stride, hkv, d, bs, nb, dtype_code(k_cache.dtype),
                                  _stream_ptr(stream)), "paged_copy_blocks")


def copy_blocks_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                    src: torch.Tensor, dst: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy-on-write copies for fp8 caches: block ``dst[i]`` takes block
    ``src[i]``'s K and V codes (uint8 ``[NB, BS, Hkv, D]``, or with a leading
    layer axis) and scales (float32 ``[NB, Hkv, BS]``, likewise)."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_scales, "k_scales"), (v_scales, "v_scales"),
                 (src, "src"), (dst, "dst")):
        _cuda(t, n)
    if k_cache.dtype != torch.uint8 or v_cache.shape != k_cache.shape or k_scales.dtype != torch.float32 \
            or v_scales.shape != k_scales.shape or not all(t.is_contiguous() for t in (k_cache, v_cache, k_scales,
                                                                                       v_scales)):
        raise KVError(1, "fp8 caches: contiguous uint8 codes and float32 scales")
    if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.numel() != dst.numel():
        raise KVError(1, "src and dst must be contiguous int32 of one length")
    if k_cache.dim() == 4:
        layers, (nb, bs, hkv, d) = 1, k_cache.shape
        stride = 0
    elif k_cache.dim() == 5:
        layers, nb, bs, hkv, d = k_cache.shape
        stride = k_cache.stride(0)
    else:
        raise KVError(1, "caches must be 4-D or 5-D")
    check(lib().paged_copy_blocks_fp8(k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
                                      v_scales.data_ptr(), src.data_ptr(), dst.data_ptr(), src.numel(), layers,
                                      stride, hkv, d, bs, nb, _stream_ptr(stream)), "paged_copy_blocks_fp8")


@dataclass
class DecodePlan:
    kernel: int            # 0 = SIMT, 1 = split TMA + tensor cores, 2 = stream-K TMA + tensor cores
    blocks_per_split: int
    num_splits: int
    workspace_bytes: int

    @property
    def launches(self) -> int:
        """Kernels one attention call launches: the split kernels add a merge
        kernel when a sequence spans several splits; stream-K merges inside."""
        return 2 if (self.kernel != 2 and self.num_splits > 1) else 1


def decode_plan(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                max_seq_len: int, dtype: torch.dtype, blocks_per_split: int = 0) -> DecodePlan:
    k, b, s = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    w = ctypes.c_size_t()
    check(lib().paged_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                                  blocks_per_split, dtype_code(dtype), ctypes.byref(k), ctypes.byref(b),
                                  ctypes.byref(s), ctypes.byref(w)), "paged_decode_plan")
    return DecodePlan(k.value, b.value, s.value, w.value)


def alloc_workspace(plan: DecodePlan, device) -> Optional[torch.Tensor]:
    if plan.workspace_bytes == 0:
        return None
    return torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=device)


def paged_decode_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                           blocks_per_split: int = 0, workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[b, qh] = softmax(scale * q[b, qh] K^T) V over seq_lens[b] tokens
    read through block_tables[b]; kvh = qh // (Hq // Hkv).  ``workspace``
    must hold ``decode_plan(...).workspace_bytes`` bytes when that is > 0
    (allocated here if omitted)."""
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _cuda(t, n)
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or not block_tables.is_contiguous() \
            or not seq_lens.is_contiguous():
        raise KVError(1, "block_tables and seq_lens must be contiguous int32")
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or out.shape != q.shape or v_cache.shape != k_cache.shape or out.dtype != q.dtype \
            or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.numel() != B:
        raise KVError(1, "block_tables must be [B, max_blocks] and seq_lens [B]")
    code = dtype_code(q.dtype)
    ws_ptr, ws_bytes = None, 0
    if workspace is None:
        plan = decode_plan(B, hq, hkv, d, bs, max_seq_len, q.dtype, blocks_per_split)
        workspace = _call_workspace(stream, alloc_workspace, plan, q.device)
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    check(lib().paged_decode_attention(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                       block_tables.data_ptr(), seq_lens.data_ptr(), B, hq, hkv, d, bs, nb,
                                       block_tables.shape[1], max_seq_len, float(scale), blocks_per_split, code,
                                       ws_ptr, ws_bytes, _stream_ptr(stream)), "paged_decode_attention")
    return out


def shared_prefix_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                            max_seq_len: int, dtype: torch.dtype, device) -> Optional[torch.Tensor]:
    """Workspace of ``paged_decode_attention_shared_prefix`` for these sizes
    and any grouping (None when it needs none)."""
    with torch.cuda.device(device):
        n = ctypes.c_size_t()
        check(lib().paged_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                       max_seq_len, dtype_code(dtype), ctypes.byref(n)),
              "paged_shared_prefix_workspace_size")
        return torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None


def paged_decode_attention_shared_prefix(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                         v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                         group_start: torch.Tensor, prefix_lens: torch.Tensor, scale: float,
                                         max_seq_len: int, workspace: Optional[torch.Tensor] = None,
                                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_decode_attention`` where sequences ``group_start[g] ..
    group_start[g + 1] - 1`` share the blocks of their first
    ``prefix_lens[g]`` tokens (int32, ``[groups + 1]`` and ``[groups]``; see
    ``KVBlockManager.prefix_groups``), which are read once for the group.
    In large batches whose shared part is less than about half of the
    lengths, ``paged_decode_attention`` is as fast or up to 15 % faster.
    ``workspace``: ``shared_prefix_workspace(...)`` (allocated here if
    omitted)."""
    dev = q.get_device()
    _check_device(dev, (q, out, k_cache, v_cache, block_tables, seq_lens, group_start, prefix_lens),
                  "q out k_cache v_cache block_tables seq_lens group_start prefix_lens")
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    for t in (block_tables, seq_lens, group_start, prefix_lens):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise KVError(1, "block_tables, seq_lens, group_start and prefix_lens must be contiguous int32")
    shape, cache, dt = q.shape, k_cache.shape, q.dtype
    if len(shape) != 3 or len(cache) != 4:
        raise KVError(1, "q [B, Hq, D], caches [NB, BS, Hkv, D]")
    B, hq, d = shape
    nb, bs, hkv, d2 = cache
    if d2 != d or out.shape != shape or v_cache.shape != cache or out.dtype != dt or k_cache.dtype != dt \
            or v_cache.dtype != dt:
        raise KVError(1, "shape or dtype mismatch")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return paged_decode_attention_shared_prefix(out, q, k_cache, v_cache, block_tables, seq_lens, group_start,
                                                        prefix_lens, scale, max_seq_len, workspace, stream)
    groups = prefix_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.numel() != B \
            or group_start.numel() != groups + 1:
        raise KVError(1, "block_tables [B, max_blocks], seq_lens [B], group_start [groups + 1], prefix_lens [groups]")
    if workspace is None:
        workspace = _call_workspace(stream, shared_prefix_workspace, B, hq, hkv, d, bs, max_seq_len, dt, q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise KVError(1, "workspace must be contiguous on q's device")
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    check(lib().paged_decode_attention_shared_prefix(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), group_start.data_ptr(), prefix_lens.data_ptr(), B, groups, hq, hkv, d, bs, nb,
        block_tables.shape[1], max_seq_len, float(scale), dtype_code(dt), ws_ptr, ws_bytes, _stream_ptr(stream)),
        "paged_decode_attention_shared_prefix")
    return out


def paged_decode_step(out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      slot_mapping: torch.Tensor, new_token_row: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                      max_seq_len: int, workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The step's cache write (``reshape_and_cache(k, v, ..., slot_mapping)``)
    and decode attention in one call: one launch when the stream-K kernel
    applies.  ``new_token_row[b]`` (int32) is the row of k/v holding
    sequence b's newest token, position ``seq_lens[b] - 1``, or -1."""
    for t, n in ((out, "out"), (q, "q"), (k, "k"), (v, "v"), (slot_mapping, "slot_mapping"),
                 (new_token_row, "new_token_row"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _cuda(t, n)
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    for t, n in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (slot_mapping, "slot_mapping"),
                 (new_token_row, "new_token_row")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise KVError(1, f"{n} must be contiguous int32")
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    n = slot_mapping.numel()
    if d2 != d or out.shape != q.shape or v_cache.shape != k_cache.shape or out.dtype != q.dtype \
            or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype or k.dtype != q.dtype or v.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.numel() != B \
            or new_token_row.numel() != B:
        raise KVError(1, "block_tables must be [B, max_blocks], seq_lens and new_token_row [B]")
    for t in (k, v):
        if t.dim() != 3 or t.shape[0] != n or t.shape[1] != hkv or t.shape[2] != d or t.stride(2) != 1 \
                or t.stride(1) != d:
            raise KVError(1, "k and v must be [N, Hkv, D] with dense heads")
    ws_ptr, ws_bytes = None, 0
    if workspace is None:
        plan = decode_plan(B, hq, hkv, d, bs, max_seq_len, q.dtype)
        workspace = _call_workspace(stream, alloc_workspace, plan, q.device)
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    check(lib().paged_decode_step(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(),
                                  n, k.stride(0), v.stride(0), new_token_row.data_ptr(), k_cache.data_ptr(),
                                  v_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), B, hq, hkv, d, bs,
                                  nb, block_tables.shape[1], max_seq_len, float(scale), dtype_code(q.dtype), ws_ptr,
                                  ws_bytes, _stream_ptr(stream)), "paged_decode_step")
    return out


def device_error(reset: bool = True) -> int:
    """Status recorded by device-side bounds checks / bounded waits (0 = none).
    Synchronises the current device."""
    st = ctypes.c_int()
    check(lib().kv_device_error(1 if reset else 0, ctypes.byref(st)), "kv_device_error")
    return st.value


def paged_decode_attention_static_scratch(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                                          v_cache: torch.Tensor, block_tables: torch.Tensor,
                                          seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                                          blocks_per_split: int = 0,
                                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``paged_decode_attention`` for callers that must not allocate device
    memory: the library's fixed scratch array stands in for the workspace
    (see include/pagedkv.h).  Nothing is allocated here either.  Raises
    KVError(WORKSPACE) when these sizes need more scratch than the array."""
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _cuda(t, n)
    if not (q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise KVError(1, "q, out and caches must be contiguous")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or not block_tables.is_contiguous() \
            or not seq_lens.is_contiguous():
        raise KVError(1, "block_tables and seq_lens must be contiguous int32")
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or out.shape != q.shape or v_cache.shape != k_cache.shape or out.dtype != q.dtype \
            or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise KVError(1, "shape or dtype mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.numel() != B:
        raise KVError(1, "block_tables must be [B, max_blocks] and seq_lens [B]")
    check(lib().paged_decode_attention_static_scratch(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), B, hq, hkv, d, bs, nb, block_tables.shape[1], max_seq_len, float(scale),
        blocks_per_split, dtype_code(q.dtype), _stream_ptr(stream)), "paged_decode_attention_static_scratch")
    return out


# Test controls of the stream-K, shared-prefix and prefill kernels (kv_debug_set keys), process-wide.
DEBUG_WAIT_LIMIT_NS = 1
DEBUG_SKIP_TILE = 2
DEBUG_DEFAULTS = {DEBUG_WAIT_LIMIT_NS: 0, DEBUG_SKIP_TILE: -1}


def debug_set(key: int, value: int) -> None:
    """Set one test control (see kv_debug_set)."""
    check(lib().kv_debug_set(int(key), int(value)), "kv_debug_set")


def debug_reset() -> None:
    """Every test control back to its default."""
    for key, value in DEBUG_DEFAULTS.items():
        debug_set(key, value)


def static_scratch_bytes() -> int:
    """Size of the fixed scratch array behind the no-allocation decode call."""
    return int(lib().paged_decode_static_scratch_bytes())
