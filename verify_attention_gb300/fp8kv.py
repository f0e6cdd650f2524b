"""Thin ctypes binding of libfp8kv.so (include/fp8kv.h), same names as the C ABI.

Only argument marshalling happens here: tensors become device pointers and
sizes, the current torch stream becomes the cudaStream_t, and a non-zero
status raises ``Fp8kvError``.  Every step of the computation runs in the
library's CUDA kernels; there is no fallback: if the library is missing, the
first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfp8kv.so")

FP8KV_CACHE_E4M3 = 0
FP8KV_CACHE_BF16 = 1
FP8KV_CACHE_INT4 = 2
INT4_ROW_BYTES = 72         # a row of an INT4 cache: 64 bytes of codes, 8 of block scales
DEV_BAD_SLOT, DEV_BAD_POSITION, DEV_BAD_SEQ_LEN, DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_TREE, DEV_BAD_PROBS = 0x10, 0x20
TREE_MAX_NODES = 64

_lib = None


class Fp8kvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({fp8kv_status_string(status)})")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m verify_attention_gb300.build` (nvcc, sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, f32, sz, i64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_float,
                                      ctypes.c_size_t, ctypes.c_int64)
        L.fp8kv_cache_insert.restype = i32
        L.fp8kv_cache_insert.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, i32, i32, vp]
        L.fp8kv_cache_gather.restype = i32
        L.fp8kv_cache_gather.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
        L.fp8kv_qk_norm_rope_insert.restype = i32
        L.fp8kv_qk_norm_rope_insert.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, i32, vp, vp, i32, i32,
                                                i32, i32, vp, vp, vp, vp, i32, i32, vp]
        L.fp8kv_prompt_attention.restype = i32
        L.fp8kv_prompt_attention.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, i32, i32, i32, f32, i32,
                                             vp, vp]
        L.fp8kv_paged_attention_plan.restype = i32
        L.fp8kv_paged_attention_plan.argtypes = [i32] * 9 + [ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.fp8kv_paged_attention_workspace_size.restype = sz
        L.fp8kv_paged_attention_workspace_size.argtypes = [i32] * 9
        L.fp8kv_paged_attention.restype = i32
        L.fp8kv_paged_attention.argtypes = [vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32, i32,
                                            i32, i32, vp, vp, f32, i32, i32, vp, sz, vp, vp]
        L.fp8kv_append_paged_attention.restype = i32
        L.fp8kv_append_paged_attention.argtypes = [vp, vp] + L.fp8kv_paged_attention.argtypes
        L.fp8kv_cache_insert_per_head.restype = i32
        L.fp8kv_cache_insert_per_head.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, i32, vp]
        L.fp8kv_paged_attention_per_head.restype = i32
        L.fp8kv_paged_attention_per_head.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32,
                                                     i32, i32, vp, vp, f32, i32, i32, vp, sz, vp, vp]
        L.fp8kv_append_paged_attention_per_head.restype = i32
        L.fp8kv_append_paged_attention_per_head.argtypes = [vp, vp] + L.fp8kv_paged_attention_per_head.argtypes
        L.fp8kv_paged_attention_noalloc.restype = i32
        L.fp8kv_paged_attention_noalloc.argtypes = [vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                                    i32, i32, i32, vp, vp, f32, i32, i32, vp, vp]
        L.fp8kv_paged_attention_layers_workspace_size.restype = sz
        L.fp8kv_paged_attention_layers_workspace_size.argtypes = [i32] * 5
        L.fp8kv_paged_attention_layers.restype = i32
        L.fp8kv_paged_attention_layers.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
        L.fp8kv_tree_metadata.restype = i32
        L.fp8kv_tree_metadata.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        L.fp8kv_rope_insert.restype = i32
        L.fp8kv_rope_insert.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i32, i32, i32, vp, vp, i32, i32, i32, i32,
                                        vp, vp, vp, vp, i32, i32, i32, vp]
        L.fp8kv_tree_attention.restype = i32
        L.fp8kv_tree_attention.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                           i32, i32, vp, vp, f32, i32, i32, vp, sz, vp, vp]
        L.fp8kv_verify_tree.restype = i32
        L.fp8kv_verify_tree.argtypes = [vp, i64, vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
        L.fp8kv_cache_keep_path.restype = i32
        L.fp8kv_cache_keep_path.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32, i32, vp,
                                            vp]
        L.fp8kv_e4m3_encode_bits.restype = i32
        L.fp8kv_e4m3_encode_bits.argtypes = [u32, sz, vp, vp]
        L.fp8kv_selftest_bounded_wait.restype = i32
        L.fp8kv_selftest_bounded_wait.argtypes = [ctypes.c_uint, vp]
        L.fp8kv_status_string.restype = ctypes.c_char_p
        L.fp8kv_status_string.argtypes = [i32]
        L.fp8kv_last_dispatch.restype = i32
        L.fp8kv_last_dispatch.argtypes = [ctypes.c_char_p, sz]
        L.fp8kv_launch_count.restype = ctypes.c_ulonglong
        L.fp8kv_launch_count.argtypes = []
        L.fp8kv_device_status.restype = i32
        L.fp8kv_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i32]
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]) -> int:
    # plain ints: ctypes converts them for c_void_p arguments without a wrapper object
    return t.data_ptr() if t is not None else 0


def _stream(stream, t=None) -> int:
    """The stream's handle; `t`, one of the call's tensors, must be on the current device."""
    if stream is None or t is not None:
        device = torch.cuda.current_device()
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on cuda:{t.get_device()}, but the current device is cuda:{device}")
        if stream is None:
            # the handle of the current stream without a Stream object (0.3 us instead of 3)
            return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _at(stream):
    """What is allocated and filled for a call on `stream` belongs there, as under
    torch.cuda.stream(stream): filled on the current stream it might be filled
    after the call; memory of the current stream's pool might still be in use by
    work queued there, and might be handed out again before the call ends.  (An
    output allocated here and used on another stream is the caller's to order
    and to record_stream, as with any tensor of torch's.)"""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _zeros(shape, device, stream):
    with _at(stream):
        return torch.empty(shape, dtype=torch.bfloat16, device=device).zero_()


def _empty_like(t, stream):
    if stream is None:
        return torch.empty_like(t)
    with _at(stream):
        return torch.empty_like(t)


def _workspace(need, device, stream):
    if not need:
        return None
    with _at(stream):
        return torch.empty(need, dtype=torch.uint8, device=device)


def _check(fn, rc):
    if rc != 0:
        raise Fp8kvError(fn, rc)


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _cache_dtype(cache: torch.Tensor) -> int:
    if cache.dtype == torch.uint8:
        return FP8KV_CACHE_INT4 if cache.dim() == 3 else FP8KV_CACHE_E4M3
    if cache.dtype == torch.bfloat16:
        return FP8KV_CACHE_BF16
    raise ValueError("cache must be uint8 (E4M3 codes, or INT4 pages) or bfloat16")


def _cache_shape(k_cache: torch.Tensor, v_cache: torch.Tensor, dt: int, D: Optional[int] = None):
    """(num_pages, Hkv, page_size) of a pair of caches.  The library takes the
    bytes of a row from D, the call's (None: the caches' own is passed)."""
    if dt != FP8KV_CACHE_INT4:
        num_pages, Hkv, page_size, row = k_cache.shape
        if D is not None and row != D:
            raise ValueError(f"k_cache and v_cache have rows of {row} elements, the call has heads of {D}")
        if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must have the same type and shape")
        return num_pages, Hkv, page_size
    num_pages, Hkv, nbytes = k_cache.shape
    if nbytes % INT4_ROW_BYTES:
        raise ValueError(f"an INT4 cache is [num_pages][Hkv][page_size * {INT4_ROW_BYTES}] bytes")
    if v_cache.dtype != torch.uint8 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same type and shape")
    return num_pages, Hkv, nbytes // INT4_ROW_BYTES


def fp8kv_int4_cache(num_pages, Hkv, page_size, device=None):
    """One INT4 cache (K or V): uint8 [num_pages][Hkv][page_size * 72], zeroed
    (every row reads as zeros)."""
    return torch.zeros((num_pages, Hkv, page_size * INT4_ROW_BYTES), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def fp8kv_status_string(status: int) -> str:
    return lib().fp8kv_status_string(status).decode()


def fp8kv_cache_insert(k, v, slot_mapping, k_scale, v_scale, k_cache, v_cache, stream=None):
    """k, v bf16 [T][Hkv][D]; slot_mapping int64 [T]; scales fp32 [1] (E4M3, INT4);
    caches [num_pages][Hkv][page_size][D] uint8 (E4M3) or bf16, or the INT4 pages
    of fp8kv_int4_cache."""
    dt = _cache_dtype(k_cache)
    _dev(k, "k", torch.bfloat16), _dev(v, "v", torch.bfloat16)
    _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    T, Hkv, D = k.shape
    num_pages, heads, page_size = _cache_shape(k_cache, v_cache, dt, D)
    if heads != Hkv or v.shape != k.shape or slot_mapping.numel() != T:
        raise ValueError(f"k, v must be [T][{heads}][D] and slot_mapping [T]")
    if dt == FP8KV_CACHE_INT4:
        _one_scale(k_scale, v_scale)
    rc = lib().fp8kv_cache_insert(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), T, Hkv, D, _ptr(k_scale),
                                  _ptr(v_scale), k_cache.data_ptr(), v_cache.data_ptr(), num_pages, page_size,
                                  dt, _stream(stream, k_cache))
    _check("fp8kv_cache_insert", rc)


def _int4_call(q, k_cache, block_table, seq_lens, k_scale, v_scale, out, num_pages):
    """Checks of an attention call over an INT4 cache beyond the library's own:
    what it cannot see from pointers."""
    B = q.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError(f"block_table must be [{B}][pages] and seq_lens [{B}]")
    _one_scale(k_scale, v_scale)
    if out is not None and _dev(out, "out", torch.bfloat16).shape != q.shape:
        raise ValueError("out must have the shape of q")
    if num_pages is not None and num_pages > k_cache.shape[0]:
        raise ValueError(f"num_pages is {num_pages}, the cache has {k_cache.shape[0]}")


def _one_scale(k_scale, v_scale):
    _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32)
    if k_scale.numel() != 1 or v_scale.numel() != 1:
        raise ValueError("k_scale and v_scale must be one fp32 each")


def fp8kv_cache_gather(slot_mapping, k_scale, v_scale, k_cache, v_cache, k_out=None, v_out=None, stream=None):
    """The stored K and V of the tokens in slot_mapping (int64 [T]) as bf16
    [T][Hkv][D]; rows with a negative slot are left as they are (zeros when the
    outputs are allocated here).  Any cache type, per-tensor scales."""
    dt = _cache_dtype(k_cache)
    _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    num_pages, Hkv, page_size = _cache_shape(k_cache, v_cache, dt)
    T, D = slot_mapping.numel(), 128 if dt == FP8KV_CACHE_INT4 else k_cache.shape[3]
    if dt != FP8KV_CACHE_BF16:
        _one_scale(k_scale, v_scale)
    if k_out is None and v_out is None:
        k_out, v_out = _zeros((2, T, Hkv, D), k_cache.device, stream).unbind(0)     # one fill instead of two
    k_out = _zeros((T, Hkv, D), k_cache.device, stream) if k_out is None else _dev(k_out, "k_out", torch.bfloat16)
    v_out = _zeros((T, Hkv, D), k_cache.device, stream) if v_out is None else _dev(v_out, "v_out", torch.bfloat16)
    if k_out.shape != (T, Hkv, D) or v_out.shape != (T, Hkv, D):
        raise ValueError(f"k_out and v_out must be {(T, Hkv, D)}, got {tuple(k_out.shape)} and {tuple(v_out.shape)}")
    rc = lib().fp8kv_cache_gather(slot_mapping.data_ptr(), T, Hkv, D, _ptr(k_scale), _ptr(v_scale),
                                  k_cache.data_ptr(), v_cache.data_ptr(), num_pages, page_size, dt, k_out.data_ptr(),
                                  v_out.data_ptr(), _stream(stream, k_cache))
    _check("fp8kv_cache_gather", rc)
    return k_out, v_out


def _head_scales(k_scale, v_scale, Hkv):
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _dev(t, n, torch.float32)
        if t.numel() != Hkv:
            raise ValueError(f"{n} must hold one fp32 scale per KV head ({Hkv}), got {t.numel()}")


def fp8kv_cache_insert_per_head(k, v, slot_mapping, k_scale, v_scale, k_cache, v_cache, stream=None):
    """fp8kv_cache_insert on an E4M3 cache with per-head scales fp32 [Hkv]."""
    _dev(k, "k", torch.bfloat16), _dev(v, "v", torch.bfloat16)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(k_cache, "k_cache", torch.uint8), _dev(v_cache, "v_cache", torch.uint8)
    T, Hkv, D = k.shape
    _head_scales(k_scale, v_scale, Hkv)
    num_pages, heads, page_size = _cache_shape(k_cache, v_cache, FP8KV_CACHE_E4M3, D)
    if heads != Hkv or v.shape != k.shape or slot_mapping.numel() != T:
        raise ValueError(f"k, v must be [T][{heads}][D] and slot_mapping [T]")
    rc = lib().fp8kv_cache_insert_per_head(_ptr(k), _ptr(v), _ptr(slot_mapping), T, Hkv, D, _ptr(k_scale),
                                           _ptr(v_scale), _ptr(k_cache), _ptr(v_cache), num_pages, page_size,
                                           _stream(stream))
    _check("fp8kv_cache_insert_per_head", rc)


def fp8kv_qk_norm_rope_insert(q, k, v, positions, q_norm_w, k_norm_w, eps, cos_sin, q_out,
                              slot_mapping, k_scale, v_scale, k_cache, v_cache, stream=None):
    """Fused Q/K RMSNorm + RoPE + E4M3 insert; writes q_out (bf16 [T][Hq][D])."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (q_out, "q_out"), (q_norm_w, "q_norm_w"),
                 (k_norm_w, "k_norm_w")):
        _dev(t, n, torch.bfloat16)
    _dev(positions, "positions", torch.int64), _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cos_sin, "cos_sin", torch.float32), _dev(k_cache, "k_cache", torch.uint8)
    _dev(v_cache, "v_cache", torch.uint8)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    num_pages, heads, page_size = _cache_shape(k_cache, v_cache, FP8KV_CACHE_E4M3, D)
    if k.shape != (T, heads, D) or v.shape != k.shape or q_out.shape != q.shape:
        raise ValueError(f"k, v must be [{T}][{heads}][{D}] and q_out of the shape of q")
    if positions.numel() != T or slot_mapping.numel() != T:
        raise ValueError(f"positions and slot_mapping must be [{T}]")
    rc = lib().fp8kv_qk_norm_rope_insert(
        _ptr(q), _ptr(k), _ptr(v), _ptr(positions), _ptr(q_norm_w), _ptr(k_norm_w), float(eps),
        _ptr(cos_sin), cos_sin.shape[0], _ptr(q_out), _ptr(slot_mapping), T, Hq, Hkv, D, _ptr(k_scale),
        _ptr(v_scale), _ptr(k_cache), _ptr(v_cache), num_pages, page_size, _stream(stream))
    _check("fp8kv_qk_norm_rope_insert", rc)


def _token_rows(t: torch.Tensor, name: str, T: int, heads: int, D: int):
    """bf16 [T][heads][D] with dense tokens; returns the elements between tokens."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    st = t.stride()
    if t.shape != (T, heads, D) or st[2] != 1 or (heads > 1 and st[1] != D):
        raise ValueError(f"{name} must be [{T}][{heads}][{D}] with dense tokens")
    return st[0] if T > 1 else heads * D


def fp8kv_prompt_attention(q, k, v, cu_seqlens, max_seq_len, sm_scale, window_left=-1, out=None, stream=None):
    """Causal attention of packed prompts: q bf16 [T][Hq][D], k, v bf16
    [T][Hkv][D] (tokens dense, any distance apart: views of a fused projection
    are fine), cu_seqlens int32 [B + 1].  Returns out bf16 [T][Hq][D]; rows of no
    sequence are left as they are (zeros when allocated here)."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    q_stride = _token_rows(q, "q", T, Hq, D)
    k_stride, v_stride = _token_rows(k, "k", T, Hkv, D), _token_rows(v, "v", T, Hkv, D)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    out = _zeros((T, Hq, D), q.device, stream) if out is None else _dev(out, "out", torch.bfloat16)
    if out.shape != (T, Hq, D):
        raise ValueError(f"out must be {(T, Hq, D)}, got {tuple(out.shape)}")
    rc = lib().fp8kv_prompt_attention(q.data_ptr(), q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
                                      cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, T, int(max_seq_len), Hq, Hkv, D,
                                      float(sm_scale), int(window_left), out.data_ptr(), _stream(stream, q))
    _check("fp8kv_prompt_attention", rc)
    return out


def fp8kv_rope_insert(q, k, v, positions, cos_sin, slot_mapping, k_scale, v_scale, k_cache, v_cache, interleaved=False,
                      q_out=None, stream=None):
    """Rotary positions on Q and K, then K and V into the cache: q bf16 [T][Hq][D],
    k, v bf16 [T][Hkv][D] (tokens dense, any distance apart), positions and
    slot_mapping int64 [T], cos_sin fp32 [max_pos][rot_dim] (the cosines of a
    position's rot_dim / 2 angles, then the sines), any cache type.  Pairs are the
    elements (k, k + rot_dim / 2), or neighbours with ``interleaved``; the rest of a
    head stays.  Returns the rotated Q, bf16 [T][Hq][D]; rows of tokens with a bad
    position are left as they are (zeros when allocated here)."""
    dt = _cache_dtype(k_cache)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    q_stride = _token_rows(q, "q", T, Hq, D)
    k_stride, v_stride = _token_rows(k, "k", T, Hkv, D), _token_rows(v, "v", T, Hkv, D)
    _dev(positions, "positions", torch.int64), _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(cos_sin, "cos_sin", torch.float32), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    num_pages, heads, page_size = _cache_shape(k_cache, v_cache, dt, D)
    if heads != Hkv:
        raise ValueError(f"k_cache and v_cache must be of {Hkv} heads")
    if positions.numel() != T or slot_mapping.numel() != T or cos_sin.dim() != 2:
        raise ValueError(f"positions and slot_mapping must be [{T}], cos_sin [max_pos][rot_dim]")
    if dt != FP8KV_CACHE_BF16:
        _one_scale(k_scale, v_scale)
    q_out = _zeros((T, Hq, D), q.device, stream) if q_out is None else _dev(q_out, "q_out", torch.bfloat16)
    if q_out.shape != (T, Hq, D):
        raise ValueError(f"q_out must be {(T, Hq, D)}, got {tuple(q_out.shape)}")
    rc = lib().fp8kv_rope_insert(q.data_ptr(), q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
                                 positions.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1],
                                 int(interleaved), q_out.data_ptr(), slot_mapping.data_ptr(), T, Hq, Hkv, D,
                                 _ptr(k_scale), _ptr(v_scale), k_cache.data_ptr(), v_cache.data_ptr(), num_pages,
                                 page_size, dt, _stream(stream, k_cache))
    _check("fp8kv_rope_insert", rc)
    return q_out


def fp8kv_paged_attention_plan(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left, split_tokens=0):
    ns, st = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().fp8kv_paged_attention_plan(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                          split_tokens, ctypes.byref(ns), ctypes.byref(st))
    _check("fp8kv_paged_attention_plan", rc)
    return ns.value, st.value


def fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                         split_tokens=0) -> int:
    n = lib().fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len,
                                                   window_left, split_tokens)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("fp8kv_paged_attention_workspace_size: bad arguments")
    return n


def fp8kv_paged_attention(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale, v_scale,
                          sm_scale, window_left=-1, split_tokens=0, workspace=None, out=None,
                          num_pages=None, stream=None):
    """q bf16 [B][M][Hq][D]; caches [num_pages][Hkv][page_size][D] (or INT4 pages,
    fp8kv_int4_cache); block_table int32 [B][max_pages_per_seq]; seq_lens int32 [B] (context incl. the M new rows).
    Returns out bf16 [B][M][Hq][D].  ``workspace`` (uint8 CUDA tensor) is
    allocated by torch here when not given and needed."""
    dt = _cache_dtype(k_cache)
    _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    B, M, Hq, D = q.shape
    P, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
    if dt == FP8KV_CACHE_INT4:
        _int4_call(q, k_cache, block_table, seq_lens, k_scale, v_scale, out, num_pages)
    if num_pages is None:
        num_pages = P
    need = fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                                split_tokens)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    if out is None:
        out = _empty_like(q, stream)
    rc = lib().fp8kv_paged_attention(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), int(max_seq_len), B, M, Hq, Hkv, D, page_size, int(num_pages), _ptr(k_scale),
        _ptr(v_scale), float(sm_scale), int(window_left), int(split_tokens), _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _ptr(out), _stream(stream, q))
    _check("fp8kv_paged_attention", rc)
    return out


def fp8kv_append_paged_attention(k_new, v_new, q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale,
                                 v_scale, sm_scale, window_left=-1, split_tokens=0, workspace=None, out=None,
                                 num_pages=None, stream=None):
    """fp8kv_paged_attention after writing the M new tokens of each sequence
    (k_new, v_new bf16 [B][M][Hkv][D]) to the cache at positions L - M + m."""
    dt = _cache_dtype(k_cache)
    _dev(k_new, "k_new", torch.bfloat16), _dev(v_new, "v_new", torch.bfloat16)
    _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    B, M, Hq, D = q.shape
    P, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
    if dt == FP8KV_CACHE_INT4:
        _int4_call(q, k_cache, block_table, seq_lens, k_scale, v_scale, out, num_pages)
    if tuple(k_new.shape) != (B, M, Hkv, D) or tuple(v_new.shape) != (B, M, Hkv, D):
        raise ValueError("k_new, v_new must be [B][M][Hkv][D]")
    if num_pages is None:
        num_pages = P
    need = fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                                split_tokens)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    if out is None:
        out = _empty_like(q, stream)
    rc = lib().fp8kv_append_paged_attention(
        _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, M, Hq, Hkv, D, page_size, int(num_pages),
        _ptr(k_scale), _ptr(v_scale), float(sm_scale), int(window_left), int(split_tokens), _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _ptr(out), _stream(stream, q))
    _check("fp8kv_append_paged_attention", rc)
    return out


def fp8kv_paged_attention_per_head(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale, v_scale,
                                   sm_scale, window_left=-1, split_tokens=0, workspace=None, out=None,
                                   num_pages=None, k_new=None, v_new=None, stream=None):
    """fp8kv_paged_attention on an E4M3 cache with per-head scales fp32 [Hkv];
    with k_new, v_new (bf16 [B][M][Hkv][D]) the append variant
    (fp8kv_append_paged_attention_per_head)."""
    _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache", torch.uint8), _dev(v_cache, "v_cache", torch.uint8)
    _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    B, M, Hq, D = q.shape
    P, Hkv, page_size = _cache_shape(k_cache, v_cache, FP8KV_CACHE_E4M3, D)
    _head_scales(k_scale, v_scale, Hkv)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        _dev(k_new, "k_new", torch.bfloat16), _dev(v_new, "v_new", torch.bfloat16)
        if tuple(k_new.shape) != (B, M, Hkv, D) or tuple(v_new.shape) != (B, M, Hkv, D):
            raise ValueError("k_new, v_new must be [B][M][Hkv][D]")
    if num_pages is None:
        num_pages = P
    need = fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                                split_tokens)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    if out is None:
        out = _empty_like(q, stream)
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
            int(max_seq_len), B, M, Hq, Hkv, D, page_size, int(num_pages), _ptr(k_scale), _ptr(v_scale),
            float(sm_scale), int(window_left), int(split_tokens), _ptr(workspace),
            workspace.numel() if workspace is not None else 0, _ptr(out), _stream(stream))
    if k_new is None:
        _check("fp8kv_paged_attention_per_head", lib().fp8kv_paged_attention_per_head(*args))
    else:
        _check("fp8kv_append_paged_attention_per_head",
               lib().fp8kv_append_paged_attention_per_head(_ptr(k_new), _ptr(v_new), *args))
    return out


def fp8kv_append_paged_attention_per_head(k_new, v_new, q, k_cache, v_cache, block_table, seq_lens, max_seq_len,
                                          k_scale, v_scale, sm_scale, window_left=-1, split_tokens=0,
                                          workspace=None, out=None, num_pages=None, stream=None):
    """fp8kv_append_paged_attention on an E4M3 cache with per-head scales fp32 [Hkv]."""
    if k_new is None or v_new is None:
        raise ValueError("k_new and v_new are required")
    return fp8kv_paged_attention_per_head(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale, v_scale,
                                          sm_scale, window_left, split_tokens, workspace, out, num_pages, k_new,
                                          v_new, stream)


class _Owned:
    """The tensors that a prepared call allocated for itself, on the stream that
    was current then.  Another stream is ordered behind that allocation before
    the first call on it, and the tensors are recorded on it, so that dropping
    them while it still runs does not hand their memory out."""

    def __init__(self, tensors):
        self.tensors = tensors
        self.handles, self.ready = None, None
        if self.tensors:
            device = self.tensors[0].get_device()
            self.handles = {torch._C._cuda_getCurrentRawStream(device)}
            with torch.cuda.device(device):
                if not torch.cuda.is_current_stream_capturing():
                    self.ready = torch.cuda.Event()
                    self.ready.record()

    def before_call(self, stream, handle):
        if self.handles is None or handle in self.handles:
            return
        raw = stream is not None and not hasattr(stream, "cuda_stream")
        s = torch.cuda.ExternalStream(handle) if raw else torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(s):
            if torch.cuda.is_current_stream_capturing():
                # (torch.cuda.graph waits for the device before it captures; an
                # event of work outside cannot be waited for inside)
                return
        if self.ready is not None:
            s.wait_event(self.ready)
        if not raw:
            # a raw handle's stream may be destroyed before the tensors are freed
            for t in self.tensors:
                t.record_stream(s)
        self.handles.add(handle)


class PreparedAttention:
    """fp8kv_append_paged_attention (k_new, v_new given),
    fp8kv_paged_attention, or with tree_mask (int64 [B][M]) fp8kv_tree_attention
    over fixed tensors, marshalled once: each call
    passes the prepared arguments and the stream, nothing else.  For serving
    loops whose caches, metadata and buffers stay at fixed addresses; the
    tensors must outlive the object, and the object its calls on a raw stream
    handle and the graphs that captured it.  Calls share the workspace and the
    output: on several streams they need one object each."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale, v_scale, sm_scale,
                 window_left=-1, split_tokens=0, workspace=None, out=None, k_new=None, v_new=None, num_pages=None,
                 tree_mask=None):
        dt = _cache_dtype(k_cache)
        _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
        _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
        B, M, Hq, D = q.shape
        P, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
        if dt == FP8KV_CACHE_INT4:
            _int4_call(q, k_cache, block_table, seq_lens, k_scale, v_scale, out, num_pages)
        if tree_mask is not None:
            _tree_call(q, k_cache, v_cache, block_table, seq_lens, tree_mask, k_scale, v_scale, out, num_pages, dt)
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        if k_new is not None:
            for t, n in ((k_new, "k_new"), (v_new, "v_new")):
                _dev(t, n, torch.bfloat16)
                if tuple(t.shape) != (B, M, Hkv, D):
                    raise ValueError(f"{n} must be [B][M][Hkv][D]")
        need = fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left,
                                                    split_tokens)
        own = []
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            own.append(workspace)
        if out is None:
            out = torch.empty_like(q)
            own.append(out)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        self._own = _Owned(own)
        self.out, self._keep = out, (q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, workspace, k_new,
                                     v_new, tree_mask)
        if tree_mask is not None:
            self._fn, self._name = lib().fp8kv_tree_attention, "fp8kv_tree_attention"
            self._args = _tree_args(q, k_cache, v_cache, dt, block_table, seq_lens, max_seq_len, tree_mask, k_scale,
                                    v_scale, sm_scale, window_left, split_tokens, workspace, out, k_new, v_new,
                                    num_pages)
            return
        args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                int(max_seq_len), B, M, Hq, Hkv, D, page_size, int(P if num_pages is None else num_pages),
                _ptr(k_scale), _ptr(v_scale), float(sm_scale), int(window_left), int(split_tokens), _ptr(workspace),
                workspace.numel() if workspace is not None else 0, _ptr(out))
        if k_new is not None:
            self._fn, self._name = lib().fp8kv_append_paged_attention, "fp8kv_append_paged_attention"
            self._args = (_ptr(k_new), _ptr(v_new), *args)
        else:
            self._fn, self._name = lib().fp8kv_paged_attention, "fp8kv_paged_attention"
            self._args = args

    def __call__(self, stream=None):
        handle = _stream(stream, self.out)
        self._own.before_call(stream, handle)
        rc = self._fn(*self._args, handle)
        if rc:
            raise Fp8kvError(self._name, rc)
        return self.out


def fp8kv_paged_attention_noalloc(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, k_scale, v_scale,
                                  sm_scale, out, window_left=-1, split_tokens=0, num_pages=None, stream=None):
    """fp8kv_paged_attention with the library's own fixed device workspace, for
    callers that cannot allocate device memory: ``out`` must be given, nothing
    is allocated here or in the library."""
    dt = _cache_dtype(k_cache)
    _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    _dev(out, "out", torch.bfloat16)
    if out.shape != q.shape or out.device != q.device:
        raise ValueError(f"out must have the shape and device of q {tuple(q.shape)}, got {tuple(out.shape)}")
    B, M, Hq, D = q.shape
    P, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
    if dt == FP8KV_CACHE_INT4:
        _int4_call(q, k_cache, block_table, seq_lens, k_scale, v_scale, out, num_pages)
    rc = lib().fp8kv_paged_attention_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), B, M, Hq, Hkv, D, page_size, int(P if num_pages is None else num_pages),
        _ptr(k_scale), _ptr(v_scale), float(sm_scale), int(window_left), int(split_tokens), _ptr(out),
        _stream(stream, q))
    _check("fp8kv_paged_attention_noalloc", rc)
    return out


def _tree_rows(t: torch.Tensor, name: str, dtype, B: int, M: int):
    _dev(t, name)
    if t.dtype != dtype and not (dtype == torch.int64 and name == "tree_mask" and t.dtype == torch.uint64):
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (B, M):
        raise ValueError(f"{name} must be {(B, M)}, got {tuple(t.shape)}")
    return t


def fp8kv_tree_metadata(parents, seq_lens, block_table, page_size, max_seq_len, num_pages, tree_mask=None,
                        positions=None, slot_mapping=None, stream=None):
    """What a step over trees of drafted tokens needs from parents (int32 [B][M],
    -1: padding; node 0 is the root): returns tree_mask (the bits of a node and its
    ancestors), positions and slot_mapping, int64 [B][M] each.  seq_lens int32 [B]
    (the M nodes included), block_table int32 [B][max_pages_per_seq]."""
    _dev(parents, "parents", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    _dev(block_table, "block_table", torch.int32)
    if parents.dim() != 2:
        raise ValueError("parents must be [B][M]")
    B, M = parents.shape
    if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError(f"block_table must be [{B}][pages] and seq_lens [{B}]")
    outs = []
    for t, n in ((tree_mask, "tree_mask"), (positions, "positions"), (slot_mapping, "slot_mapping")):
        if t is not None:
            _tree_rows(t, n, torch.int64, B, M)
        elif stream is None:
            # (three allocations are faster than the views of one)
            t = torch.empty((B, M), dtype=torch.int64, device=parents.device)
        else:
            with _at(stream):
                t = torch.empty((B, M), dtype=torch.int64, device=parents.device)
        outs.append(t)
    tree_mask, positions, slot_mapping = outs
    rc = lib().fp8kv_tree_metadata(parents.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                                   block_table.shape[1], int(max_seq_len), B, M, int(num_pages), int(page_size),
                                   tree_mask.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(),
                                   _stream(stream, parents))
    _check("fp8kv_tree_metadata", rc)
    return tree_mask, positions, slot_mapping


def _tree_call(q, k_cache, v_cache, block_table, seq_lens, tree_mask, k_scale, v_scale, out, num_pages, dt):
    """Checks of a tree call beyond the library's own: what it cannot see from pointers."""
    B, M = q.shape[:2]
    _tree_rows(tree_mask, "tree_mask", torch.int64, B, M)
    if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError(f"block_table must be [{B}][pages] and seq_lens [{B}]")
    if dt != FP8KV_CACHE_BF16:
        _one_scale(k_scale, v_scale)
    if out is not None and _dev(out, "out", torch.bfloat16).shape != q.shape:
        raise ValueError("out must have the shape of q")
    if num_pages is not None and num_pages > k_cache.shape[0]:
        raise ValueError(f"num_pages is {num_pages}, the cache has {k_cache.shape[0]}")


def _tree_args(q, k_cache, v_cache, dt, block_table, seq_lens, max_seq_len, tree_mask, k_scale, v_scale, sm_scale,
               window_left, split_tokens, workspace, out, k_new, v_new, num_pages):
    B, M, Hq, D = q.shape
    P, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
    return (_ptr(k_new), _ptr(v_new), _ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), int(max_seq_len), _ptr(tree_mask), B, M, Hq, Hkv, D, page_size,
            int(P if num_pages is None else num_pages), _ptr(k_scale), _ptr(v_scale), float(sm_scale),
            int(window_left), int(split_tokens), _ptr(workspace), workspace.numel() if workspace is not None else 0,
            _ptr(out))


def fp8kv_tree_attention(q, k_cache, v_cache, block_table, seq_lens, tree_mask, max_seq_len, k_scale, v_scale, sm_scale,
                         window_left=-1, split_tokens=0, workspace=None, out=None, num_pages=None, k_new=None,
                         v_new=None, stream=None):
    """fp8kv_paged_attention for the M nodes of a tree: row m sees the cached keys
    before the nodes and the nodes in tree_mask (int64 [B][M], fp8kv_tree_metadata).
    Padding rows (mask 0) become zeros.  With k_new, v_new (bf16 [B][M][Hkv][D]) the
    nodes' rows are appended first.  Any cache type, M up to 64."""
    dt = _cache_dtype(k_cache)
    _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache")
    _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
    B, M, Hq, D = q.shape
    _, Hkv, page_size = _cache_shape(k_cache, v_cache, dt, D)
    _tree_call(q, k_cache, v_cache, block_table, seq_lens, tree_mask, k_scale, v_scale, out, num_pages, dt)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        for t, n in ((k_new, "k_new"), (v_new, "v_new")):
            if _dev(t, n, torch.bfloat16).shape != (B, M, Hkv, D):
                raise ValueError(f"{n} must be [B][M][Hkv][D]")
    need = fp8kv_paged_attention_workspace_size(B, M, Hq, Hkv, D, page_size, max_seq_len, window_left, split_tokens)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    if out is None:
        out = _empty_like(q, stream)
    args = _tree_args(q, k_cache, v_cache, dt, block_table, seq_lens, max_seq_len, tree_mask, k_scale, v_scale,
                      sm_scale, window_left, split_tokens, workspace, out, k_new, v_new, num_pages)
    _check("fp8kv_tree_attention", lib().fp8kv_tree_attention(*args, _stream(stream, q)))
    return out


def _prob_rows(t: torch.Tensor, name: str, B: int, M: int, V: int) -> int:
    """Probabilities [B][M][V] with dense rows; returns the elements between rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    st = t.stride()
    if t.shape != (B, M, V) or (V > 1 and st[2] != 1) or (B > 1 and M > 1 and st[0] != M * st[1]):
        raise ValueError(f"{name} must be {(B, M, V)} with dense rows, all the same distance apart")
    step = st[1] if M > 1 else st[0] if B > 1 else V
    if step < V:
        raise ValueError(f"{name} must have rows that do not overlap")
    return step


def fp8kv_verify_tree(target_probs, draft_probs, tokens, parents, uniforms, out_tokens=None, num_tokens=None, path=None,
                      stream=None):
    """Which drafted tokens of a tree stand, and the token after them: target_probs
    fp32 or bf16 [B][M][V] (row n: the token behind node n), draft_probs the same or
    None (what n's children were drawn from; None: they were chosen), tokens and
    parents int32 [B][M], uniforms fp32 [B][M] in [0, 1).  Returns out_tokens int32
    [B][M] (the tokens that stand, the next one, -1s), num_tokens int32 [B] (how many
    those are: 0 .. M, 0 where a root row without a sum has none to draw) and path int32 [B][M] (node 0, the nodes that stand, -1s)."""
    if target_probs.dim() != 3:
        raise ValueError("target_probs must be [B][M][V]")
    B, M, V = target_probs.shape
    if target_probs.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"target_probs must be {torch.float32} or {torch.bfloat16}, got {target_probs.dtype}")
    p_stride, q_stride = _prob_rows(target_probs, "target_probs", B, M, V), 0
    if draft_probs is not None:
        if draft_probs.dtype != target_probs.dtype:
            raise ValueError(f"draft_probs must be {target_probs.dtype}, got {draft_probs.dtype}")
        q_stride = _prob_rows(draft_probs, "draft_probs", B, M, V)
    _tree_rows(tokens, "tokens", torch.int32, B, M), _tree_rows(parents, "parents", torch.int32, B, M)
    _tree_rows(uniforms, "uniforms", torch.float32, B, M)
    if out_tokens is None or num_tokens is None or path is None:
        with _at(stream):
            made = torch.empty((2 * M + 1) * B, dtype=torch.int32, device=target_probs.device)
        out_tokens = made[:B * M].view(B, M) if out_tokens is None else out_tokens
        path = made[B * M:2 * B * M].view(B, M) if path is None else path
        num_tokens = made[2 * B * M:] if num_tokens is None else num_tokens
    _tree_rows(out_tokens, "out_tokens", torch.int32, B, M), _tree_rows(path, "path", torch.int32, B, M)
    if _dev(num_tokens, "num_tokens", torch.int32).shape != (B,):
        raise ValueError(f"num_tokens must be {(B,)}, got {tuple(num_tokens.shape)}")
    rc = lib().fp8kv_verify_tree(target_probs.data_ptr(), p_stride, _ptr(draft_probs), q_stride,
                                 0 if target_probs.dtype == torch.float32 else 1, tokens.data_ptr(), parents.data_ptr(),
                                 uniforms.data_ptr(), B, M, V, out_tokens.data_ptr(), num_tokens.data_ptr(),
                                 path.data_ptr(), _stream(stream, target_probs))
    _check("fp8kv_verify_tree", rc)
    return out_tokens, num_tokens, path


class PreparedKeepPath:
    """fp8kv_cache_keep_path over fixed tensors, marshalled once: in every layer's
    caches (lists of tensors of one type and shape) the rows of the nodes in path
    (int32 [B][M], fp8kv_verify_tree) go to the first of the tree's indices, and
    new_seq_lens (int32 [B]) becomes the length up to them.  The tensors must outlive
    the object, and the object its calls on a raw stream handle and the graphs that
    captured it."""

    def __init__(self, k_caches, v_caches, block_table, seq_lens, path, max_seq_len, new_seq_lens=None, num_pages=None):
        n = len(k_caches)
        if n == 0 or len(v_caches) != n:
            raise ValueError("k_caches and v_caches must be lists of the same length, one entry a layer")
        first = k_caches[0]
        dt = _cache_dtype(first)
        P, Hkv, page_size = _cache_shape(first, v_caches[0], dt)
        for t in (*k_caches, *v_caches):
            if _dev(t, "caches").dtype != first.dtype or t.shape != first.shape or t.device != first.device:
                raise ValueError("all caches must have the same type, shape and device")
        at, size = sorted(t.data_ptr() for t in (*k_caches, *v_caches)), first.numel() * first.element_size()
        if any(b - a < size for a, b in zip(at, at[1:])):
            raise ValueError("every layer must have a K and a V cache of its own")
        _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32)
        _dev(path, "path", torch.int32)
        if path.dim() != 2:
            raise ValueError("path must be [B][M]")
        B, M = path.shape
        if block_table.dim() != 2 or block_table.shape[0] != B or seq_lens.numel() != B:
            raise ValueError(f"block_table must be [{B}][pages] and seq_lens [{B}]")
        if num_pages is not None and num_pages > P:
            raise ValueError(f"num_pages is {num_pages}, the caches have {P}")
        own = []
        if new_seq_lens is None:
            new_seq_lens = torch.empty(B, dtype=torch.int32, device=path.device)
            own.append(new_seq_lens)
        if _dev(new_seq_lens, "new_seq_lens", torch.int32).numel() != B:
            raise ValueError(f"new_seq_lens must be [{B}]")
        self._own = _Owned(own)
        self.new_seq_lens = new_seq_lens
        self._keep = (list(k_caches), list(v_caches), block_table, seq_lens, path)
        ptrs = ctypes.c_void_p * n
        self._k, self._v = (ptrs(*(t.data_ptr() for t in c)) for c in (k_caches, v_caches))
        self._args = (ctypes.addressof(self._k), ctypes.addressof(self._v), n, dt, block_table.data_ptr(),
                      block_table.shape[1], seq_lens.data_ptr(), int(max_seq_len), path.data_ptr(), B, M, Hkv,
                      128 if dt == FP8KV_CACHE_INT4 else first.shape[3], int(P if num_pages is None else num_pages),
                      page_size, new_seq_lens.data_ptr())
        self._fn = lib().fp8kv_cache_keep_path

    def __call__(self, stream=None):
        handle = _stream(stream, self.new_seq_lens)
        self._own.before_call(stream, handle)
        _check("fp8kv_cache_keep_path", self._fn(*self._args, handle))
        return self.new_seq_lens


def fp8kv_cache_keep_path(k_caches, v_caches, block_table, seq_lens, path, max_seq_len, new_seq_lens=None,
                          num_pages=None, stream=None):
    """Move the accepted path's rows together in every layer's caches (see
    PreparedKeepPath); returns new_seq_lens."""
    with _at(stream):
        call = PreparedKeepPath(k_caches, v_caches, block_table, seq_lens, path, max_seq_len, new_seq_lens, num_pages)
    return call(stream)


class fp8kv_layer(ctypes.Structure):
    """One layer of fp8kv_paged_attention_layers (include/fp8kv.h)."""
    _fields_ = [("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int), ("max_seq_len", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("window_left", ctypes.c_int), ("sm_scale", ctypes.c_float)]


def fp8kv_paged_attention_layers_workspace_size(n_layers, B, M, Hq, Hkv) -> int:
    n = lib().fp8kv_paged_attention_layers_workspace_size(n_layers, B, M, Hq, Hkv)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("fp8kv_paged_attention_layers_workspace_size: bad arguments")
    return n


class PagedAttentionLayers:
    """A prepared fp8kv_paged_attention_layers call over fixed tensors (the
    layers' persistent caches, metadata and buffers): the descriptors are
    marshalled once; each call passes them, the workspace and the stream.

    layers: dicts with q, k_new, v_new (or None), k_cache, v_cache,
    block_table, seq_lens, max_seq_len, k_scale, v_scale, sm_scale,
    window_left, out -- the arguments of fp8kv_append_paged_attention."""

    def __init__(self, layers, workspace=None):
        if not layers:
            raise ValueError("no layers")
        q0 = layers[0]["q"]
        B, M, Hq, D = q0.shape
        P0, Hkv, page_size, _ = layers[0]["k_cache"].shape
        self.shape = (B, M, Hq, Hkv, D, page_size)
        arr = (fp8kv_layer * len(layers))()
        self._keep = []
        for i, d in enumerate(layers):
            q, kc, vc = d["q"], d["k_cache"], d["v_cache"]
            _dev(q, "q", torch.bfloat16), _dev(kc, "k_cache", torch.uint8), _dev(vc, "v_cache", torch.uint8)
            _dev(d["block_table"], "block_table", torch.int32), _dev(d["seq_lens"], "seq_lens", torch.int32)
            _dev(d["out"], "out", torch.bfloat16)
            if tuple(q.shape) != (B, M, Hq, D) or tuple(d["out"].shape) != (B, M, Hq, D):
                raise ValueError(f"layer {i}: q and out must be {(B, M, Hq, D)}")
            if tuple(kc.shape[1:]) != (Hkv, page_size, D) or kc.shape != vc.shape:
                raise ValueError(f"layer {i}: caches must be [pages][{Hkv}][{page_size}][{D}]")
            kn, vn = d.get("k_new"), d.get("v_new")
            if (kn is None) != (vn is None):
                raise ValueError(f"layer {i}: k_new and v_new go together")
            if kn is not None:
                for t, n in ((kn, "k_new"), (vn, "v_new")):
                    _dev(t, n, torch.bfloat16)
                    if tuple(t.shape) != (B, M, Hkv, D):
                        raise ValueError(f"layer {i}: {n} must be {(B, M, Hkv, D)}")
            bt = d["block_table"]
            arr[i] = fp8kv_layer(_ptr(q), _ptr(kn), _ptr(vn), _ptr(kc), _ptr(vc), _ptr(bt), _ptr(d["seq_lens"]),
                                 _ptr(d["k_scale"]), _ptr(d["v_scale"]), _ptr(d["out"]), bt.shape[1],
                                 int(d["max_seq_len"]), int(d.get("num_pages") or kc.shape[0]),
                                 int(d.get("window_left", -1)), float(d["sm_scale"]))
            self._keep.append(d)
        self.layers = arr
        self.n = len(layers)
        self.ws_bytes = fp8kv_paged_attention_layers_workspace_size(self.n, B, M, Hq, Hkv)
        own = []
        if workspace is None:
            # the counters at its start must be zero before the first call, on
            # whatever stream that is
            workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=q0.device)
            own.append(workspace)
        self._own = _Owned(own)
        self.workspace = workspace

    def __call__(self, stream=None):
        B, M, Hq, Hkv, D, page_size = self.shape
        handle = _stream(stream)
        self._own.before_call(stream, handle)
        rc = lib().fp8kv_paged_attention_layers(ctypes.byref(self.layers), self.n, B, M, Hq, Hkv, D, page_size,
                                                FP8KV_CACHE_E4M3, _ptr(self.workspace), self.workspace.numel(), handle)
        _check("fp8kv_paged_attention_layers", rc)


def fp8kv_paged_attention_layers(layers, workspace=None, stream=None):
    """Run the verifier step of several layers in one launch (see
    PagedAttentionLayers); returns the prepared call for reuse."""
    call = PagedAttentionLayers(layers, workspace)
    call(stream)
    return call


def fp8kv_e4m3_encode_bits(first: int, n: int, out: torch.Tensor, stream=None):
    _dev(out, "out", torch.uint8)
    rc = lib().fp8kv_e4m3_encode_bits(first, n, _ptr(out), _stream(stream))
    _check("fp8kv_e4m3_encode_bits", rc)


def fp8kv_selftest_bounded_wait(limit_us: int, stream=None):
    """Launch the kernel whose barrier wait runs out after limit_us (sets
    DEV_WAIT_TIMEOUT in the device status word)."""
    _check("fp8kv_selftest_bounded_wait", lib().fp8kv_selftest_bounded_wait(int(limit_us), _stream(stream)))


def fp8kv_last_dispatch() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().fp8kv_last_dispatch(buf, 512)
    return buf.value.decode()


def fp8kv_launch_count():
    """Kernel launches the library has made in this process."""
    return int(lib().fp8kv_launch_count())


def fp8kv_device_status(clear: bool = False) -> int:
    s = ctypes.c_uint(0)
    _check("fp8kv_device_status", lib().fp8kv_device_status(ctypes.byref(s), int(clear)))
    return s.value
