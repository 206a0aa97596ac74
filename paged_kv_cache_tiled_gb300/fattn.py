"""ctypes binding of libfattn (include/fattn.h).

Argument marshalling only: every function here checks dtypes/shapes, passes
device pointers, sizes and the current CUDA stream to the C entry point of the
same name, and raises ``FattnError`` on a non-OK status.  All arithmetic runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing this module fails loudly when ``libfattn.so`` has not been built.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfattn.so")

(FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_BOUNDS, FA_ERR_WORKSPACE,
 FA_ERR_NO_BLOCKS) = range(8)
FA_BF16, FA_F32 = 0, 1

# every symbol declared in include/fattn.h
EXPORTS = [
    "fa_status_string", "fa_prefill", "fa_prefill_masked_workspace_size", "fa_prefill_masked", "fa_stage_bf16",
    "fa_cache_append", "fa_paged_attn_workspace_size", "fa_paged_attn", "fa_get_error", "fa_debug_gather_kv",
    "fa_debug_set_wait_limit", "fa_debug_force_timeout", "fa_last_launch_count", "fa_paged_attn_noalloc",
    "fa_cache_append_rope", "fa_decode_graph_create", "fa_decode_graph_launch", "fa_decode_graph_kernel_count",
    "fa_decode_graph_destroy", "fa_pool_create", "fa_pool_destroy", "fa_pool_add_seq", "fa_pool_fork",
    "fa_pool_append", "fa_pool_release", "fa_pool_tables", "fa_pool_num_free", "fa_pool_refcount", "fa_pool_seq_len",
    "fa_copy_blocks", "fa_cache_append_fp8", "fa_paged_attn_fp8", "fa_prefill_host", "fa_mask_tile_classes",
    "fa_prefill_rows", "fa_prefill_mod_workspace_size", "fa_prefill_mod", "fa_cache_append_mrope",
    "fa_paged_attn_mod_workspace_size", "fa_paged_attn_mod", "fa_paged_attn_accum_workspace_size",
    "fa_paged_attn_accum", "fa_cache_evict_workspace_size", "fa_cache_evict", "fa_cache_append_fp8_scaled",
    "fa_paged_attn_fp8_scaled_workspace_size", "fa_paged_attn_fp8_scaled", "fa_block_bounds",
    "fa_block_select_workspace_size", "fa_block_select", "fa_paged_attn_blocks",
]
NOALLOC_SCRATCH_BYTES = 32 << 20  # FA_NOALLOC_SCRATCH_BYTES


class FattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with paged_kv_cache_tiled_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    Z = ctypes.c_size_t
    sig = {
        "fa_status_string": (ctypes.c_char_p, [I]),
        "fa_prefill": (I, [P, P, P, P, I, I, I, I, I, I, F, P, P]),
        "fa_prefill_host": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]),
        "fa_prefill_rows": (I, [P, P, P, P, I, I, I, I, I, I, F, I, I, I, P]),
        "fa_prefill_masked_workspace_size": (Z, [I]),
        "fa_prefill_masked": (I, [P, P, P, P, P, I, I, I, I, I, I, F, P, P, Z, P]),
        "fa_stage_bf16": (I, [P, P, Z, P]),
        "fa_mask_tile_classes": (I, [P, I, I, P, P, P]),
        "fa_cache_append": (I, [P, P, P, P, P, I, I, I, I, I, P]),
        "fa_paged_attn_workspace_size": (Z, [I, I, I, I, I, I]),
        "fa_paged_attn": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I, P, Z, P]),
        "fa_get_error": (I, [P]),
        "fa_debug_gather_kv": (I, [P, P, P, P, I, I, I, I, I, I, P]),
        "fa_debug_set_wait_limit": (None, [ctypes.c_ulonglong]),
        "fa_cache_append_rope": (I, [P, P, P, P, P, I, P, P, P, P, I, I, I, I, I, I, P]),
        "fa_decode_graph_create": (I, [P, P, P, P, I, I, P, P, P, P, P, P, P, I, I, I, I, I, I, I,
                                       ctypes.c_float, I, I, P, ctypes.c_size_t]),
        "fa_decode_graph_launch": (I, [P, P]),
        "fa_decode_graph_kernel_count": (I, [P]),
        "fa_decode_graph_destroy": (None, [P]),
        "fa_pool_create": (I, [P, I, I]),
        "fa_pool_destroy": (None, [P]),
        "fa_pool_add_seq": (I, [P, P]),
        "fa_pool_fork": (I, [P, I, I, P, P, P]),
        "fa_pool_append": (I, [P, I, I, P]),
        "fa_pool_release": (I, [P, I]),
        "fa_pool_tables": (I, [P, P, I, P, P]),
        "fa_pool_num_free": (I, [P]),
        "fa_pool_refcount": (I, [P, I]),
        "fa_pool_seq_len": (I, [P, I]),
        "fa_copy_blocks": (I, [P, P, P, I, I, I, I, P]),
        "fa_cache_append_fp8": (I, [P, P, P, P, P, I, I, I, I, ctypes.c_float, ctypes.c_float, I, P]),
        "fa_paged_attn_fp8": (I, [P, P, P, ctypes.c_float, ctypes.c_float, P, P, P, P, I, I, I, I, I, I, I, I,
                                  ctypes.c_float, I, I, P, ctypes.c_size_t, P]),
        "fa_debug_force_timeout": (None, [I]),
        "fa_paged_attn_noalloc": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I, P]),
        "fa_last_launch_count": (I, []),
        "fa_prefill_mod_workspace_size": (Z, [I, I]),
        "fa_prefill_mod": (I, [P, P, P, P, P, I, I, I, I, I, I, F, F, P, I, P, P, P, Z, P]),
        "fa_cache_append_mrope": (I, [P, P, P, P, I, P, P, I, P, P, P, P, I, I, I, I, I, I, P]),
        "fa_paged_attn_mod_workspace_size": (Z, [I, I, I, I, I, I, I]),
        "fa_paged_attn_mod": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, F, P, I, P, I, I, P, Z, P]),
        "fa_paged_attn_accum_workspace_size": (Z, [I, I, I, I, I, I, I]),
        "fa_paged_attn_accum": (I, [P, P, P, P, P, P, P, P, P, P, I, F, I, I, I, I, I, I, I, I, F, F, P, I, P, I, I, P,
                                    Z, P]),
        "fa_cache_evict_workspace_size": (Z, [I, I, I, I]),
        "fa_cache_evict": (I, [P, P, P, I, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, I, I, P, Z, P]),
        "fa_cache_append_fp8_scaled": (I, [P, P, P, P, P, I, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P]),
        "fa_paged_attn_fp8_scaled_workspace_size": (Z, [I, I, I, I, I, I, I]),
        "fa_paged_attn_fp8_scaled": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I, P, Z, P]),
        "fa_block_bounds": (I, [P, P, P, P, P, P, I, I, I, I, I, I, I, P]),
        "fa_block_select_workspace_size": (Z, [I, I, I, I, I, I]),
        "fa_block_select": (I, [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, I, I, P, Z, P]),
        "fa_paged_attn_blocks": (I, [P, P, P, P, P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, I, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.fa_status_string(int(status)).decode()


fa_status_string = status_string


def _check(st: int, where: str):
    if st != FA_OK:
        raise FattnError(st, where)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _device_of(q, name: str) -> int:
    """The current device, on which q must live: a call runs on a stream of the current device."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch._C._cuda_getDevice()
    if q.get_device() != cur:
        raise ValueError(f"{name} is on {q.device}, but the current device is cuda:{cur}")
    return cur


def _arg(t, name: str, dtype, shape, dev: int):
    """Checks a tensor's type, shape, layout and device in as few attribute reads as a small call can
    afford; returns its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name: str, dtype, shape, dev: int):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _tensor(t, name: str, dtype, dev: int):
    """_arg for a tensor that the call takes its sizes from."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _arg(t, name, dtype, getattr(t, "shape", ()), dev)


def _dims(t, name: str, n: int):
    """The shape of a tensor of n dims."""
    shape = getattr(t, "shape", ())
    if len(shape) != n or not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor of {n} dims")
    return shape


def _empty(shape, dtype, dev: int, stream):
    """A tensor that a call makes itself.  For a call on a stream other than the current one it is memory of that
    stream (the current stream's may still be in use by work queued there), kept until the current stream, on which
    the caller may go on to use it, is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")
    t.record_stream(torch.cuda.current_stream())
    return t


def _int(x, name: str) -> int:
    """x, which a C int has to hold (ctypes would cut it off)."""
    x = operator.index(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits")
    return x


def _workspace(ws, nbytes: int, dev: int, stream):
    """(address, bytes) of the workspace given, or of a new one; the tensor comes last to be kept alive."""
    if nbytes == 0 and ws is None:
        return None, 0, None
    if ws is None:
        ws = _empty(nbytes, torch.uint8, dev, stream)
    elif not isinstance(ws, torch.Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on cuda:{dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _current_stream(stream, dev: int):
    return _stream(stream) if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


# ------------------------------------------------------------------ prefill
def fa_prefill(q, k, v, causal: bool = True, scale: float | None = None, out=None, lse=None, stream=None):
    """softmax(scale * Q K^T [+ causal mask]) V for q [B,T,Hq,d], k/v [B,T,Hkv,d] (bf16)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need(t, n, torch.bfloat16, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if lse is not None:
        _need(lse, "lse", torch.float32)
    _check(_lib.fa_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, Hq, Hkv, d, int(causal), float(scale),
                           _ptr(lse), _stream(stream)), "fa_prefill")
    return out


def fa_prefill_rows(q, k, v, q0: int, Tq: int, Tk: int, causal: bool = True, scale: float | None = None, out=None,
                    stream=None):
    """Query rows [q0, q0+Tq) of every sequence against keys [0, Tk); q/k/v/out
    hold whole sequences [B, T, H, d] and only those rows of `out` are written."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need(t, n, torch.bfloat16, 4)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    _check(_lib.fa_prefill_rows(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, Hq, Hkv, d, int(causal), float(scale),
                                int(q0), int(Tq), int(Tk), _stream(stream)), "fa_prefill_rows")
    return out


def fa_prefill_host(q_host, k_host, v_host, out_host, q, k, v, out, causal: bool = True,
                    scale: float | None = None, stream=None):
    """fa_prefill from and to host memory: the host tensors (bf16, contiguous,
    ideally pinned) are copied into the caller's device buffers q/k/v and the
    result back into out_host, one sequence at a time, with the copies
    overlapping the kernels.  Ordered on `stream`; the host is not synchronised."""
    for n, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _need(t, n, torch.bfloat16, 4)
    for n, t, dev in (("q_host", q_host, q), ("k_host", k_host, k), ("v_host", v_host, v), ("out_host", out_host, out)):
        if not isinstance(t, torch.Tensor) or t.is_cuda:
            raise ValueError(f"{n} must be a host tensor")
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.shape != dev.shape:
            raise ValueError(f"{n} must be a contiguous bf16 tensor shaped like its device buffer")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(_lib.fa_prefill_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), out_host.data_ptr(),
                                _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, T, Hq, Hkv, d, int(causal), float(scale),
                                _stream(stream)), "fa_prefill_host")
    return out_host


def fa_prefill_masked_workspace_size(T: int) -> int:
    return int(_lib.fa_prefill_masked_workspace_size(int(T)))


def fa_prefill_masked(q, k, v, mask, causal: bool = False, scale: float | None = None, out=None, lse=None, ws=None,
                      stream=None):
    """softmax(scale * Q K^T + M [+ causal]) V with an additive fp32 mask M [T, T]."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need(t, n, torch.bfloat16, 4)
    _need(mask, "mask", torch.float32, 2)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    nbytes = fa_prefill_masked_workspace_size(T)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(_lib.fa_prefill_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), B, T, Hq, Hkv, d, int(causal),
                                  float(scale), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "fa_prefill_masked")
    return out


def fa_prefill_mod_workspace_size(B: int, T: int) -> int:
    return int(_lib.fa_prefill_mod_workspace_size(int(B), int(T)))


def fa_prefill_mod(q, k, v, causal: bool = True, scale: float | None = None, softcap: float = 0.0,
                   alibi_slopes=None, window: int = 0, prefix_lens=None, doc_ids=None, out=None, lse=None, ws=None,
                   stream=None):
    """fa_prefill with modified scores: logits f(scale q.k) - alibi_slopes[h] |i - j|, f(z) = softcap
    tanh(z / softcap) (softcap > 0); a key is visible when every mask given allows it: causal (or below
    prefix_lens[b]), window, doc_ids [B, T] (runs of equal ids; negative: padding)."""
    B, T, Hq, d = _dims(q, "q", 4)
    Hkv = _dims(k, "k", 4)[2]
    dev, bf16, f32, i32 = _device_of(q, "q"), torch.bfloat16, torch.float32, torch.int32
    if out is None:
        out = _empty(q.shape, bf16, dev, stream)
    window = _int(window, "window")
    wp, wn, ws = _workspace(ws, fa_prefill_mod_workspace_size(B, T), dev, stream) if doc_ids is not None else (None, 0, None)
    _check(_lib.fa_prefill_mod(
        _arg(q, "q", bf16, (B, T, Hq, d), dev), _arg(k, "k", bf16, (B, T, Hkv, d), dev),
        _arg(v, "v", bf16, (B, T, Hkv, d), dev), _arg(out, "out", bf16, (B, T, Hq, d), dev),
        _opt(lse, "lse", f32, (B, Hq, T), dev), B, T, Hq, Hkv, d, 1 if causal else 0,
        d ** -0.5 if scale is None else float(scale), float(softcap), _opt(alibi_slopes, "alibi_slopes", f32, (Hq,), dev), window,
        _opt(prefix_lens, "prefix_lens", i32, (B,), dev), _opt(doc_ids, "doc_ids", i32, (B, T), dev), wp, wn,
        _current_stream(stream, dev)), "fa_prefill_mod")
    return out


def fa_mask_tile_classes(mask, out=None, intervals=None, stream=None):
    """uint8 [ceil(Tq/128), ceil(Tk/128)] classes of an fp32 mask [Tq, Tk]: 0 all -inf, 1 all zero,
    3 zeros forming one run per row among -inf, 2 otherwise.  `intervals` (optional, uint8
    [ceil(Tq/128), ceil(Tk/128), 128, 2]) receives each row's run [lo, hi) in class-3 tiles."""
    _need(mask, "mask", torch.float32, 2)
    Tq, Tk = mask.shape
    shape = ((Tq + 127) // 128, (Tk + 127) // 128)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=mask.device)
    _need(out, "out", torch.uint8, 2)
    if tuple(out.shape) != shape:
        raise ValueError(f"out must have shape {shape}")
    if intervals is not None:
        _need(intervals, "intervals", torch.uint8, 4)
        if tuple(intervals.shape) != shape + (128, 2):
            raise ValueError(f"intervals must have shape {shape + (128, 2)}")
    _check(_lib.fa_mask_tile_classes(_ptr(mask), Tq, Tk, _ptr(out), _ptr(intervals) if intervals is not None else None,
                                     _stream(stream)), "fa_mask_tile_classes")
    return out


def fa_stage_bf16(src, dst=None, stream=None):
    """fp32 -> bf16 (round to nearest even)."""
    _need(src, "src", torch.float32)
    if dst is None:
        dst = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device)
    _need(dst, "dst", torch.bfloat16)
    _check(_lib.fa_stage_bf16(_ptr(src), _ptr(dst), src.numel(), _stream(stream)), "fa_stage_bf16")
    return dst


# -------------------------------------------------------------------- paged
def fa_cache_append(k, v, k_cache, v_cache, slot_mapping, stream=None):
    """Writes k/v [N, Hkv, d] (bf16 or fp32) into the caches [num_blocks, Hkv, 16, d] at slot_mapping[N]."""
    if k.dtype not in (torch.bfloat16, torch.float32) or v.dtype != k.dtype:
        raise ValueError("k, v must both be bf16 or both fp32")
    _need(k, "k", k.dtype, 3)
    _need(v, "v", k.dtype, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    N, Hkv, d = k.shape
    dt = FA_F32 if k.dtype == torch.float32 else FA_BF16
    _check(_lib.fa_cache_append(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), N, Hkv, d,
                                k_cache.shape[0], dt, _stream(stream)), "fa_cache_append")


def fa_cache_append_rope(q, k, v, positions, cos_sin, k_cache, v_cache, slot_mapping, q_out=None, stream=None):
    """Rotary embedding of q [N,Hq,d] and k [N,Hkv,d] at table rows positions[N]
    (cos_sin fp32 [max_pos, d]: cosines then sines), fused with the cache
    append of the rotated k and of v; returns the rotated queries (bf16)."""
    if q.dtype not in (torch.bfloat16, torch.float32) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must all be bf16 or all fp32")
    _need(q, "q", q.dtype, 3)
    _need(k, "k", q.dtype, 3)
    _need(v, "v", q.dtype, 3)
    _need(positions, "positions", torch.int32, 1)
    _need(cos_sin, "cos_sin", torch.float32, 2)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    if q_out is None:
        q_out = torch.empty(N, Hq, d, dtype=torch.bfloat16, device=q.device)
    _need(q_out, "q_out", torch.bfloat16, 3)
    dt = FA_F32 if q.dtype == torch.float32 else FA_BF16
    _check(_lib.fa_cache_append_rope(_ptr(q), _ptr(k), _ptr(v), _ptr(positions), _ptr(cos_sin), cos_sin.shape[0],
                                     _ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), N, Hq, Hkv, d,
                                     k_cache.shape[0], dt, _stream(stream)), "fa_cache_append_rope")
    return q_out


def _pair_axes(x, n: int) -> bytes:
    """n axis numbers as the C call reads them; it checks that there are so many axes.  (bytes() of a number would be that
    many zeros, and of an array its memory.)"""
    try:
        b = x if isinstance(x, bytes) else bytes(x if isinstance(x, (list, tuple)) else [operator.index(a) for a in x])
    except (TypeError, ValueError):  # not a sequence, not whole numbers, outside 0 .. 255
        b = b""
    if len(b) != n:
        raise ValueError(f"pair_axes must be {n} axis numbers")
    return b


def fa_cache_append_mrope(q, k, v, positions, pair_axes, cos_sin, k_cache, v_cache, slot_mapping, q_out=None,
                          stream=None):
    """fa_cache_append_rope with positions [n_axes, N]: channel pair j turns by the table row of
    positions[pair_axes[j]] (pair_axes: d/2 small integers on the host)."""
    N, Hq, d = _dims(q, "q", 3)
    Hkv = _dims(k, "k", 3)[1]
    n_axes = _dims(positions, "positions", 2)[0]
    nb, max_pos = _dims(k_cache, "k_cache", 4)[0], _dims(cos_sin, "cos_sin", 2)[0]
    dev, dt, bf16 = _device_of(q, "q"), q.dtype, torch.bfloat16
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError("q, k, v must all be bf16 or all fp32")
    pair_axes = _pair_axes(pair_axes, d // 2)
    if q_out is None:
        q_out = _empty((N, Hq, d), bf16, dev, stream)
    _check(_lib.fa_cache_append_mrope(
        _arg(q, "q", dt, (N, Hq, d), dev), _arg(k, "k", dt, (N, Hkv, d), dev), _arg(v, "v", dt, (N, Hkv, d), dev),
        _arg(positions, "positions", torch.int32, (n_axes, N), dev), n_axes, pair_axes,
        _arg(cos_sin, "cos_sin", torch.float32, (max_pos, d), dev), max_pos,
        _arg(q_out, "q_out", bf16, (N, Hq, d), dev), _arg(k_cache, "k_cache", bf16, (nb, Hkv, 16, d), dev),
        _arg(v_cache, "v_cache", bf16, (nb, Hkv, 16, d), dev), _arg(slot_mapping, "slot_mapping", torch.int32, (N,), dev),
        N, Hq, Hkv, d, nb, FA_F32 if dt is torch.float32 else FA_BF16, _current_stream(stream, dev)),
        "fa_cache_append_mrope")
    return q_out


class BlockPool:
    """fa_pool_*: host-side block pool with reference counts and prefix
    sharing.  Methods mirror the C functions; arrays are numpy."""

    def __init__(self, num_blocks: int, max_blocks_per_seq: int):
        h = ctypes.c_void_p()
        _check(_lib.fa_pool_create(ctypes.byref(h), num_blocks, max_blocks_per_seq), "fa_pool_create")
        self._h, self.num_blocks, self.max_blocks_per_seq = h, num_blocks, max_blocks_per_seq

    def add_seq(self) -> int:
        s = ctypes.c_int()
        _check(_lib.fa_pool_add_seq(self._h, ctypes.byref(s)), "fa_pool_add_seq")
        return s.value

    def fork(self, parent: int, prefix_len: int):
        """Returns (child, (copy_src, copy_dst)) with (-1, -1) when no copy is needed."""
        c, a, b = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(_lib.fa_pool_fork(self._h, parent, prefix_len, ctypes.byref(c), ctypes.byref(a), ctypes.byref(b)),
               "fa_pool_fork")
        return c.value, (a.value, b.value)

    def append(self, seq: int, n: int) -> np.ndarray:
        slots = np.zeros(max(n, 1), np.int32)
        _check(_lib.fa_pool_append(self._h, seq, n, slots.ctypes.data_as(ctypes.c_void_p)), "fa_pool_append")
        return slots[:n]

    def release(self, seq: int):
        _check(_lib.fa_pool_release(self._h, seq), "fa_pool_release")

    def tables(self, seqs):
        seqs = np.ascontiguousarray(seqs, dtype=np.int32)
        n = len(seqs)
        table = np.zeros((max(n, 1), self.max_blocks_per_seq), np.int32)
        lens = np.zeros(max(n, 1), np.int32)
        _check(_lib.fa_pool_tables(self._h, seqs.ctypes.data_as(ctypes.c_void_p), n,
                                   table.ctypes.data_as(ctypes.c_void_p), lens.ctypes.data_as(ctypes.c_void_p)),
               "fa_pool_tables")
        return table[:n], lens[:n]

    def num_free(self) -> int:
        return int(_lib.fa_pool_num_free(self._h))

    def refcount(self, block: int) -> int:
        return int(_lib.fa_pool_refcount(self._h, block))

    def seq_len(self, seq: int) -> int:
        return int(_lib.fa_pool_seq_len(self._h, seq))

    def close(self):
        if getattr(self, "_h", None):
            _lib.fa_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fa_copy_blocks(k_cache, v_cache, pairs, stream=None):
    """Copies cache block pairs[i, 0] onto pairs[i, 1] (pairs: int32 [n, 2] on the device)."""
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(pairs, "pairs", torch.int32, 2)
    num_blocks, Hkv, _, d = k_cache.shape
    _check(_lib.fa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(pairs), pairs.shape[0], Hkv, d, num_blocks,
                               _stream(stream)), "fa_copy_blocks")


class DecodeGraph:
    """fa_decode_graph_*: the append of k_new/v_new (if given) plus paged
    attention, captured once with these tensors and replayed with one
    submission.  Keep every tensor alive and rewrite contents only."""

    def __init__(self, q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, ws, *, k_new=None, v_new=None,
                 slot_mapping=None, causal: bool = True, scale: float | None = None, max_q_len: int | None = None):
        total_q, Hq, d = q.shape
        num_blocks, Hkv, _, _ = k_cache.shape
        num_seqs, mbps = block_table.shape
        n_new, dt = 0, FA_BF16
        if k_new is not None:
            n_new = k_new.shape[0]
            dt = FA_F32 if k_new.dtype == torch.float32 else FA_BF16
        self._keep = (q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, ws, k_new, v_new, slot_mapping)
        h = ctypes.c_void_p()
        _check(_lib.fa_decode_graph_create(
            ctypes.byref(h), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n_new, dt, _ptr(q), _ptr(k_cache),
            _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(q_lens), _ptr(out), num_seqs, mbps, num_blocks,
            Hq, Hkv, d, int(causal), float(scale if scale is not None else 1.0 / math.sqrt(d)), total_q,
            int(max_q_len if max_q_len is not None else total_q), _ptr(ws), ws.numel() * ws.element_size()),
            "fa_decode_graph_create")
        self._h = h

    @property
    def kernel_count(self) -> int:
        return int(_lib.fa_decode_graph_kernel_count(self._h))

    def replay(self, stream=None):
        _check(_lib.fa_decode_graph_launch(self._h, _stream(stream)), "fa_decode_graph_launch")

    def close(self):
        if getattr(self, "_h", None):
            _lib.fa_decode_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fa_cache_append_fp8(k, v, k_cache, v_cache, slot_mapping, k_scale: float, v_scale: float, stream=None):
    """E4M3 codes of k/v [N, Hkv, d] (bf16 or fp32) / scale into k_cache uint8 [nb, Hkv, 16, d] and
    v_cache uint8 [nb, Hkv, d, 16] at slot_mapping[N]."""
    if k.dtype not in (torch.bfloat16, torch.float32) or v.dtype != k.dtype:
        raise ValueError("k, v must both be bf16 or both fp32")
    _need(k, "k", k.dtype, 3)
    _need(v, "v", k.dtype, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    N, Hkv, d = k.shape
    dt = FA_F32 if k.dtype == torch.float32 else FA_BF16
    _check(_lib.fa_cache_append_fp8(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), N, Hkv, d,
                                    k_cache.shape[0], float(k_scale), float(v_scale), dt, _stream(stream)),
           "fa_cache_append_fp8")


def fa_paged_attn_fp8(q, k_cache, v_cache, k_scale: float, v_scale: float, block_table, ctx_lens, q_lens,
                      causal: bool = True, scale: float | None = None, out=None, max_q_len: int | None = None,
                      ws=None, stream=None):
    """Decode rows of q [total_q, Hq, d] against the 8-bit caches."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(ctx_lens, "ctx_lens", torch.int32, 1)
    _need(q_lens, "q_lens", torch.int32, 1)
    total_q, Hq, d = q.shape
    num_blocks, Hkv = k_cache.shape[0], k_cache.shape[1]
    num_seqs, mbps = block_table.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    max_q_len = total_q if max_q_len is None else max_q_len
    nbytes = fa_paged_attn_workspace_size(num_seqs, mbps, Hq, Hkv, d, total_q)
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(_lib.fa_paged_attn_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale),
                                  _ptr(block_table), _ptr(ctx_lens), _ptr(q_lens), _ptr(out), num_seqs, mbps,
                                  num_blocks, Hq, Hkv, d, 16, int(causal), float(scale), total_q, int(max_q_len),
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "fa_paged_attn_fp8")
    return out


def fa_paged_attn_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q) -> int:
    return int(_lib.fa_paged_attn_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q))


def fa_paged_attn(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal: bool = True,
                  scale: float | None = None, out=None, max_q_len: int | None = None, ws=None, stream=None):
    """Attention of packed queries q [total_q, Hq, d] against the paged cache."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(ctx_lens, "ctx_lens", torch.int32, 1)
    _need(q_lens, "q_lens", torch.int32, 1)
    total_q, Hq, d = q.shape
    num_blocks, Hkv, bs, _ = k_cache.shape
    num_seqs, mbps = block_table.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if max_q_len is None:
        max_q_len = total_q
    nbytes = fa_paged_attn_workspace_size(num_seqs, mbps, Hq, Hkv, d, total_q)
    if ws is None:
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(_lib.fa_paged_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
                              _ptr(q_lens), _ptr(out), num_seqs, mbps, num_blocks, Hq, Hkv, d, bs, int(causal),
                              float(scale), total_q, int(max_q_len), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "fa_paged_attn")
    return out


def fa_paged_attn_mod_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len) -> int:
    return int(_lib.fa_paged_attn_mod_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len))


def fa_paged_attn_accum_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len) -> int:
    return int(_lib.fa_paged_attn_accum_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len))


def _paged_mod_args(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal, scale, softcap, alibi_slopes, window,
                    prefix_lens, out, lse, max_q_len):
    """Checks shared by the paged calls with modified scores: (device, the arguments up to lse, those from num_seqs to
    max_q_len, the workspace queries' sizes)."""
    total_q, Hq, d = _dims(q, "q", 3)
    nb, Hkv, bs, _ = _dims(k_cache, "k_cache", 4)
    S, mbps = _dims(block_table, "block_table", 2)
    dev, bf16, i32 = _device_of(q, "q"), torch.bfloat16, torch.int32
    max_q_len = total_q if max_q_len is None else _int(max_q_len, "max_q_len")
    window = _int(window, "window")
    head = (_arg(q, "q", bf16, (total_q, Hq, d), dev), _arg(k_cache, "k_cache", bf16, (nb, Hkv, bs, d), dev),
            _arg(v_cache, "v_cache", bf16, (nb, Hkv, bs, d), dev), _arg(block_table, "block_table", i32, (S, mbps), dev),
            _arg(ctx_lens, "ctx_lens", i32, (S,), dev), _arg(q_lens, "q_lens", i32, (S,), dev),
            _arg(out, "out", bf16, (total_q, Hq, d), dev), _opt(lse, "lse", torch.float32, (total_q, Hq), dev))
    tail = (S, mbps, nb, Hq, Hkv, d, bs, 1 if causal else 0, d ** -0.5 if scale is None else float(scale), float(softcap),
            _opt(alibi_slopes, "alibi_slopes", torch.float32, (Hq,), dev), window,
            _opt(prefix_lens, "prefix_lens", i32, (S,), dev), total_q, max_q_len)
    return dev, head, tail, (S, mbps, Hq, Hkv, d, total_q, max_q_len)


def fa_paged_attn_mod(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal: bool = True,
                      scale: float | None = None, softcap: float = 0.0, alibi_slopes=None, window: int = 0,
                      prefix_lens=None, out=None, lse=None, max_q_len: int | None = None, ws=None, stream=None):
    """fa_paged_attn with modified scores (as fa_prefill_mod, in cache positions); lse (optional, fp32
    [total_q, Hq]) receives the log-sum-exp of every row."""
    if out is None:
        out = _empty(q.shape, torch.bfloat16, _device_of(q, "q"), stream)
    dev, head, tail, sizes = _paged_mod_args(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal, scale, softcap,
                                             alibi_slopes, window, prefix_lens, out, lse, max_q_len)
    wp, wn, ws = _workspace(ws, 0 if ws is not None else fa_paged_attn_mod_workspace_size(*sizes), dev, stream)
    _check(_lib.fa_paged_attn_mod(*head, *tail, wp, wn, _current_stream(stream, dev)), "fa_paged_attn_mod")
    return out


def fa_paged_attn_accum(q, k_cache, v_cache, block_table, ctx_lens, q_lens, acc_in, acc_out, decay: float = 1.0,
                        causal: bool = True, scale: float | None = None, softcap: float = 0.0, alibi_slopes=None,
                        window: int = 0, prefix_lens=None, out=None, lse=None, max_q_len: int | None = None, ws=None,
                        stream=None):
    """fa_paged_attn_mod that also writes acc_out [num_seqs, Hkv, acc_len] = decay * acc_in (0 for the chunk's own
    tokens, and where acc_in is None) + the softmax weights every cached token received from the chunk's queries and
    the group's heads.  acc_in and acc_out may be the same tensor."""
    if out is None:
        out = _empty(q.shape, torch.bfloat16, _device_of(q, "q"), stream)
    if lse is None:
        lse = _empty(q.shape[:2], torch.float32, _device_of(q, "q"), stream)
    dev, head, tail, sizes = _paged_mod_args(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal, scale, softcap,
                                             alibi_slopes, window, prefix_lens, out, lse, max_q_len)
    rows = (sizes[0], sizes[3], _dims(acc_out, "acc_out", 3)[2])
    wp, wn, ws = _workspace(ws, 0 if ws is not None else fa_paged_attn_accum_workspace_size(*sizes), dev, stream)
    _check(_lib.fa_paged_attn_accum(*head, _opt(acc_in, "acc_in", torch.float32, rows, dev),
                                    _arg(acc_out, "acc_out", torch.float32, rows, dev), rows[2], float(decay), *tail, wp, wn,
                                    _current_stream(stream, dev)), "fa_paged_attn_accum")
    return out


def fa_cache_evict_workspace_size(num_seqs, max_blocks_per_seq, Hkv, keep) -> int:
    return int(_lib.fa_cache_evict_workspace_size(num_seqs, max_blocks_per_seq, Hkv, keep))


def fa_cache_evict(k_cache, v_cache, acc, block_table, ctx_lens, dst_table, keep: int, recent: int = 0, sink: int = 0,
                   acc_out=None, new_lens=None, kept=None, ws=None, stream=None):
    """Copies, per sequence and kv head, the first `sink`, the last `recent` and the tokens of largest acc
    [num_seqs, Hkv, acc_len] (`keep` in all) from the blocks of block_table to those of dst_table, in order of
    position; returns the new lengths int32 [num_seqs].  acc_out and kept (int32 [num_seqs, Hkv, keep], old
    positions) are optional outputs."""
    nb, Hkv, bs, d = _dims(k_cache, "k_cache", 4)
    S, mbps = _dims(block_table, "block_table", 2)
    acc_len, dmbps = _dims(acc, "acc", 3)[2], _dims(dst_table, "dst_table", 2)[1]
    dev, bf16, f32, i32 = _device_of(k_cache, "k_cache"), torch.bfloat16, torch.float32, torch.int32
    if new_lens is None:
        new_lens = _empty(S, i32, dev, stream)
    keep, recent, sink = _int(keep, "keep"), _int(recent, "recent"), _int(sink, "sink")
    out_len = 0 if acc_out is None else _dims(acc_out, "acc_out", 3)[2]
    need = fa_cache_evict_workspace_size(S, mbps, Hkv, keep) if kept is None and ws is None else 0
    wp, wn, ws = _workspace(ws, need, dev, stream)
    _check(_lib.fa_cache_evict(
        _arg(k_cache, "k_cache", bf16, (nb, Hkv, bs, d), dev), _arg(v_cache, "v_cache", bf16, (nb, Hkv, bs, d), dev),
        _arg(acc, "acc", f32, (S, Hkv, acc_len), dev), acc_len, _arg(block_table, "block_table", i32, (S, mbps), dev),
        _arg(ctx_lens, "ctx_lens", i32, (S,), dev), _arg(dst_table, "dst_table", i32, (S, dmbps), dev),
        _opt(acc_out, "acc_out", f32, (S, Hkv, out_len), dev), out_len, _arg(new_lens, "new_lens", i32, (S,), dev),
        _opt(kept, "kept", i32, (S, Hkv, keep), dev), S, mbps, dmbps, nb, Hkv, d, bs, keep, recent, sink, wp, wn,
        _current_stream(stream, dev)), "fa_cache_evict")
    return new_lens


def _cache_shapes(k_cache, v_cache, k_exp, v_exp, dev: int):
    """Checks a cache, bf16 or (k_exp, v_exp given) in 8 bits with block scales: (num_blocks, Hkv, block_size, d, the four
    addresses)."""
    nb, Hkv, bs, d = _dims(k_cache, "k_cache", 4)
    if (k_exp is None) != (v_exp is None):
        raise ValueError("k_exp and v_exp go together")
    if k_exp is None:
        ptrs = (_tensor(k_cache, "k_cache", torch.bfloat16, dev),
                _arg(v_cache, "v_cache", torch.bfloat16, (nb, Hkv, bs, d), dev), None, None)
    else:
        u8 = torch.uint8
        ptrs = (_tensor(k_cache, "k_cache", u8, dev), _arg(v_cache, "v_cache", u8, (nb, Hkv, d, bs), dev),
                _arg(k_exp, "k_exp", u8, (nb, Hkv), dev), _arg(v_exp, "v_exp", u8, (nb, Hkv), dev))
    return nb, Hkv, bs, d, ptrs


def _batch(block_table, ctx_lens, q_lens, dev: int):
    """Checks a batch's tables: (num_seqs, max_blocks_per_seq, the three addresses)."""
    S, mbps = _dims(block_table, "block_table", 2)
    i32 = torch.int32
    return S, mbps, (_tensor(block_table, "block_table", i32, dev), _arg(ctx_lens, "ctx_lens", i32, (S,), dev),
                     _arg(q_lens, "q_lens", i32, (S,), dev))


def fa_cache_append_fp8_scaled(k, v, k_cache, v_cache, k_exp, v_exp, block_table, ctx_lens, q_lens, q=None, positions=None,
                               cos_sin=None, q_out=None, stream=None):
    """Writes the last q_lens[s] tokens of every sequence (k, v packed [total_q, Hkv, d], bf16 or fp32; ctx_lens count
    them) to the 8-bit cache, k_cache uint8 [nb, Hkv, 16, d] and v_cache uint8 [nb, Hkv, d, 16], with a power-of-two scale
    for each block and head, k_exp and v_exp uint8 [nb, Hkv].  With cos_sin (fp32 [max_pos, d]) the keys are turned by the
    rows of `positions` (int32 [total_q]; None: the cache positions), and so are the queries q [total_q, Hq, d], which
    are returned (bf16)."""
    N, Hkv, d = _dims(k, "k", 3)
    dev, dt, bf16 = _device_of(k, "k"), k.dtype, torch.bfloat16
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError("q, k, v must all be bf16 or all fp32")
    if k_exp is None or v_exp is None:
        raise ValueError("k_exp and v_exp are needed")
    nb, Hkv_c, bs, d_c, cache = _cache_shapes(k_cache, v_cache, k_exp, v_exp, dev)
    if (Hkv_c, d_c) != (Hkv, d):
        raise ValueError(f"k_cache must have {Hkv} heads of {d} channels")
    S, mbps, tables = _batch(block_table, ctx_lens, q_lens, dev)
    Hq, max_pos = 0, 0
    if cos_sin is not None:
        max_pos = _dims(cos_sin, "cos_sin", 2)[0]
    elif q is not None or positions is not None:
        raise ValueError("q and positions need cos_sin")
    if q is not None:
        Hq = _dims(q, "q", 3)[1]
        if q_out is None:
            q_out = _empty((N, Hq, d), bf16, dev, stream)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _check(_lib.fa_cache_append_fp8_scaled(
        _opt(q, "q", dt, (N, Hq, d), dev), _tensor(k, "k", dt, dev), _arg(v, "v", dt, (N, Hkv, d), dev),
        _opt(positions, "positions", torch.int32, (N,), dev), _opt(cos_sin, "cos_sin", torch.float32, (max_pos, d), dev),
        max_pos, _opt(q_out, "q_out", bf16, (N, Hq, d), dev), *cache, *tables, S, mbps, nb, N, Hq, Hkv, d, bs,
        FA_F32 if dt is torch.float32 else FA_BF16, _current_stream(stream, dev)), "fa_cache_append_fp8_scaled")
    return q_out


def fa_paged_attn_fp8_scaled_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len) -> int:
    return int(_lib.fa_paged_attn_fp8_scaled_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len))


def fa_paged_attn_fp8_scaled(q, k_cache, v_cache, k_exp, v_exp, block_table, ctx_lens, q_lens, causal: bool = True,
                             scale: float | None = None, out=None, lse=None, max_q_len: int | None = None, ws=None,
                             stream=None):
    """fa_paged_attn over the 8-bit cache with block scales, single tokens and chunks; lse (optional, fp32 [total_q, Hq])
    receives the log-sum-exp of every row."""
    total_q, Hq, d = _dims(q, "q", 3)
    dev, bf16 = _device_of(q, "q"), torch.bfloat16
    if k_exp is None or v_exp is None:
        raise ValueError("k_exp and v_exp are needed")
    nb, Hkv, bs, d_c, cache = _cache_shapes(k_cache, v_cache, k_exp, v_exp, dev)
    if d_c != d:
        raise ValueError(f"k_cache must have heads of {d} channels")
    S, mbps, tables = _batch(block_table, ctx_lens, q_lens, dev)
    if out is None:
        out = _empty(q.shape, bf16, dev, stream)
    max_q_len = total_q if max_q_len is None else _int(max_q_len, "max_q_len")
    need = 0 if ws is not None else fa_paged_attn_fp8_scaled_workspace_size(S, mbps, Hq, Hkv, d, total_q, max_q_len)
    wp, wn, ws = _workspace(ws, need, dev, stream)
    _check(_lib.fa_paged_attn_fp8_scaled(
        _tensor(q, "q", bf16, dev), *cache, *tables, _arg(out, "out", bf16, (total_q, Hq, d), dev),
        _opt(lse, "lse", torch.float32, (total_q, Hq), dev), S, mbps, nb, Hq, Hkv, d, bs, 1 if causal else 0,
        d ** -0.5 if scale is None else float(scale), total_q, max_q_len, wp, wn, _current_stream(stream, dev)),
        "fa_paged_attn_fp8_scaled")
    return out


def fa_block_bounds(k_cache, block_table, ctx_lens, q_lens, bounds, *, total_q: int, k_exp=None, stream=None):
    """Writes the smallest and the largest value of every channel over a block's keys to bounds (bf16 [nb, Hkv, 2, d]),
    for the blocks that the last q_lens[s] tokens of each sequence lie in; total_q is the sum of q_lens.  k_cache is bf16
    [nb, Hkv, 16, d], or with k_exp the 8-bit cache."""
    nb, Hkv, bs, d = _dims(k_cache, "k_cache", 4)
    dev, bf16 = _device_of(k_cache, "k_cache"), torch.bfloat16
    S, mbps, tables = _batch(block_table, ctx_lens, q_lens, dev)
    _check(_lib.fa_block_bounds(
        _tensor(k_cache, "k_cache", bf16 if k_exp is None else torch.uint8, dev),
        _opt(k_exp, "k_exp", torch.uint8, (nb, Hkv), dev), *tables, _arg(bounds, "bounds", bf16, (nb, Hkv, 2, d), dev), S,
        mbps, nb, _int(total_q, "total_q"), Hkv, d, bs, _current_stream(stream, dev)), "fa_block_bounds")
    return bounds


def fa_block_select_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q) -> int:
    return int(_lib.fa_block_select_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q))


def fa_block_select(q, bounds, block_table, ctx_lens, q_lens, keep: int, recent: int = 1, sink: int = 0, sel=None,
                    max_q_len: int | None = None, ws=None, stream=None):
    """For each query of q [total_q, Hq, d] and kv head the numbers of `keep` blocks of its sequence, ascending (-1 behind
    the last): the first `sink`, the last `recent`, and those whose bounds (bf16 [nb, Hkv, 2, d]) allow the largest
    scores.  Returns sel int32 [total_q, Hkv, keep]."""
    total_q, Hq, d = _dims(q, "q", 3)
    nb, Hkv = _dims(bounds, "bounds", 4)[:2]
    dev, bf16 = _device_of(q, "q"), torch.bfloat16
    S, mbps, tables = _batch(block_table, ctx_lens, q_lens, dev)
    keep, recent, sink = _int(keep, "keep"), _int(recent, "recent"), _int(sink, "sink")
    max_q_len = total_q if max_q_len is None else _int(max_q_len, "max_q_len")
    if sel is None:
        sel = _empty((total_q, Hkv, max(keep, 0)), torch.int32, dev, stream)
    need = 0 if ws is not None else fa_block_select_workspace_size(S, mbps, Hq, Hkv, d, total_q)
    wp, wn, ws = _workspace(ws, need, dev, stream)
    _check(_lib.fa_block_select(
        _tensor(q, "q", bf16, dev), _arg(bounds, "bounds", bf16, (nb, Hkv, 2, d), dev), *tables,
        _arg(sel, "sel", torch.int32, (total_q, Hkv, max(keep, 0)), dev), S, mbps, nb, Hq, Hkv, d, 16, keep, recent, sink,
        total_q, max_q_len, wp, wn, _current_stream(stream, dev)), "fa_block_select")
    return sel


def fa_paged_attn_blocks(q, k_cache, v_cache, block_table, ctx_lens, q_lens, sel, k_exp=None, v_exp=None,
                         scale: float | None = None, out=None, lse=None, stream=None):
    """Attention of each query of q [total_q, Hq, d] over the blocks of its sequence listed in sel (int32 [total_q, Hkv,
    keep], negative entries passed over), up to its own position.  The cache is bf16, or with k_exp and v_exp the 8-bit
    cache with block scales; lse (optional, fp32 [total_q, Hq]) receives the log-sum-exp of every row."""
    total_q, Hq, d = _dims(q, "q", 3)
    dev, bf16 = _device_of(q, "q"), torch.bfloat16
    nb, Hkv, bs, d_c, cache = _cache_shapes(k_cache, v_cache, k_exp, v_exp, dev)
    if d_c != d:
        raise ValueError(f"k_cache must have heads of {d} channels")
    S, mbps, tables = _batch(block_table, ctx_lens, q_lens, dev)
    keep = _dims(sel, "sel", 3)[2]
    if out is None:
        out = _empty(q.shape, bf16, dev, stream)
    _check(_lib.fa_paged_attn_blocks(
        _tensor(q, "q", bf16, dev), *cache, *tables, _arg(sel, "sel", torch.int32, (total_q, Hkv, keep), dev),
        keep, _arg(out, "out", bf16, (total_q, Hq, d), dev), _opt(lse, "lse", torch.float32, (total_q, Hq), dev), S, mbps, nb,
        Hq, Hkv, d, bs, d ** -0.5 if scale is None else float(scale), total_q, _current_stream(stream, dev)),
        "fa_paged_attn_blocks")
    return out


def fa_paged_attn_noalloc(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal: bool = True,
                          scale: float | None = None, out=None, max_q_len: int | None = None, stream=None):
    """fa_paged_attn without a workspace, for callers that cannot allocate device
    scratch: the library's fixed 32 MiB per-device array is used instead.  Calls
    must not overlap on the GPU (they share that array)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(ctx_lens, "ctx_lens", torch.int32, 1)
    _need(q_lens, "q_lens", torch.int32, 1)
    total_q, Hq, d = q.shape
    num_blocks, Hkv, bs, _ = k_cache.shape
    num_seqs, mbps = block_table.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if max_q_len is None:
        max_q_len = total_q
    _check(_lib.fa_paged_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
                                      _ptr(q_lens), _ptr(out), num_seqs, mbps, num_blocks, Hq, Hkv, d, bs,
                                      int(causal), float(scale), total_q, int(max_q_len), _stream(stream)),
           "fa_paged_attn_noalloc")
    return out


# --------------------------------------------------------------- utilities
def fa_get_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status."""
    return int(_lib.fa_get_error(_stream(stream)))


def fa_debug_gather_kv(cache, block_table, ctx_lens, max_ctx: int, out=None, stream=None):
    _need(cache, "cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(ctx_lens, "ctx_lens", torch.int32, 1)
    num_blocks, Hkv, _, d = cache.shape
    num_seqs, mbps = block_table.shape
    if out is None:
        out = torch.zeros(num_seqs, max_ctx, Hkv, d, dtype=torch.bfloat16, device=cache.device)
    _check(_lib.fa_debug_gather_kv(_ptr(cache), _ptr(block_table), _ptr(ctx_lens), _ptr(out), num_seqs, mbps,
                                   num_blocks, Hkv, d, max_ctx, _stream(stream)), "fa_debug_gather_kv")
    return out


def fa_debug_set_wait_limit(nanoseconds: int):
    _lib.fa_debug_set_wait_limit(int(nanoseconds))


def fa_debug_force_timeout(enable):
    _lib.fa_debug_force_timeout(enable if isinstance(enable, int) else int(bool(enable)))


def fa_last_launch_count() -> int:
    return int(_lib.fa_last_launch_count())
