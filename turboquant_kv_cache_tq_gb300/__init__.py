"""GB300 TurboQuant KV-cache codec: Python binding of the C ABI in include/tq.h.

This module only marshals torch tensors (device pointers, sizes and the
current CUDA stream) into ``libtq.so``; every step of encode and decode runs
in the library's CUDA kernels. There is no fallback: if the library is not
built, importing works but every call raises.

Names follow the C ABI: ``tq_packed_dim``, ``tq_encode_kv``, ``tq_decode_kv``,
``tq_lloyd_max_index``, ``tq_status_string``; ``alloc_cache`` allocates the
five packed-cache buffers with torch.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

__all__ = [
    "TQError", "lib", "tq_packed_dim", "tq_encode_kv", "tq_decode_kv", "tq_decode_kv_rotated",
    "tq_unrotate", "tq_lloyd_max_index", "tq_decode_attention", "tq_decode_attention_workspace_size",
    "tq_cache_assemble", "merge_rows", "extend_rows", "extract_row", "filter_rows", "tq_lloyd_max_fit",
    "tq_lloyd_max_fit_status", "tq_tree_attention", "tq_tree_attention_workspace_size", "tq_attention_weights",
    "tq_evict_select", "tq_cache_gather", "commit_path", "evict_rows",
    "tq_status_string", "alloc_cache", "HEAD_DIMS", "VALUE_BITS", "KEY_MODES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq.so")
HEAD_DIMS = (64, 128, 256, 512)
VALUE_BITS = (2, 3, 4, 5, 8)
KEY_MODES = ((2, False), (4, False), (5, False), (8, False), (8, True))
GROUP = 32
TQ_F32, TQ_BF16 = 0, 1
_DTYPE = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16}
_NAMES = ("TQ_OK", "TQ_ERR_INVALID_ARG", "TQ_ERR_HEAD_DIM", "TQ_ERR_BITS", "TQ_ERR_ALIGNMENT",
          "TQ_ERR_DTYPE", "TQ_ERR_CUDA", "TQ_ERR_TIMEOUT", "TQ_ERR_DEVICE_CHECK")

_lock = threading.Lock()
_lib = None


class TQError(RuntimeError):
    """A non-OK tq_status from the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        name = _NAMES[status] if 0 <= status < len(_NAMES) else str(status)
        super().__init__("%s: %s (%s)" % (what, name, tq_status_string(status)))


def lib() -> ctypes.CDLL:
    """The loaded libtq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libtq.so is not built (%s); run python -m turboquant_kv_cache_tq_gb300.build" % LIB_PATH)
            _lib = load_library(LIB_PATH)
    return _lib


def load_library(path: str) -> ctypes.CDLL:
    """A build of the C ABI at `path` (libtq.so or its debug variant
    libtq_debug.so) with every entry point's argument types declared."""
    L = ctypes.CDLL(path)
    P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.tq_packed_dim.restype = I64
    L.tq_packed_dim.argtypes = [I64, I]
    L.tq_encode_kv.restype = I
    L.tq_encode_kv.argtypes = [P, P, I, I64, I64, I64, I64, I, I, I, P, P, P, P, P, I64, I64, P]
    L.tq_decode_kv.restype = I
    L.tq_decode_kv.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, I, I, I, P, P, I, P]
    L.tq_decode_kv_rotated.restype = I
    L.tq_decode_kv_rotated.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I64, I, I, I, P, P, I, P]
    L.tq_unrotate.restype = I
    L.tq_unrotate.argtypes = [P, I, I64, I64, P, P]
    L.tq_lloyd_max_index.restype = I
    L.tq_lloyd_max_index.argtypes = [P, I64, I, P, P]
    L.tq_decode_attention.restype = I
    L.tq_decode_attention.argtypes = [P, I64, I64, I64, P, P, P, P, P, I64, I64, I64, I64, I, I, I, P,
                                      ctypes.c_float, P, I, P, I64, P]
    L.tq_decode_attention_noalloc.restype = I
    L.tq_decode_attention_noalloc.argtypes = [P, I64, I64, I64, P, P, P, P, P, I64, I64, I64, I64, I, I,
                                              I, P, ctypes.c_float, P, I, P]
    L.tq_decode_attention_workspace_size.restype = I64
    L.tq_decode_attention_workspace_size.argtypes = [I64, I64, I64, I64]
    L.tq_cache_assemble.restype = I
    L.tq_cache_assemble.argtypes = [P, I64, I64, I64, I, I, P, P, P, P, P, I64, I64, P]
    L.tq_tree_attention.restype = I
    L.tq_tree_attention.argtypes = [P, I64, I64, I64, P, I64, I64, I64, P, P, I, I, I, P, P, ctypes.c_float, P, I,
                                    P, P, I64, P]
    L.tq_tree_attention_workspace_size.restype = I64
    L.tq_tree_attention_workspace_size.argtypes = [I64, I64, I64, I64, I64]
    L.tq_attention_weights.restype = I
    L.tq_attention_weights.argtypes = [P, P, I64, I64, I64, P, P, P, I64, I64, I64, I64, I, I, P, P, P, P, I64,
                                       ctypes.c_float, P, P, I64, P]
    L.tq_evict_select.restype = I
    L.tq_evict_select.argtypes = [P, I64, I64, I64, I64, P, P, I64, I64, P, P, P]
    L.tq_cache_gather.restype = I
    L.tq_cache_gather.argtypes = [P, P, I64, I64, I64, I, I, P, I64, I, P, P, P, P, P, P]
    L.tq_lloyd_max_fit.restype = I
    L.tq_lloyd_max_fit.argtypes = [P, I64, I, I, P, P, P, P, I64, P]
    L.tq_lloyd_max_fit_bounded.restype = I
    L.tq_lloyd_max_fit_bounded.argtypes = [P, I64, I, I, P, P, P, P, I64, I64, I, P]
    L.tq_lloyd_max_fit_status.restype = I
    L.tq_lloyd_max_fit_status.argtypes = [P, P]
    L.tq_lloyd_max_fit_workspace_size.restype = I64
    L.tq_lloyd_max_fit_workspace_size.argtypes = [I]
    L.tq_device_status.restype = I
    L.tq_device_status.argtypes = [P]
    L.tq_debug_checks.restype = I
    L.tq_debug_checks.argtypes = []
    L.tq_status_string.restype = ctypes.c_char_p
    L.tq_status_string.argtypes = [I]
    return L


def tq_status_string(status: int) -> str:
    return lib().tq_status_string(int(status)).decode()


def _stream_handle(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status != 0:
        raise TQError(status, what)


def tq_packed_dim(dim: int, bits: int) -> int:
    """Bytes of one packed row of `dim` codes at `bits` bits (raises if not byte-aligned)."""
    r = int(lib().tq_packed_dim(int(dim), int(bits)))
    if r < 0:
        raise TQError(-r, "tq_packed_dim(%d, %d)" % (dim, bits))
    return r


def alloc_cache(B: int, H: int, t_cap: int, D: int, k_bits: int, v_bits: int, device="cuda") -> dict:
    """The five packed-cache buffers [B,H,t_cap,X] (codes uint8, scales/zeros fp16)."""
    G = D // GROUP
    return dict(
        k_codes=torch.zeros((B, H, t_cap, tq_packed_dim(D, k_bits)), dtype=torch.uint8, device=device),
        k_scales=torch.zeros((B, H, t_cap, G), dtype=torch.float16, device=device),
        k_zeros=torch.zeros((B, H, t_cap, G), dtype=torch.float16, device=device),
        v_codes=torch.zeros((B, H, t_cap, tq_packed_dim(D, v_bits)), dtype=torch.uint8, device=device),
        v_scales=torch.zeros((B, H, t_cap, G), dtype=torch.float16, device=device),
    )


def _cache_ptrs(cache: dict):
    for name in ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales"):
        t = cache[name]
        if not t.is_contiguous():
            raise ValueError("cache buffer %s must be contiguous" % name)
    return [cache[n].data_ptr() for n in ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales")]


def tq_encode_kv(k: torch.Tensor, v: torch.Tensor, k_bits: int, k_signed: bool, v_bits: int,
                 cache: dict, t_off: int = 0, stream=None) -> dict:
    """Encode K, V [B,H,T,D] (fp32 or bf16, contiguous, on the GPU) into tokens
    [t_off, t_off+T) of `cache` (capacity = its token axis). Asynchronous on
    `stream` (default: the current stream)."""
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
        raise ValueError("K and V must be [B,H,T,D] tensors of one shape and dtype")
    if k.dtype not in _DTYPE:
        raise ValueError("K/V dtype must be float32 or bfloat16, got %s" % k.dtype)
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("K and V must be contiguous")
    B, H, T, D = k.shape
    t_cap = cache["k_codes"].shape[2]
    st = lib().tq_encode_kv(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], B, H, T, D, int(k_bits),
                            int(bool(k_signed)), int(v_bits), *_cache_ptrs(cache), t_cap, int(t_off),
                            _stream_handle(stream, k.device))
    _check(st, "tq_encode_kv")
    return cache


def _decode(fn, name, cache, T, k_bits, k_signed, v_bits, out_dtype, k_out, v_out, stream):
    B, H, t_cap, _ = cache["k_codes"].shape
    D = cache["k_scales"].shape[-1] * GROUP
    dev = cache["k_codes"].device
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if k_out is None:
        k_out = torch.empty((B, H, T, D), dtype=out_dtype, device=dev)
    if v_out is None:
        v_out = torch.empty((B, H, T, D), dtype=out_dtype, device=dev)
    for t in (k_out, v_out):
        if t.dtype != out_dtype or tuple(t.shape) != (B, H, T, D) or not t.is_contiguous():
            raise ValueError("k_out/v_out must be contiguous [B,H,T,D] tensors of out_dtype")
    st = fn(*_cache_ptrs(cache), B, H, T, D, t_cap, int(k_bits), int(bool(k_signed)), int(v_bits),
            k_out.data_ptr(), v_out.data_ptr(), _DTYPE[out_dtype], _stream_handle(stream, dev))
    _check(st, name)
    return k_out, v_out


def tq_decode_kv(cache: dict, T: int, k_bits: int, k_signed: bool, v_bits: int,
                 out_dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """Decode tokens [0,T) of `cache` into K, V [B,H,T,D] of `out_dtype`
    (allocated when not given). Asynchronous on `stream`."""
    return _decode(lib().tq_decode_kv, "tq_decode_kv", cache, T, k_bits, k_signed, v_bits, out_dtype,
                   k_out, v_out, stream)


def tq_decode_kv_rotated(cache: dict, T: int, k_bits: int, k_signed: bool, v_bits: int,
                         out_dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """As tq_decode_kv, but V stays in the rotated domain (centroid * scale,
    no inverse transform); undo it on an attention output with tq_unrotate."""
    return _decode(lib().tq_decode_kv_rotated, "tq_decode_kv_rotated", cache, T, k_bits, k_signed, v_bits,
                   out_dtype, k_out, v_out, stream)


def tq_unrotate(x: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """Inverse value rotation of the rows of `x` ([..., D], fp32 or bf16,
    contiguous), computed in fp32 and returned in x's dtype. `out` must not
    overlap x."""
    if x.dtype not in _DTYPE or not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous float32 or bfloat16 tensor")
    D = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of x's shape and dtype")
    n = x.numel() // D if D else 0
    st = lib().tq_unrotate(x.data_ptr(), _DTYPE[x.dtype], n, D, out.data_ptr(), _stream_handle(stream, x.device))
    _check(st, "tq_unrotate")
    return out


def tq_lloyd_max_index(u: torch.Tensor, v_bits: int, out=None, stream=None) -> torch.Tensor:
    """count(boundaries < u) for each fp32 element of `u` (uint8 result)."""
    if u.dtype != torch.float32 or not u.is_contiguous():
        raise ValueError("u must be a contiguous float32 tensor")
    if out is None:
        out = torch.empty(u.shape, dtype=torch.uint8, device=u.device)
    st = lib().tq_lloyd_max_index(u.data_ptr(), u.numel(), int(v_bits), out.data_ptr(),
                                  _stream_handle(stream, u.device))
    _check(st, "tq_lloyd_max_index")
    return out


def tq_decode_attention_workspace_size(B: int, Hkv: int, T: int, D: int) -> int:
    """Bytes of scratch tq_decode_attention needs (on the current device)."""
    r = int(lib().tq_decode_attention_workspace_size(int(B), int(Hkv), int(T), int(D)))
    if r < 0:
        raise TQError(-r, "tq_decode_attention_workspace_size")
    return r


def tq_decode_attention(q: torch.Tensor, cache: dict, T: int, k_bits: int, k_signed: bool, v_bits: int,
                        left_pad=None, scale=None, out_dtype=torch.bfloat16, out=None, workspace=None,
                        stream=None) -> torch.Tensor:
    """Attention of bf16 queries q [B,Hq,Nq,D] over tokens [0,T) of a packed
    cache [B,Hkv,t_cap,*] (t_cap a multiple of 16), output unrotated
    [B,Hq,Nq,D] of out_dtype. left_pad: int32 device tensor [B] or None.
    workspace: a uint8 device tensor of at least
    tq_decode_attention_workspace_size bytes (allocated when None)."""
    if q.dtype != torch.bfloat16 or q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B,Hq,Nq,D] bfloat16 tensor")
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    B, Hq, Nq, D = q.shape
    Bc, Hkv, t_cap, _ = cache["k_codes"].shape
    if Bc != B:
        raise ValueError("q and the cache must have the same batch size")
    dev = q.device
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, Nq, D), dtype=out_dtype, device=dev)
    if out.dtype != out_dtype or tuple(out.shape) != (B, Hq, Nq, D) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B,Hq,Nq,D] tensor of out_dtype")
    lp = 0
    if left_pad is not None:
        if left_pad.dtype != torch.int32 or tuple(left_pad.shape) != (B,) or not left_pad.is_contiguous():
            raise ValueError("left_pad must be a contiguous int32 tensor [B]")
        lp = left_pad.data_ptr()
    need = tq_decode_attention_workspace_size(B, Hkv, T, D)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = lib().tq_decode_attention(q.data_ptr(), B, Hq, Nq, *_cache_ptrs(cache), Hkv, int(T), D, t_cap,
                                   int(k_bits), int(bool(k_signed)), int(v_bits), lp or None, float(scale),
                                   out.data_ptr(), _DTYPE[out_dtype], workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(st, "tq_decode_attention")
    return out


# ---- batched packed-cache rows (batched-quant.ts) ---------------------------------
class TQRowSource(ctypes.Structure):
    """tq_row_source of include/tq.h."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("k_zeros", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("B", ctypes.c_int64),
                ("b", ctypes.c_int64), ("t_cap", ctypes.c_int64), ("t_start", ctypes.c_int64),
                ("len", ctypes.c_int64)]


def _cache_geometry(cache: dict):
    B, H, t_cap, xk = cache["k_codes"].shape
    D = cache["k_scales"].shape[-1] * GROUP
    return B, H, t_cap, D, xk * 8 // D, cache["v_codes"].shape[-1] * 8 // D


def tq_cache_assemble(sources, dst: dict, width: int, stream=None) -> dict:
    """Assemble destination batch row r from sources[r] = (cache, b, t_start,
    length) or None (an all-padding row): width - length zero tokens, then the
    source's tokens [t_start, t_start + length), for every head and buffer."""
    n, H, t_cap, D, kb, vb = _cache_geometry(dst)
    if len(sources) != n:
        raise ValueError("one source per destination batch row")
    arr = (TQRowSource * max(n, 1))()
    for r, src in enumerate(sources):
        if src is None:
            arr[r] = TQRowSource(None, None, None, None, None, 0, 0, 0, 0, 0)
            continue
        cache, b, t0, length = src
        Bs, Hs, tcs, Ds, kbs, vbs = _cache_geometry(cache)
        if (Hs, Ds, kbs, vbs) != (H, D, kb, vb):
            raise ValueError("source and destination caches differ in heads, head_dim or bit widths")
        arr[r] = TQRowSource(*_cache_ptrs(cache), Bs, int(b), tcs, int(t0), int(length))
    st = lib().tq_cache_assemble(ctypes.cast(arr, ctypes.c_void_p), n, H, D, kb, vb, *_cache_ptrs(dst), t_cap,
                                 int(width), _stream_handle(stream, dst["k_codes"].device))
    _check(st, "tq_cache_assemble")
    return dst


def _alloc_like(cache: dict, B: int, t_cap: int) -> dict:
    _, H, _, D, kb, vb = _cache_geometry(cache)
    return alloc_cache(B, H, t_cap, D, kb, vb, device=cache["k_codes"].device)


def merge_rows(rows, t_cap=None, stream=None):
    """mergeQuantRows: rows = [(cache, length)] single-row caches ([1,H,*,X],
    tokens [0, length) valid) -> (batch cache [N,H,t_cap,X], left pads, width)
    with every row right-justified in width = max length."""
    width = max(int(n) for _, n in rows)
    pads = [width - int(n) for _, n in rows]
    dst = _alloc_like(rows[0][0], len(rows), width if t_cap is None else t_cap)
    tq_cache_assemble([(c, 0, 0, n) for c, n in rows], dst, width, stream)
    return dst, pads, width


def extend_rows(batch, S: int, pads, row, t_cap=None, stream=None):
    """extendQuantRows: append row = (cache, length) to a batch whose window
    is S tokens wide; the narrower side is padded on the left."""
    rc, n = row
    width = max(int(S), int(n))
    B = batch["k_codes"].shape[0]
    dst = _alloc_like(batch, B + 1, width if t_cap is None else t_cap)
    srcs = [(batch, b, 0, S) for b in range(B)] + [(rc, 0, 0, n)]
    tq_cache_assemble(srcs, dst, width, stream)
    return dst, [p + (width - S) for p in pads] + [width - int(n)], width


def extract_row(batch, S: int, pad: int, i: int, stream=None) -> dict:
    """extractQuantRow: batch row i past its left pad as a fresh single-row
    cache [1, H, S - pad, X]."""
    dst = _alloc_like(batch, 1, int(S) - int(pad))
    tq_cache_assemble([(batch, i, pad, int(S) - int(pad))], dst, int(S) - int(pad), stream)
    return dst


def filter_rows(batch, S: int, keep, stream=None) -> dict:
    """filterQuantRows: the batch rows `keep`, in that order, same window."""
    dst = _alloc_like(batch, len(keep), batch["k_codes"].shape[2])
    tq_cache_assemble([(batch, int(b), 0, S) for b in keep], dst, S, stream)
    return dst


# ---- ragged packed caches: draft trees and eviction --------------------------------
class TQPackedCache(ctypes.Structure):
    """tq_packed_cache of include/tq.h."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("k_zeros", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("t_cap", ctypes.c_int64)]


_BUFFERS = ("k_codes", "k_scales", "k_zeros", "v_codes", "v_scales")


def _refuse_cache(cache, B, H, D, k_bits, v_bits, device, names):
    t_cap = cache["k_codes"].shape[2] if cache["k_codes"].dim() == 4 else -1
    for name in names:
        t = cache[name]
        x = D // GROUP if name[2:] in ("scales", "zeros") else D * (k_bits if name == "k_codes" else v_bits) // 8
        dtype = torch.uint8 if name[2:] == "codes" else torch.float16
        if t.dtype != dtype or tuple(t.shape) != (B, H, t_cap, x) or not t.is_contiguous() or t.device != device:
            raise ValueError("cache buffer %s must be a contiguous [%d,%d,t_cap,%d] %s tensor on %s"
                             % (name, B, H, x, dtype, device))
    raise ValueError("not a packed cache on %s" % device)


def _keys_ok(cache, B, H, D, k_bits, dev):
    """The key buffers, or None where they are not [B,H,t_cap,X] on GPU dev."""
    c, s, z = cache["k_codes"], cache["k_scales"], cache["k_zeros"]
    if c.dim() != 4:
        return None
    t_cap = c.shape[2]
    g = (B, H, t_cap, D // GROUP)
    if (c.shape == (B, H, t_cap, D * k_bits // 8) and s.shape == g and z.shape == g and c.dtype is torch.uint8
            and s.dtype is torch.float16 and z.dtype is torch.float16 and c.is_contiguous() and s.is_contiguous()
            and z.is_contiguous() and c.get_device() == dev and s.get_device() == dev and z.get_device() == dev):
        return c, s, z, t_cap
    return None


def _packed(cache: dict, B, H, D, k_bits, v_bits, device) -> TQPackedCache:
    """The checked buffers of a packed cache as the library takes them."""
    dev = device.index
    keys = _keys_ok(cache, B, H, D, k_bits, dev)
    if keys is not None:
        c, s, z, t_cap = keys
        v, w = cache["v_codes"], cache["v_scales"]
        if (v.shape == (B, H, t_cap, D * v_bits // 8) and w.shape == s.shape and v.dtype is torch.uint8
                and w.dtype is torch.float16 and v.is_contiguous() and w.is_contiguous() and v.get_device() == dev
                and w.get_device() == dev):
            return TQPackedCache(c.data_ptr(), s.data_ptr(), z.data_ptr(), v.data_ptr(), w.data_ptr(), t_cap)
    _refuse_cache(cache, B, H, D, k_bits, v_bits, device, _BUFFERS)


def _int_ptr(t, shape, what, device):
    """Device pointer of an optional int32 tensor of a given shape."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous int32 tensor %s on %s" % (what, list(shape), device))
    return t.data_ptr()


def _float_ptr(t, shape, what, device):
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous float32 tensor %s on %s" % (what, list(shape), device))
    return t.data_ptr()


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _elsewhere(device, stream) -> bool:
    """Whether a call has to switch to another device or stream than the current
    one: for its allocations (the allocator gives memory back in the current
    stream's order) and because the library asks the current device for its size
    and error word."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device, got %s" % device)
    if stream is not None and stream.device != device:
        raise ValueError("the stream is of %s, the tensors are on %s" % (stream.device, device))
    return stream is not None or device.index != torch.cuda.current_device()


def _current_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def tq_tree_attention_workspace_size(B: int, Hq: int, Hkv: int, N: int, D: int) -> int:
    """Bytes of scratch tq_tree_attention needs (on the current device)."""
    r = int(lib().tq_tree_attention_workspace_size(int(B), int(Hq), int(Hkv), int(N), int(D)))
    if r < 0:
        raise TQError(-r, "tq_tree_attention_workspace_size")
    return r


def tq_tree_attention(q: torch.Tensor, cache: dict, T: int, tree: dict, k_bits: int, k_signed: bool, v_bits: int,
                      parents=None, lens=None, left_pad=None, scale=None, out_dtype=torch.bfloat16, out=None,
                      lse=None, workspace=None, stream=None):
    """Attention of a tree of N drafted tokens, q [B,Hq,N,D] bf16, over tokens
    [left_pad[b], lens[b]) of a packed cache and over the nodes' own keys and
    values in the packed cache `tree` (tokens [0,N)): node i attends to itself
    and its ancestors by parents [B,N] (int32; -1: follows the sequence; other
    values outside [0,i): the node is absent; None: a chain). lens and left_pad:
    int32 device tensors [B] or None; lens <= T. Returns (out [B,Hq,N,D] of
    out_dtype, lse [B,Hq,N] fp32). workspace: a uint8 device tensor of at least
    tq_tree_attention_workspace_size bytes (allocated when None)."""
    if q.dtype != torch.bfloat16 or q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B,Hq,N,D] bfloat16 tensor")
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    dev = q.device
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return tq_tree_attention(q, cache, T, tree, k_bits, k_signed, v_bits, parents, lens, left_pad, scale,
                                     out_dtype, out, lse, workspace)
    B, Hq, N, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    cv = _packed(cache, B, Hkv, D, k_bits, v_bits, dev)
    tv = _packed(tree, B, Hkv, D, k_bits, v_bits, dev)
    if out is None:
        out = torch.empty((B, Hq, N, D), dtype=out_dtype, device=dev)
    elif out.dtype != out_dtype or out.shape != q.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous [B,Hq,N,D] tensor of out_dtype on q's device")
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=dev)
    if workspace is None:
        need = tq_tree_attention_workspace_size(B, Hq, Hkv, N, D)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    st = lib().tq_tree_attention(
        q.data_ptr(), B, Hq, N, ctypes.byref(cv), Hkv, int(T), D, ctypes.byref(tv),
        _int_ptr(parents, (B, N), "parents", dev), int(k_bits), int(bool(k_signed)), int(v_bits),
        _int_ptr(lens, (B,), "lens", dev), _int_ptr(left_pad, (B,), "left_pad", dev),
        D ** -0.5 if scale is None else float(scale), out.data_ptr(), _DTYPE[out_dtype],
        _float_ptr(lse, (B, Hq, N), "lse", dev), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _current_stream(dev))
    _check(st, "tq_tree_attention")
    return out, lse


def tq_attention_weights(q: torch.Tensor, lse: torch.Tensor, cache: dict, T: int, k_bits: int, k_signed: bool,
                         path=None, n_path=None, lens=None, left_pad=None, scale=None, weights=None, out=None,
                         stream=None) -> torch.Tensor:
    """weights + the attention weights that the last n_path[b] tokens of each
    sequence give to its tokens, [B,Hkv,w_cap] fp32 (w_cap >= T): observer i is
    query row path[b,i] of q [B,Hq,N,D] with log-sum-exp lse [B,Hq,N]
    (tq_tree_attention). path: int32 [B,P] or None (rows 0..N-1, P = N);
    n_path: int32 [B] or None (P). weights: None (zeros), or the sums so far;
    out: None (a new tensor), or where to write, `weights` itself for an update
    in place."""
    if q.dtype != torch.bfloat16 or q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B,Hq,N,D] bfloat16 tensor")
    dev = q.device
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return tq_attention_weights(q, lse, cache, T, k_bits, k_signed, path, n_path, lens, left_pad, scale,
                                        weights, out)
    B, Hq, N, D = q.shape
    Hkv = cache["k_codes"].shape[1]
    keys = _keys_ok(cache, B, Hkv, D, k_bits, dev.index)
    if keys is None:
        _refuse_cache(cache, B, Hkv, D, k_bits, 0, dev, _BUFFERS[:3])
    P = N if path is None else path.shape[-1]
    if out is None:
        w_cap = int(T) if weights is None else weights.shape[-1]
        out = torch.empty((B, Hkv, w_cap), dtype=torch.float32, device=dev)
    w_cap = out.shape[-1]
    st = lib().tq_attention_weights(
        q.data_ptr(), _float_ptr(lse, (B, Hq, N), "lse", dev), B, Hq, N, keys[0].data_ptr(), keys[1].data_ptr(),
        keys[2].data_ptr(), Hkv, int(T), D, keys[3], int(k_bits), int(bool(k_signed)),
        _int_ptr(lens, (B,), "lens", dev), _int_ptr(left_pad, (B,), "left_pad", dev),
        _int_ptr(path, (B, P), "path", dev), _int_ptr(n_path, (B,), "n_path", dev), P,
        D ** -0.5 if scale is None else float(scale), _float_ptr(weights, (B, Hkv, w_cap), "weights", dev),
        _float_ptr(out, (B, Hkv, w_cap), "out", dev), w_cap, _current_stream(dev))
    _check(st, "tq_attention_weights")
    return out


def tq_evict_select(weights: torch.Tensor, T: int, keep: int, recent: int, lens=None, left_pad=None, index=None,
                    count=None, stream=None):
    """The tokens that stay when each (batch row, head) is cut to `keep` tokens:
    the last `recent` ones and the largest weights [B,H,w_cap] among the others
    (equal weights: the lowest token). Returns (index int32 [B,H,keep],
    ascending, then -1; count int32 [B])."""
    if weights.dim() != 3:
        raise ValueError("weights must be a [B,H,w_cap] tensor")
    if keep < 0:
        raise ValueError("keep must not be negative")
    dev = weights.device
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return tq_evict_select(weights, T, keep, recent, lens, left_pad, index, count)
    B, H, w_cap = weights.shape
    keep = int(keep)
    if index is None:
        index = torch.empty((B, H, keep), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((B,), dtype=torch.int32, device=dev)
    st = lib().tq_evict_select(
        _float_ptr(weights, (B, H, w_cap), "weights", dev), B, H, int(T), w_cap, _int_ptr(lens, (B,), "lens", dev),
        _int_ptr(left_pad, (B,), "left_pad", dev), keep, int(recent), _int_ptr(index, (B, H, keep), "index", dev),
        _int_ptr(count, (B,), "count", dev), _current_stream(dev))
    _check(st, "tq_evict_select")
    return index, count


def tq_cache_gather(src: dict, dst: dict, index: torch.Tensor, count=None, dst_off=None, src_weights=None,
                    dst_weights=None, dst_len=None, stream=None):
    """Copies tokens index [B,n] or [B,H,n] (int32) of the packed cache src to
    tokens dst_off[b] + j, j < count[b], of dst (with their weights, or zero
    weights, when dst_weights is given). Returns (dst, dst_len), dst_len int32
    [B] = min(dst_off + count, capacity)."""
    dev = src["k_codes"].device
    if _elsewhere(dev, stream):
        with _switched(dev, stream):
            return tq_cache_gather(src, dst, index, count, dst_off, src_weights, dst_weights, dst_len)
    B, H, _, D, kb, vb = _cache_geometry(src)
    sv, dv = _packed(src, B, H, D, kb, vb, dev), _packed(dst, B, H, D, kb, vb, dev)
    heads = index.dim() == 3
    n = index.shape[-1]
    if dst_len is None:
        dst_len = torch.empty((B,), dtype=torch.int32, device=dev)
    st = lib().tq_cache_gather(
        ctypes.byref(sv), ctypes.byref(dv), B, H, D, kb, vb,
        _int_ptr(index, (B, H, n) if heads else (B, n), "index", dev), n, int(heads),
        _int_ptr(count, (B,), "count", dev), _int_ptr(dst_off, (B,), "dst_off", dev),
        _int_ptr(dst_len, (B,), "dst_len", dev), _float_ptr(src_weights, (B, H, sv.t_cap), "src_weights", dev),
        _float_ptr(dst_weights, (B, H, dv.t_cap), "dst_weights", dev), _current_stream(dev))
    _check(st, "tq_cache_gather")
    return dst, dst_len


def commit_path(cache: dict, lens: torch.Tensor, tree: dict, path: torch.Tensor, n_path: torch.Tensor, weights=None,
                stream=None) -> torch.Tensor:
    """Appends the accepted nodes path[b, :n_path[b]] of a draft tree's cache to
    each sequence of `cache` (weights, when given, start at zero). Returns the
    new lengths. A sequence takes no more tokens than its row has room for: the
    rest of its path is dropped, and the new length is the capacity. So what was
    appended is new - lens (lens within the capacity), not n_path: give
    tq_attention_weights that, or its observers sit at wrong tokens where a row was
    full."""
    return tq_cache_gather(tree, cache, path, count=n_path, dst_off=lens, dst_weights=weights, stream=stream)[1]


def evict_rows(cache: dict, weights: torch.Tensor, T: int, keep: int, recent: int, lens=None, left_pad=None,
               t_cap=None, stream=None):
    """Cuts every (batch row, head) to at most `keep` tokens by their attention
    weights -> (a fresh cache whose rows start at token 0, its weights, its
    lengths). t_cap: the fresh cache's capacity (keep when None), room for every
    token that may stay."""
    B, H, cap = cache["k_codes"].shape[:3]
    if weights.shape[-1] != cap:
        raise ValueError("weights must be [B,H,%d], the cache's capacity" % cap)
    if t_cap is not None and t_cap < min(keep, T):
        raise ValueError("t_cap must be at least %d, the tokens that may stay" % min(keep, T))
    if _elsewhere(weights.device, stream):
        with _switched(weights.device, stream):
            return evict_rows(cache, weights, T, keep, recent, lens, left_pad, t_cap)
    dst = _alloc_like(cache, B, keep if t_cap is None else t_cap)
    new = torch.zeros((B, H, dst["k_codes"].shape[2]), dtype=torch.float32, device=weights.device)
    index, count = tq_evict_select(weights, T, keep, recent, lens=lens, left_pad=left_pad)
    _, length = tq_cache_gather(cache, dst, index, count=count, src_weights=weights, dst_weights=new)
    return dst, new, length


# ---- Lloyd-Max table fit (turboquant-tables.ts) -----------------------------------
def tq_lloyd_max_fit(x: torch.Tensor, init: torch.Tensor, iters: int, workspace=None, stream=None,
                     spin_limit: int = 0, absent_block: int = -1):
    """Lloyd-Max fit of len(init) levels to the fp32 samples x (device), from
    the ascending centroids init -> (centroids, boundaries), fp32 tensors.
    spin_limit / absent_block: see tq_lloyd_max_fit_bounded (0 / -1: the
    plain fit); tq_lloyd_max_fit_status(workspace) reports a give-up."""
    if x.dtype != torch.float32 or init.dtype != torch.float32 or not (x.is_contiguous() and init.is_contiguous()):
        raise ValueError("x and init must be contiguous float32 tensors")
    K = init.numel()
    r = int(lib().tq_lloyd_max_fit_workspace_size(K))
    if r < 0:
        raise TQError(-r, "tq_lloyd_max_fit_workspace_size")
    if workspace is None:
        workspace = torch.empty(r, dtype=torch.uint8, device=x.device)
    c = torch.empty(K, dtype=torch.float32, device=x.device)
    b = torch.empty(max(K - 1, 1), dtype=torch.float32, device=x.device)
    st = lib().tq_lloyd_max_fit_bounded(x.data_ptr(), x.numel(), K, int(iters), init.data_ptr(), c.data_ptr(),
                                        b.data_ptr(), workspace.data_ptr(), workspace.numel(), int(spin_limit),
                                        int(absent_block), _stream_handle(stream, x.device))
    _check(st, "tq_lloyd_max_fit")
    return c, b[: K - 1]


def tq_lloyd_max_fit_status(workspace: torch.Tensor, stream=None) -> int:
    """Waits for `stream`, then returns the status of the last fit run with
    `workspace`: 0 (TQ_OK) or 7 (TQ_ERR_TIMEOUT: a grid-barrier wait gave up)."""
    st = int(lib().tq_lloyd_max_fit_status(workspace.data_ptr(), _stream_handle(stream, workspace.device)))
    if st not in (0, 7):
        raise TQError(st, "tq_lloyd_max_fit_status")
    return st
