"""Thin Python binding of the C ABI (include/tq.h): argument marshalling only.

Every function has the name of the C entry point it calls and forwards
device pointers of torch tensors (``data_ptr()``) and the current CUDA
stream.  No arithmetic of the method happens here.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import (TQ_BF16, TQ_F16, TQ_F32, TQ_KV8, TQ_MAX_TOPK, TQ_POLAR, TQ_MSE, TQ_PROD, TQ_STATUS_LAYOUT,
                   TQ_STATUS_RANGE, TQ_STATUS_TIMEOUT, TQError, check, lib)

__all__ = [
    "TQ_MSE", "TQ_PROD", "TQ_F32", "TQ_BF16", "TQ_F16", "TQ_MAX_TOPK", "TQ_STATUS_TIMEOUT", "TQ_STATUS_LAYOUT", "TQError", "Handle", "code_words", "sign_words",
    "tq_make_codebook", "tq_make_rotation", "tq_create", "tq_quant_mse", "tq_dequant_mse", "tq_quant_prod",
    "tq_quant_prod_workspace",
    "tq_ip_scores", "tq_ip_scores_workspace", "tq_attn_decode", "tq_attn_decode_workspace", "tq_version",
    "tq_attn_decode_static", "tq_quant_gather", "tq_attn_logits", "tq_attn_logits_workspace", "tq_device_status",
    "tq_attn_decode_partial", "tq_attn_decode_partial_workspace", "tq_attn_merge", "tq_topk_merge",
    "tq_quant_paged", "tq_attn_decode_paged", "tq_quant_gather_groups", "tq_attn_prefill",
    "tq_attn_prefill_workspace", "TQ_POLAR", "tq_polar_codebook", "tq_create_polar", "tq_quant_polar",
    "tq_dequant_polar", "TQ_KV8", "TQ_STATUS_RANGE", "tq_create_kv8", "tq_quant_kv8", "tq_dequant_kv8",
    "tq_attn_prompt", "tq_attn_prompt_workspace", "tq_attn_tree", "tq_attn_tree_workspace",
]


def code_words(b: int, d: int) -> int:
    return ((d + 31) // 32) * b


def sign_words(d: int) -> int:
    return (d + 31) // 32


def _dptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor (this library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def tq_version() -> str:
    return lib.tq_version().decode()


def tq_make_codebook(b: int, d: int) -> tuple[np.ndarray, np.ndarray]:
    c = np.zeros(2 ** b)
    t = np.zeros(2 ** b - 1)
    check("tq_make_codebook", lib.tq_make_codebook(b, d, _dptr(c), _dptr(t)))
    return c, t


def tq_make_rotation(G: np.ndarray) -> np.ndarray:
    G = np.ascontiguousarray(G, dtype=np.float64)
    d = G.shape[0]
    Pi = np.zeros((d, d))
    check("tq_make_rotation", lib.tq_make_rotation(d, _dptr(G), _dptr(Pi)))
    return Pi


class Handle:
    """Owns a tq_handle (device constants); destroyed with the object."""

    def __init__(self, ptr: int, d: int, b: int, variant: int, bh: int = 0):
        self.ptr = ptr
        self.d, self.b, self.variant, self.bh = d, b, variant, bh
        self.bm = b - 1 if variant == TQ_PROD else b
        # where its constants and status word are: the device that was current when it was made
        self.device = torch.cuda.current_device() if ptr and torch.cuda.is_available() else -1

    @property
    def words(self) -> int:
        if self.variant == TQ_POLAR:
            return code_words(self.b, self.d // 2) + code_words(self.bh, self.d // 2 - 1)
        if self.variant == TQ_KV8:
            return self.d // 4
        return code_words(self.bm, self.d)

    def close(self):
        if self.ptr:
            check("tq_destroy", lib.tq_destroy(self.ptr))
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tq_create(d: int, b: int, variant: int, Pi: np.ndarray, S: np.ndarray | None = None,
              centroids: np.ndarray | None = None) -> Handle:
    Pi = np.ascontiguousarray(Pi, dtype=np.float64)
    Sa = None if S is None else np.ascontiguousarray(S, dtype=np.float64)
    ca = None if centroids is None else np.ascontiguousarray(centroids, dtype=np.float64)
    h = ctypes.c_void_p()
    check("tq_create", lib.tq_create(ctypes.byref(h), d, b, variant, _dptr(Pi),
                                     None if Sa is None else _dptr(Sa), None if ca is None else _dptr(ca)))
    return Handle(h.value, d, b, variant)


def tq_polar_codebook(b: int, level: int) -> tuple[np.ndarray, np.ndarray]:
    c = np.zeros(2 ** b)
    t = np.zeros(2 ** b - 1)
    check("tq_polar_codebook", lib.tq_polar_codebook(b, level, _dptr(c), _dptr(t)))
    return c, t


def tq_create_polar(d: int, b1: int, bh: int, Pi: np.ndarray) -> Handle:
    """A PolarQuant instance: b1 bits for level-1 angles, bh for the others."""
    Pi = np.ascontiguousarray(Pi, dtype=np.float64)
    h = ctypes.c_void_p()
    check("tq_create_polar", lib.tq_create_polar(ctypes.byref(h), d, b1, bh, _dptr(Pi)))
    return Handle(h.value, d, b1, TQ_POLAR, bh)


def tq_quant_polar(h: Handle, x: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor, out_stride: int = 1,
                   stream=None) -> None:
    check("tq_quant_polar", lib.tq_quant_polar(h.ptr, _ptr(x), _dtype_code(x), x.shape[0], x.shape[1], _ptr(codes),
                                               _ptr(norms), out_stride, _stream(stream)))


def tq_dequant_polar(h: Handle, codes: torch.Tensor, norms: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    check("tq_dequant_polar", lib.tq_dequant_polar(h.ptr, _ptr(codes), _ptr(norms), codes.shape[0], _ptr(out),
                                                   _dtype_code(out), _stream(stream)))


def tq_quant_mse(h: Handle, x: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor,
                 out_stride: int = 1, stream=None) -> None:
    N = x.shape[0]
    check("tq_quant_mse", lib.tq_quant_mse(h.ptr, _ptr(x), _dtype_code(x), N, x.shape[1], _ptr(codes),
                                           _ptr(norms), out_stride, _stream(stream)))


def tq_dequant_mse(h: Handle, codes: torch.Tensor, norms: torch.Tensor, out: torch.Tensor,
                   stream=None) -> None:
    check("tq_dequant_mse", lib.tq_dequant_mse(h.ptr, _ptr(codes), _ptr(norms), codes.shape[0], _ptr(out),
                                               _dtype_code(out), _stream(stream)))


def tq_quant_prod_workspace(h: Handle, N: int) -> int:
    return int(lib.tq_quant_prod_workspace(h.ptr, N))


def tq_quant_prod(h: Handle, x: torch.Tensor, codes: torch.Tensor, signs: torch.Tensor,
                  norms: torch.Tensor, rnorms: torch.Tensor, out_stride: int = 1, workspace=None,
                  stream=None) -> None:
    """TurboQuant_prod quantization (tq_quant_prod_ws; the workspace, needed only
    above d = 256, is allocated here when none is passed)."""
    N = x.shape[0]
    if workspace is None:
        nbytes = tq_quant_prod_workspace(h, N)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    check("tq_quant_prod_ws", lib.tq_quant_prod_ws(h.ptr, _ptr(x), _dtype_code(x), N, x.shape[1], _ptr(codes),
                                                   _ptr(signs), _ptr(norms), _ptr(rnorms), out_stride,
                                                   _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                                   _stream(stream)))


def tq_ip_scores_workspace(h: Handle, nq: int, N: int, topk: int = 0) -> int:
    return int(lib.tq_ip_scores_workspace(h.ptr, nq, N, topk))


def tq_ip_scores(h: Handle, q: torch.Tensor, codes: torch.Tensor, signs, norms: torch.Tensor, rnorms,
                 scores=None, topk: int = 0, top_idx=None, top_val=None, workspace=None,
                 stream=None) -> None:
    nq, N = q.shape[0], codes.shape[0]
    if workspace is None:
        workspace = torch.empty(max(1, tq_ip_scores_workspace(h, nq, N, topk)), dtype=torch.uint8,
                                device=q.device)
    check("tq_ip_scores", lib.tq_ip_scores(h.ptr, _ptr(q), nq, _ptr(codes), _ptr(signs), _ptr(norms),
                                           _ptr(rnorms), N, _ptr(scores), topk, _ptr(top_idx),
                                           _ptr(top_val), _ptr(workspace), workspace.numel(),
                                           _stream(stream)))


def tq_attn_decode_workspace(hk: Handle, B: int, Hq: int, Hkv: int, T: int) -> int:
    return int(lib.tq_attn_decode_workspace(hk.ptr, B, Hq, Hkv, T))


def tq_attn_decode(hk: Handle, hv: Handle, q: torch.Tensor, Hkv: int, T: int, kv_stride: int,
                   kcodes, ksigns, knorms, krnorms, vcodes, vnorms, scale: float, out: torch.Tensor,
                   workspace=None, stream=None) -> None:
    B, Hq, _ = q.shape
    if workspace is None:
        workspace = torch.empty(max(1, tq_attn_decode_workspace(hk, B, Hq, Hkv, T)), dtype=torch.uint8,
                                device=q.device)
    check("tq_attn_decode", lib.tq_attn_decode(hk.ptr, hv.ptr, _ptr(q), _dtype_code(q), B, Hq, Hkv, T,
                                               kv_stride, _ptr(kcodes), _ptr(ksigns), _ptr(knorms),
                                               _ptr(krnorms), _ptr(vcodes), _ptr(vnorms), float(scale),
                                               _ptr(out), _ptr(workspace), workspace.numel(),
                                               _stream(stream)))


def tq_attn_decode_static(hk: Handle, hv: Handle, q: torch.Tensor, Hkv: int, T: int, kv_stride: int,
                          kcodes, ksigns, knorms, krnorms, vcodes, vnorms, scale: float, out: torch.Tensor,
                          stream=None) -> None:
    """tq_attn_decode without a workspace, for callers that may not allocate
    device memory: the scratch lives in a fixed array inside the library (see
    include/tq.h for its limit and for the rule that overlapping calls race)."""
    B, Hq, _ = q.shape
    check("tq_attn_decode_static", lib.tq_attn_decode_static(
        hk.ptr, hv.ptr, _ptr(q), _dtype_code(q), B, Hq, Hkv, T, kv_stride, _ptr(kcodes), _ptr(ksigns),
        _ptr(knorms), _ptr(krnorms), _ptr(vcodes), _ptr(vnorms), float(scale), _ptr(out), _stream(stream)))


def tq_attn_decode_partial_workspace(hk: Handle, B: int, Hq: int, Hkv: int, T: int) -> int:
    return int(lib.tq_attn_decode_partial_workspace(hk.ptr, B, Hq, Hkv, T))


def tq_attn_decode_partial(hk: Handle, hv: Handle, q: torch.Tensor, Hkv: int, T: int, kv_stride: int,
                           kcodes, ksigns, knorms, krnorms, vcodes, vnorms, scale: float, partial: torch.Tensor,
                           workspace=None, stream=None) -> None:
    """Softmax state [B*Hq][d + 2] (acc in the rotated value frame, m, l) of the
    decode step over the context slice held here (T may be 0)."""
    B, Hq, _ = q.shape
    if workspace is None:
        workspace = torch.empty(max(1, tq_attn_decode_partial_workspace(hk, B, Hq, Hkv, T)), dtype=torch.uint8,
                                device=q.device)
    check("tq_attn_decode_partial", lib.tq_attn_decode_partial(
        hk.ptr, hv.ptr, _ptr(q), _dtype_code(q), B, Hq, Hkv, T, kv_stride, _ptr(kcodes), _ptr(ksigns),
        _ptr(knorms), _ptr(krnorms), _ptr(vcodes), _ptr(vnorms), float(scale), _ptr(partial), _ptr(workspace),
        workspace.numel(), _stream(stream)))


def tq_attn_merge(hv: Handle, partials: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Combine [R][rows][d + 2] slice records into out [rows][d]."""
    R, rows = partials.shape[0], partials.shape[1]
    check("tq_attn_merge", lib.tq_attn_merge(hv.ptr, _ptr(partials), R, rows, _ptr(out), _stream(stream)))


def tq_topk_merge(val: torch.Tensor, idx: torch.Tensor, offsets, out_idx: torch.Tensor, out_val: torch.Tensor,
                  stream=None) -> None:
    """Global top-k from [R][nq][k] per-slice lists; offsets[r] = first global index of slice r."""
    R, nq, k = val.shape
    offs = (ctypes.c_int64 * R)(*[int(o) for o in offsets])
    check("tq_topk_merge", lib.tq_topk_merge(_ptr(val), _ptr(idx), R, nq, k, offs, _ptr(out_idx), _ptr(out_val),
                                             _stream(stream)))


def _rn_code(t) -> int:
    return TQ_F16 if t.dtype == torch.float16 else TQ_F32


def tq_quant_paged(h: Handle, x: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor,
                   signs=None, rnorms=None, channels=None, stream=None) -> None:
    """Quantize the rows of x into cache rows slots[i] (int64); rnorms may be
    float32 or float16 storage."""
    rn_dtype = _rn_code(rnorms) if rnorms is not None else TQ_F32
    check("tq_quant_paged", lib.tq_quant_paged(h.ptr, _ptr(x), _dtype_code(x), x.shape[0], x.shape[1], _ptr(channels),
                                               _ptr(slots), _ptr(codes), _ptr(signs), _ptr(norms), _ptr(rnorms),
                                               rn_dtype, _stream(stream)))


def tq_attn_decode_paged(hk: Handle, hv: Handle, q: torch.Tensor, Hkv: int, T: int, block_table: torch.Tensor,
                         page_size: int, kcodes, ksigns, knorms, krnorms, vcodes, vnorms, scale: float,
                         out: torch.Tensor, workspace=None, stream=None) -> None:
    """Decode over a paged cache; block_table is [B*Hkv][max_pages] int32."""
    B, Hq, _ = q.shape
    if workspace is None:
        workspace = torch.empty(max(1, tq_attn_decode_workspace(hk, B, Hq, Hkv, T)), dtype=torch.uint8,
                                device=q.device)
    check("tq_attn_decode_paged", lib.tq_attn_decode_paged(
        hk.ptr, hv.ptr, _ptr(q), _dtype_code(q), B, Hq, Hkv, T, _ptr(block_table), block_table.shape[1], page_size,
        _ptr(kcodes), _ptr(ksigns), _ptr(knorms), _ptr(krnorms), _rn_code(krnorms), _ptr(vcodes), _ptr(vnorms),
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)))


def tq_attn_prefill_workspace(hk: Handle, B: int, nq: int, Hq: int, Hkv: int, T: int) -> int:
    return int(lib.tq_attn_prefill_workspace(hk.ptr, B, nq, Hq, Hkv, T))


def tq_attn_prefill(hk: Handle, hv: Handle, q: torch.Tensor, Hkv: int, T: int, kv_stride: int, kcodes, ksigns,
                    knorms, krnorms, vcodes, vnorms, scale: float, out: torch.Tensor, workspace=None,
                    stream=None) -> None:
    """Causal attention of a block of nq new tokens, q [B][nq][Hq][d], over a
    cache of T tokens that ends with them; out [B][nq][Hq][d] float32."""
    B, nq, Hq, _ = q.shape
    if workspace is None:
        workspace = torch.empty(max(1, tq_attn_prefill_workspace(hk, B, nq, Hq, Hkv, T)), dtype=torch.uint8,
                                device=q.device)
    check("tq_attn_prefill", lib.tq_attn_prefill(
        hk.ptr, hv.ptr, _ptr(q), _dtype_code(q), B, nq, Hq, Hkv, T, kv_stride, _ptr(kcodes), _ptr(ksigns),
        _ptr(knorms), _ptr(krnorms), _ptr(vcodes), _ptr(vnorms), float(scale), _ptr(out), _ptr(workspace),
        workspace.numel(), _stream(stream)))


# ---- the 8-bit cache

_DTYPES = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}


def _dtype3(t: torch.Tensor) -> int:
    """The type code of a call that also takes float16 activations."""
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


# These calls are made for every layer of every step, so their checks are written
# to cost little: device numbers instead of device objects, sizes instead of shapes.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_on(stream, t: torch.Tensor) -> int:
    """The given stream, or the current one of the device that holds t."""
    if stream is None:
        return _raw_stream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _same_device(h: Handle, first: torch.Tensor, *rest) -> None:
    try:
        dev = first.get_device()
        if dev < 0:
            raise ValueError("expected a CUDA tensor (this library has no CPU path)")
        if dev != h.device and h.device >= 0:
            raise ValueError(f"tensors on {first.device}, a handle of device {h.device}")
        for t in rest:
            if t is not None and t.get_device() != dev:
                raise ValueError("expected a CUDA tensor (this library has no CPU path)" if t.get_device() < 0 else
                                 f"tensors on {first.device} and {t.device}")
    except AttributeError:
        raise TypeError("expected a torch.Tensor") from None


def _dense(*tensors) -> list:
    """The addresses of contiguous tensors (None for None)."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.is_contiguous():
            out.append(t.data_ptr())
        else:
            raise ValueError("expected a contiguous tensor")
    return out


def _token_rows(t: torch.Tensor, name: str, heads: int, d: int) -> int:
    """Checks [tokens][heads][d] with whole heads side by side; returns the
    elements from one token to the next (a slice of a fused projection has more
    than heads d of them)."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name}: expected [tokens][{heads}][{d}], got {tuple(shape)}")
    if t.is_contiguous():
        return heads * d
    if (d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    return t.stride(0) if shape[0] > 1 else heads * d


def _cache_rows(h: Handle, kcodes, kscales, vcodes, vscales) -> int:
    """Checks the four cache arrays (the values' may be None); returns their rows."""
    rows = kcodes.size(0)
    shape, flat, int8, f32 = (rows, h.d), (rows,), torch.int8, torch.float32
    if (kcodes.dtype is not int8 or kcodes.shape != shape or
            (vcodes is not None and (vcodes.dtype is not int8 or vcodes.shape != shape))):
        raise ValueError(f"codes: expected int8 [rows][{h.d}], the same rows for keys and values")
    if (kscales is None or kscales.dtype is not f32 or kscales.shape != flat or (vscales is None) != (vcodes is None) or
            (vscales is not None and (vscales.dtype is not f32 or vscales.shape != flat))):
        raise ValueError("scales: expected float32 [rows], as many as the codes")
    return rows


def tq_create_kv8(d: int) -> Handle:
    """A handle of the 8-bit cache for heads of dimension d."""
    h = ctypes.c_void_p()
    check("tq_create_kv8", lib.tq_create_kv8(ctypes.byref(h), d))
    return Handle(h.value, d, 8, TQ_KV8)


def tq_quant_kv8(h: Handle, k: torch.Tensor, v, slots: torch.Tensor, kcodes: torch.Tensor, kscales: torch.Tensor,
                 vcodes=None, vscales=None, stream=None) -> None:
    """Quantize the keys and values of n tokens, [n][Hkv][d] each (a token
    stride is allowed; v may be None), into cache rows slots [n][Hkv] (int64,
    negative: left out)."""
    _same_device(h, k, v, slots, kcodes, kscales, vcodes, vscales)
    if k.dim() != 3:
        raise ValueError(f"k: expected [tokens][heads][d], got {tuple(k.shape)}")
    n, Hkv = k.size(0), k.size(1)
    ks = _token_rows(k, "k", Hkv, h.d)
    vs = 0 if v is None else _token_rows(v, "v", Hkv, h.d)
    if v is not None and (v.size(0) != n or v.dtype != k.dtype or vcodes is None or vscales is None):
        raise ValueError("v: expected as many tokens as k, of its type, and arrays for their codes and scales")
    if slots.dtype is not torch.int64 or slots.numel() != n * Hkv:
        raise ValueError(f"slots: expected int64 [{n}][{Hkv}], got {slots.dtype} {tuple(slots.shape)}")
    rows = _cache_rows(h, kcodes, kscales, vcodes, vscales)
    if n == 0 or Hkv == 0:
        return
    check("tq_quant_kv8", lib.tq_quant_kv8(h.ptr, k.data_ptr(), None if v is None else v.data_ptr(), _dtype3(k), n, Hkv,
                                           ks, vs, *_dense(slots, kcodes, kscales, vcodes, vscales), rows,
                                           _stream_on(stream, k)))


def tq_dequant_kv8(h: Handle, slots: torch.Tensor, kcodes: torch.Tensor, kscales: torch.Tensor, vcodes, vscales,
                   k: torch.Tensor, v=None, stream=None) -> None:
    """Read cache rows slots [n] (int64; outside the cache: zeros) back into k
    and v, [n][d] each (v may be None)."""
    _same_device(h, slots, kcodes, kscales, vcodes, vscales, k, v)
    n, d = slots.numel(), h.d
    if slots.dtype is not torch.int64:
        raise ValueError(f"slots: expected int64, got {slots.dtype}")
    for t in (k,) if v is None else (k, v):
        if t.numel() != n * d or t.size(-1) != d or t.dtype is not k.dtype:
            raise ValueError(f"outputs: expected [{n}][{d}] of one type, got {tuple(t.shape)} {t.dtype}")
    if v is not None and (vcodes is None or vscales is None):
        raise ValueError("v: needs the values' codes and scales")
    rows = _cache_rows(h, kcodes, kscales, vcodes, vscales)
    if n == 0:
        return
    check("tq_dequant_kv8", lib.tq_dequant_kv8(h.ptr, n, *_dense(slots, kcodes, kscales, vcodes, vscales), rows,
                                               *_dense(k, v), _dtype3(k), _stream_on(stream, k)))


# ---- attention over prompts and over the 8-bit cache

def _scratch(nbytes: int, like: torch.Tensor, stream):
    """A workspace that belongs to the stream the call runs on (so that it may be
    freed when the call returns), or None where none is needed."""
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_on(stream, like), device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _outputs(q: torch.Tensor, out: torch.Tensor, lse) -> None:
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError(f"out: expected {tuple(q.shape)} {q.dtype}, got {tuple(out.shape)} {out.dtype}")
    if lse is not None and (lse.shape != q.shape[:-1] or lse.dtype is not torch.float32):
        raise ValueError(f"lse: expected float32 {tuple(q.shape[:-1])}, got {lse.dtype} {tuple(lse.shape)}")


def tq_attn_prompt_workspace(h: Handle, nseq: int, total: int, Hq: int, Hkv: int) -> int:
    return int(lib.tq_attn_prompt_workspace(h.ptr, nseq, total, Hq, Hkv))


def tq_attn_prompt(h: Handle, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                   scale: float, out: torch.Tensor, lse=None, workspace=None, stream=None) -> None:
    """Causal attention over packed prompts: q [total][Hq][d], k and v
    [total][Hkv][d] (bfloat16 or float16, a token stride allowed), sequence s in
    tokens cu_seqlens[s] .. cu_seqlens[s+1]-1 (int32 [nseq+1]); out
    [total][Hq][d], lse [total][Hq] float32.  h gives d: any handle."""
    _same_device(h, q, k, v, cu_seqlens, out, lse, workspace)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k: expected [tokens][heads][d]")
    total, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    strides = _token_rows(q, "q", Hq, h.d), _token_rows(k, "k", Hkv, h.d), _token_rows(v, "v", Hkv, h.d)
    if k.shape[0] != total or v.shape[0] != total or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v: expected the same tokens and one type")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: expected int32 [nseq + 1]")
    _outputs(q, out, lse)
    nseq = cu_seqlens.numel() - 1
    if workspace is None:
        workspace = _scratch(tq_attn_prompt_workspace(h, nseq, total, Hq, Hkv), q, stream)
    check("tq_attn_prompt", lib.tq_attn_prompt(
        h.ptr, q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype3(q), *_dense(cu_seqlens), nseq, total, Hq, Hkv, *strides,
        float(scale), *_dense(out, lse, workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_on(stream, q)))


def tq_attn_tree_workspace(h: Handle, B: int, n: int, Hq: int, Hkv: int) -> int:
    return int(lib.tq_attn_tree_workspace(h.ptr, B, n, Hq, Hkv))


def tq_attn_tree(h: Handle, q: torch.Tensor, Hkv: int, ctx_lens: torch.Tensor, block_table: torch.Tensor,
                 page_size: int, kcodes: torch.Tensor, kscales: torch.Tensor, vcodes: torch.Tensor,
                 vscales: torch.Tensor, scale: float, out: torch.Tensor, lse=None, mask=None, draft_lens=None,
                 workspace=None, stream=None) -> None:
    """Attention of n drafted tokens per sequence, q [B][n][Hq][d] (bfloat16 or
    float16), over the 8-bit paged cache: ctx_lens [B] context tokens that all
    of them see, then draft_lens [B] (n each if None) drafted ones, of which
    token i sees those in its bits mask [B][n][ceil(n/32)] (int32; a chain if
    None); block_table is [B*Hkv][max_pages] int32."""
    _same_device(h, q, ctx_lens, block_table, kcodes, kscales, vcodes, vscales, out, lse, mask, draft_lens, workspace)
    if q.dim() != 4 or q.shape[3] != h.d:
        raise ValueError(f"q: expected [B][n][Hq][{h.d}], got {tuple(q.shape)}")
    B, n, Hq, d = q.shape
    # tokens a constant number of elements apart, each with its heads side by side
    qs = q.stride(1) if n > 1 else q.stride(0) if B > 1 else Hq * d
    if q.numel() and (q.stride(3) != 1 or (Hq > 1 and q.stride(2) != d) or (B > 1 and n > 1 and q.stride(0) != n * qs)):
        raise ValueError("q: tokens must lie a constant stride apart, their heads side by side")
    for name, t, shape in (("ctx_lens", ctx_lens, (B,)), ("draft_lens", draft_lens, (B,)),
                           ("mask", mask, (B, n, (n + 31) // 32))):
        if t is not None and (t.dtype is not torch.int32 or t.shape != shape):
            raise ValueError(f"{name}: expected int32 {shape}, got {t.dtype} {tuple(t.shape)}")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B * Hkv:
        raise ValueError(f"block_table: expected int32 [{B * Hkv}][max_pages], got {block_table.dtype} {tuple(block_table.shape)}")
    rows = _cache_rows(h, kcodes, kscales, vcodes, vscales)
    _outputs(q, out, lse)
    if workspace is None:
        workspace = _scratch(tq_attn_tree_workspace(h, B, n, Hq, Hkv), q, stream)
    check("tq_attn_tree", lib.tq_attn_tree(
        h.ptr, q.data_ptr(), _dtype3(q), qs, B, n, Hq, Hkv, *_dense(ctx_lens, draft_lens, mask, block_table),
        block_table.size(1), page_size, *_dense(kcodes, kscales, vcodes, vscales), rows, float(scale),
        *_dense(out, lse, workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_on(stream, q)))


def tq_device_status(h: Handle) -> int:
    v = ctypes.c_int(0)
    check("tq_device_status", lib.tq_device_status(h.ptr, ctypes.byref(v)))
    return v.value


def tq_quant_gather(h: Handle, x: torch.Tensor, channels: torch.Tensor, codes: torch.Tensor, norms: torch.Tensor,
                    signs=None, rnorms=None, out_stride: int = 1, stream=None) -> None:
    """Quantize x[:, channels] (one channel group of a split cache)."""
    check("tq_quant_gather", lib.tq_quant_gather(h.ptr, _ptr(x), _dtype_code(x), x.shape[0], x.shape[1],
                                                 _ptr(channels), _ptr(codes), _ptr(signs), _ptr(norms),
                                                 _ptr(rnorms), out_stride, _stream(stream)))


def tq_quant_gather_groups(handles, x: torch.Tensor, channels: torch.Tensor, codes, norms, signs=None, rnorms=None,
                           out_stride: int = 1, stream=None) -> None:
    """Every channel group of the rows of x in one launch; codes / norms /
    signs / rnorms are lists with one tensor (or None) per group."""
    n = len(handles)
    hs = (ctypes.c_void_p * n)(*[h.ptr for h in handles])
    signs = signs or [None] * n
    rnorms = rnorms or [None] * n
    check("tq_quant_gather_groups", lib.tq_quant_gather_groups(
        hs, n, _ptr(x), _dtype_code(x), x.shape[0], x.shape[1], _ptr(channels), _ptr_array(codes),
        _ptr_array(signs), _ptr_array(norms), _ptr_array(rnorms), out_stride, _stream(stream)))


def _ptr_array(items):
    arr = (ctypes.c_void_p * len(items))()
    for i, t in enumerate(items):
        arr[i] = _ptr(t)
    return arr


def tq_attn_logits_workspace(handles, B: int, Hq: int) -> int:
    hs = (ctypes.c_void_p * len(handles))(*[h.ptr for h in handles])
    return int(lib.tq_attn_logits_workspace(hs, len(handles), B, Hq))


def tq_attn_logits(handles, channels, q: torch.Tensor, Hkv: int, T: int, kv_stride: int, kcodes, ksigns, knorms,
                   krnorms, scale: float, logits: torch.Tensor, workspace=None, stream=None) -> None:
    """Logits [B][Hq][T] over a key cache of one or two channel groups (lists
    of per-group tensors); q is [B][Hq][dq]."""
    B, Hq, dq = q.shape
    hs = (ctypes.c_void_p * len(handles))(*[h.ptr for h in handles])
    if workspace is None:
        workspace = torch.empty(max(1, tq_attn_logits_workspace(handles, B, Hq)), dtype=torch.uint8,
                                device=q.device)
    check("tq_attn_logits", lib.tq_attn_logits(hs, len(handles), _ptr(channels), _ptr(q), _dtype_code(q), dq, B, Hq,
                                               Hkv, T, kv_stride, _ptr_array(kcodes), _ptr_array(ksigns),
                                               _ptr_array(knorms), _ptr_array(krnorms), float(scale), _ptr(logits),
                                               _ptr(workspace), workspace.numel(), _stream(stream)))
