"""ctypes binding of the operators between the projections of an attention layer
(include/wq.h): norm + rotation of queries and keys, the paged 4-bit key / value cache,
and attention over it.  Argument checks and marshalling only; the work is in libwq.so.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import _check, _i32, _i64, _ptr, _stream, _sz, lib




class Kv4Layout(ctypes.Structure):
    _fields_ = [("num_pages", _i64), ("kv_heads", _i32), ("head_dim", _i32), ("group", _i32), ("page_size", _i32),
                ("dtype", _i32)]


_DTYPES = {torch.float16: _lib.WQ_F16, torch.bfloat16: _lib.WQ_BF16}


def _dtype(dtype: torch.dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"keys, values and queries must be float16 or bfloat16, got {dtype}")
    return code


def _rows(t, name, dtype=None, shape=None, device=None):
    """A [T, heads, D] tensor whose heads of a token are contiguous (any stride from token to token)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    _, h, d = t.shape
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")


def _step(t):
    """Elements from token to token (a single token's stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _flat(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _layout(pages, head_dim: int, group: int, page_size: int, dtype: torch.dtype) -> Kv4Layout:
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda or pages.dtype != torch.uint8 or pages.dim() != 3:
        raise ValueError("pages must be a uint8 CUDA tensor [num_pages, kv_heads, block_bytes]")
    if not pages.is_contiguous():
        raise ValueError("pages must be contiguous")
    n, heads, block = pages.shape
    if group <= 0 or block != page_size * (head_dim + 8 * (head_dim // group)):
        raise ValueError(f"pages: a block of {page_size} tokens with head_dim {head_dim} in groups of {group} has "
                         f"{page_size * (head_dim + 8 * (head_dim // max(1, group)))} bytes, got {block}")
    return Kv4Layout(n, heads, head_dim, group, page_size, _dtype(dtype))


# ------------------------------------------------------------------ queries and keys

def wq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                    q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, eps: float = 1e-6,
                    interleaved: bool = False, q_out: torch.Tensor = None, k_out: torch.Tensor = None):
    """Norm (where a weight is given) and rotation of q [T, Hq, D] and k [T, Hkv, D] -> (q_out, k_out).

    positions int64 [T]; cos_sin fp32 [max_pos, rot]: a row's rot / 2 cosines, then its sines.  q and k may be
    slices of one packed projection; q_out / k_out may be q / k themselves."""
    _rows(q, "q")
    T, Hq, D = q.shape
    dt, dev = _dtype(q.dtype), q.device
    _rows(k, "k", q.dtype, device=dev)
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k must be [{T}, heads, {D}], got {tuple(k.shape)}")
    Hkv = k.shape[1]
    _flat(positions, "positions", torch.int64, (T,), dev)
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_pos, rot]")
    _flat(cos_sin, "cos_sin", torch.float32, cos_sin.shape, dev)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _flat(w, name, q.dtype, (D,), dev)
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    else:
        _rows(q_out, "q_out", q.dtype, q.shape, dev)
    if k_out is None:
        k_out = torch.empty((T, Hkv, D), dtype=q.dtype, device=dev)
    else:
        _rows(k_out, "k_out", q.dtype, k.shape, dev)
    _check(lib().wq_qk_norm_rope(_ptr(q), _step(q), _ptr(k), _step(k), dt, T, Hq, Hkv, D, _ptr(q_weight),
                                 _ptr(k_weight), eps, _ptr(positions), _ptr(cos_sin), cos_sin.shape[0],
                                 cos_sin.shape[1], int(interleaved), _ptr(q_out), _step(q_out), _ptr(k_out),
                                 _step(k_out), _stream(q)), "wq_qk_norm_rope")
    return q_out, k_out


# ------------------------------------------------------------------ 4-bit cache

def wq_kv4_page_bytes(kv_heads: int, head_dim: int, group: int, page_size: int) -> int:
    """Bytes of one page of the cache, all heads."""
    b = _sz(0)
    _check(lib().wq_kv4_page_bytes(ctypes.byref(Kv4Layout(0, kv_heads, head_dim, group, page_size, 0)),
                                   ctypes.byref(b)), "wq_kv4_page_bytes")
    return b.value


def wq_kv4_pages(num_pages: int, kv_heads: int, head_dim: int, group: int, page_size: int, device) -> torch.Tensor:
    """A zeroed cache: uint8 [num_pages, kv_heads, block_bytes]."""
    block = wq_kv4_page_bytes(kv_heads, head_dim, group, page_size) // kv_heads
    return torch.zeros((num_pages, kv_heads, block), dtype=torch.uint8, device=device)


def wq_kv4_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pages: torch.Tensor, group: int,
                 page_size: int) -> None:
    """Quantises k, v [T, kv_heads, D] into slots (int64 [T]: page * page_size + place; negative: skip)."""
    _rows(k, "k")
    T, H, D = k.shape
    _rows(v, "v", k.dtype, k.shape, k.device)
    _flat(slots, "slots", torch.int64, (T,), k.device)
    lay = _layout(pages, D, group, page_size, k.dtype)
    if lay.kv_heads != H or pages.device != k.device:
        raise ValueError(f"pages must hold {H} heads on {k.device}")
    _check(lib().wq_kv4_write(_ptr(k), _step(k), _ptr(v), _step(v), _ptr(slots), T, ctypes.byref(lay), _ptr(pages),
                              _stream(k)), "wq_kv4_write")


def wq_kv4_read(pages: torch.Tensor, slots: torch.Tensor, head_dim: int, group: int, page_size: int,
                dtype: torch.dtype, k: torch.Tensor = None, v: torch.Tensor = None):
    """The cache's values in slots (int64 [T]; negative: zeros) -> (k, v) [T, kv_heads, head_dim]."""
    lay = _layout(pages, head_dim, group, page_size, dtype)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be int64 [T]")
    dev = pages.device
    _flat(slots, "slots", torch.int64, slots.shape, dev)
    shape = (slots.shape[0], lay.kv_heads, head_dim)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _rows(k, "k", dtype, shape, dev)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _rows(v, "v", dtype, shape, dev)
    _check(lib().wq_kv4_read(_ptr(pages), ctypes.byref(lay), _ptr(slots), shape[0], _ptr(k), _step(k), _ptr(v),
                             _step(v), _stream(pages)), "wq_kv4_read")
    return k, v


# ------------------------------------------------------------------ attention

_ws_cache: dict = {}


def attn_kv4_workspace(lay: Kv4Layout, q_heads: int, max_q: int, device):
    """(tensor or None, bytes): a zero-filled workspace shared by calls on one stream.

    A call that is being captured into a graph gets its own, which the graph keeps and clears."""
    need = _sz(0)
    _check(lib().wq_attn_kv4_workspace_bytes(ctypes.byref(lay), q_heads, max_q, ctypes.byref(need)),
           "wq_attn_kv4_workspace_bytes")
    if need.value == 0:
        return None, 0
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(need.value, dtype=torch.uint8, device=device), need.value
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need.value:
        buf = torch.zeros(need.value, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf, buf.numel()


def wq_attn_kv4(q: torch.Tensor, pages: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, group: int,
                page_size: int, cu_q: torch.Tensor = None, max_q: int = 1, scale: float = None, causal: bool = True,
                window: int = 0, out: torch.Tensor = None, lse: torch.Tensor = None,
                ws: torch.Tensor = None) -> torch.Tensor:
    """Attention of q [T, q_heads, D] over the 4-bit cache -> out [T, q_heads, D].

    block_table int32 [B, pages of a sequence], kv_lens int32 [B] (the new tokens included); cu_q int32 [B + 1]
    gives each sequence's queries (None: one each), max_q their largest number.  scale defaults to
    1 / sqrt(D); window > 0 keeps the last `window` tokens of each query; lse: fp32 [T, q_heads] to fill."""
    _rows(q, "q")
    T, Hq, D = q.shape
    dev = q.device
    lay = _layout(pages, D, group, page_size, q.dtype)
    if pages.device != dev:
        raise ValueError(f"pages must be on {dev}")
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise ValueError("kv_lens must be int32 [B]")
    B = kv_lens.shape[0]
    _flat(kv_lens, "kv_lens", torch.int32, (B,), dev)
    if (not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.shape[0] != B):
        raise ValueError(f"block_table must be int32 [{B}, pages]")
    _flat(block_table, "block_table", torch.int32, block_table.shape, dev)
    if cu_q is not None:
        _flat(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    else:
        _rows(out, "out", q.dtype, q.shape, dev)
    if lse is not None:
        _flat(lse, "lse", torch.float32, (T, Hq), dev)
    if ws is None:
        ws, ws_bytes = attn_kv4_workspace(lay, Hq, max_q, dev)
    else:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().wq_attn_kv4(_ptr(q), _step(q), Hq, _ptr(cu_q), B, T, max_q, _ptr(pages), ctypes.byref(lay),
                             _ptr(block_table), block_table.shape[1], _ptr(kv_lens),
                             1.0 / math.sqrt(D) if scale is None else scale, int(causal), window, _ptr(out),
                             _step(out), _ptr(lse), _ptr(ws), ws_bytes, _stream(q)), "wq_attn_kv4")
    return out
