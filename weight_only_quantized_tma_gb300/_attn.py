"""ctypes binding of the operators between the projections of an attention layer
(include/wq.h): norm + rotation of queries and keys, the paged 4-bit key / value cache,
and attention over it.  Argument checks and marshalling only; the work is in libwq.so.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import WQError, _i32, _i64, _sz, lib


class Kv4Layout(ctypes.Structure):
    _fields_ = [("num_pages", _i64), ("kv_heads", _i32), ("head_dim", _i32), ("group", _i32), ("page_size", _i32),
                ("dtype", _i32)]


_DTYPES = {torch.float16: _lib.WQ_F16, torch.bfloat16: _lib.WQ_BF16}
_fns: dict = {}
_layouts: dict = {}


_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_several = None     # whether there is more than one device (with one, nothing is asked: 0.1 us of a call's 6)


def _foreign(device) -> bool:
    """Whether another device is current."""
    global _several
    if _several is None:
        _several = torch.cuda.device_count() > 1
    return _several and device.index != _current()


def _call(name: str, device, *args) -> None:
    """The library function `name`; a decode step's calls are short, so it is looked up once.

    The library works on the current device, so the tensors' own is made that (None: host only)."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    if _several is not False and device is not None and _foreign(device):
        with torch.cuda.device(device):
            status = fn(*args)
    else:
        status = fn(*args)
    if status != 0:
        raise WQError(status, name)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    """The current stream's handle (torch's short way to it where there is one: 0.1 against 2 us)."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dtype(dtype: torch.dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"keys, values and queries must be float16 or bfloat16, got {dtype}")
    return code


def _rows(t, name, dtype=None, shape=None, device=None):
    """A [T, heads, D] tensor whose heads of a token are contiguous (any stride from token to token);
    returns the elements from token to token (a single token's stride says nothing)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    got = t.shape
    if len(got) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(got)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and got != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(got)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    n, h, d = got
    step, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return step if n > 1 else h * d


def _flat(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _int32(**sizes):
    """ctypes would drop the high bits of what an int32 does not hold, and a wrong size pass for a right one."""
    for name, x in sizes.items():
        if not -(1 << 31) <= x < 1 << 31:
            raise ValueError(f"{name} is out of range: {x}")


def _layout(pages, head_dim: int, group: int, page_size: int, dtype: torch.dtype):
    """(the layout, a reference to pass); pages [num_pages, kv_heads, block_bytes] gives the rest."""
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda or pages.dtype is not torch.uint8 or pages.dim() != 3:
        raise ValueError("pages must be a uint8 CUDA tensor [num_pages, kv_heads, block_bytes]")
    if not pages.is_contiguous():
        raise ValueError("pages must be contiguous")
    key = (pages.shape, head_dim, group, page_size, dtype)
    got = _layouts.get(key)
    if got is None:
        n, heads, block = pages.shape
        _int32(kv_heads=heads, head_dim=head_dim, group=group, page_size=page_size)
        if group <= 0 or block != page_size * (head_dim + 8 * (head_dim // group)):
            raise ValueError(f"pages: a block of {page_size} tokens with head_dim {head_dim} in groups of {group} has "
                             f"{page_size * (head_dim + 8 * (head_dim // max(1, group)))} bytes, got {block}")
        lay = Kv4Layout(n, heads, head_dim, group, page_size, _dtype(dtype))
        if len(_layouts) > 256:
            _layouts.clear()
        got = _layouts[key] = (lay, ctypes.byref(lay))
    return got


def _empty(t):
    """A contiguous tensor of t's shape, type and device (empty_like takes less time where t is contiguous itself:
    16.7 against 17.5 us for a call of wq_qk_norm_rope)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


# ------------------------------------------------------------------ queries and keys

def wq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                    q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, eps: float = 1e-6,
                    interleaved: bool = False, q_out: torch.Tensor = None, k_out: torch.Tensor = None):
    """Norm (where a weight is given) and rotation of q [T, Hq, D] and k [T, Hkv, D] -> (q_out, k_out).

    positions int64 [T]; cos_sin fp32 [max_pos, rot]: a row's rot / 2 cosines, then its sines.  q and k may be
    slices of one packed projection; q_out / k_out may be q / k themselves."""
    q_step = _rows(q, "q")
    T, Hq, D = q.shape
    dtype, dev = q.dtype, q.device
    dt = _dtype(dtype)
    k_step = _rows(k, "k", dtype, None, dev)
    Hkv = k.shape[1]
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k must be [{T}, heads, {D}], got {tuple(k.shape)}")
    _flat(positions, "positions", torch.int64, (T,), dev)
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_pos, rot]")
    most, rot = cos_sin.shape
    _flat(cos_sin, "cos_sin", torch.float32, (most, rot), dev)
    if q_weight is not None:
        _flat(q_weight, "q_weight", dtype, (D,), dev)
    if k_weight is not None:
        _flat(k_weight, "k_weight", dtype, (D,), dev)
    if q_out is None:
        q_out, qo_step = _empty(q), Hq * D
    else:
        qo_step = _rows(q_out, "q_out", dtype, q.shape, dev)
    if k_out is None:
        k_out, ko_step = _empty(k), Hkv * D
    else:
        ko_step = _rows(k_out, "k_out", dtype, k.shape, dev)
    _call("wq_qk_norm_rope", dev, q.data_ptr(), q_step, k.data_ptr(), k_step, dt, T, Hq, Hkv, D,
          None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps,
          positions.data_ptr(), cos_sin.data_ptr(), most, rot, int(interleaved), q_out.data_ptr(), qo_step,
          k_out.data_ptr(), ko_step, _stream(dev))
    return q_out, k_out


# ------------------------------------------------------------------ 4-bit cache

def wq_kv4_page_bytes(kv_heads: int, head_dim: int, group: int, page_size: int) -> int:
    """Bytes of one page of the cache, all heads."""
    _int32(kv_heads=kv_heads, head_dim=head_dim, group=group, page_size=page_size)
    b = _sz(0)
    _call("wq_kv4_page_bytes", None, ctypes.byref(Kv4Layout(0, kv_heads, head_dim, group, page_size, 0)),
          ctypes.byref(b))
    return b.value


def wq_kv4_pages(num_pages: int, kv_heads: int, head_dim: int, group: int, page_size: int, device) -> torch.Tensor:
    """A zeroed cache: uint8 [num_pages, kv_heads, block_bytes]."""
    block = wq_kv4_page_bytes(kv_heads, head_dim, group, page_size) // kv_heads
    return torch.zeros((num_pages, kv_heads, block), dtype=torch.uint8, device=device)


def wq_kv4_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, pages: torch.Tensor, group: int,
                 page_size: int) -> None:
    """Quantises k, v [T, kv_heads, D] into slots (int64 [T]: page * page_size + place; negative: skip; no two
    alike: a shared one may hold parts of both tokens)."""
    k_step = _rows(k, "k")
    T, H, D = shape = k.shape
    dev = k.device
    v_step = _rows(v, "v", k.dtype, shape, dev)
    _flat(slots, "slots", torch.int64, (T,), dev)
    lay, ref = _layout(pages, D, group, page_size, k.dtype)
    if lay.kv_heads != H or pages.device != dev:
        raise ValueError(f"pages must hold {H} heads on {dev}")
    _call("wq_kv4_write", dev, k.data_ptr(), k_step, v.data_ptr(), v_step, slots.data_ptr(), T, ref, pages.data_ptr(),
          _stream(dev))


def wq_kv4_read(pages: torch.Tensor, slots: torch.Tensor, head_dim: int, group: int, page_size: int,
                dtype: torch.dtype, k: torch.Tensor = None, v: torch.Tensor = None):
    """The cache's values in slots (int64 [T]; negative: zeros) -> (k, v) [T, kv_heads, head_dim]."""
    lay, ref = _layout(pages, head_dim, group, page_size, dtype)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be int64 [T]")
    dev = pages.device
    T = slots.shape[0]
    _flat(slots, "slots", torch.int64, (T,), dev)
    shape = (T, lay.kv_heads, head_dim)
    if k is None:
        k, k_step = torch.empty(shape, dtype=dtype, device=dev), shape[1] * head_dim
    else:
        k_step = _rows(k, "k", dtype, shape, dev)
    if v is None:
        v, v_step = _empty(k), shape[1] * head_dim
    else:
        v_step = _rows(v, "v", dtype, shape, dev)
    _call("wq_kv4_read", dev, pages.data_ptr(), ref, slots.data_ptr(), T, k.data_ptr(), k_step, v.data_ptr(), v_step,
          _stream(dev))
    return k, v


# ------------------------------------------------------------------ attention

_LONGEST = (1 << 31) - 1   # no sequence is longer, so a longer window or max_q is this one
_ws_need: dict = {}
_ws_cache: dict = {}
_lib._ws_caches.append(_ws_cache)


def _capturing(device) -> bool:
    """Whether the device's current stream is being captured into a graph."""
    if _several is not False and _foreign(device):
        with torch.cuda.device(device):
            return torch.cuda.is_current_stream_capturing()
    return torch.cuda.is_current_stream_capturing()


def _workspace_bytes(layout, q_heads: int, max_q: int, device) -> int:
    lay, ref = layout
    key = (device.index, lay.kv_heads, lay.head_dim, lay.group, lay.dtype, q_heads, max_q)
    need = _ws_need.get(key)
    if need is None:
        b = _sz(0)
        _call("wq_attn_kv4_workspace_bytes", device, ref, q_heads, max_q, ctypes.byref(b))
        if len(_ws_need) > 4096:
            _ws_need.clear()
        need = _ws_need[key] = b.value
    return need


def wq_attn_kv4_workspace_bytes(pages: torch.Tensor, q_heads: int, head_dim: int, group: int, page_size: int,
                                dtype: torch.dtype, max_q: int = 1) -> int:
    """Bytes of a workspace for wq_attn_kv4 over these pages, whatever the lengths and the number of sequences."""
    _int32(q_heads=q_heads)
    return _workspace_bytes(_layout(pages, head_dim, group, page_size, dtype), q_heads, max(min(max_q, _LONGEST), 0),
                            pages.device)


def attn_kv4_workspace(layout, q_heads: int, max_q: int, device, stream: int):
    """(tensor or None, bytes): a zero-filled workspace shared by calls on one stream.

    A call that is being captured into a graph gets its own, which the graph keeps and clears."""
    need = _workspace_bytes(layout, q_heads, max_q, device)
    if need == 0:
        return None, 0
    if _capturing(device):
        return torch.zeros(need, dtype=torch.uint8, device=device), need
    key = (device.index, stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.zeros(need, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf, buf.numel()


def wq_attn_kv4(q: torch.Tensor, pages: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, group: int,
                page_size: int, cu_q: torch.Tensor = None, max_q: int = 1, scale: float = None, causal: bool = True,
                window: int = 0, out: torch.Tensor = None, lse: torch.Tensor = None,
                ws: torch.Tensor = None) -> torch.Tensor:
    """Attention of q [T, q_heads, D] over the 4-bit cache -> out [T, q_heads, D].

    block_table int32 [B, pages of a sequence], kv_lens int32 [B] (the new tokens included); cu_q int32 [B + 1]
    gives each sequence's queries (None: one each), max_q their largest number.  scale defaults to
    1 / sqrt(D); window > 0 keeps the last `window` tokens of each query; lse: fp32 [T, q_heads] to fill.
    ws: a workspace of your own, zero-filled once, of wq_attn_kv4_workspace_bytes bytes or more, for calls that do
    not overlap (None: the binding keeps one for each stream)."""
    q_step = _rows(q, "q")
    T, Hq, D = shape = q.shape
    dtype, dev = q.dtype, q.device
    layout = _layout(pages, D, group, page_size, dtype)
    if pages.device != dev:
        raise ValueError(f"pages must be on {dev}")
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise ValueError("kv_lens must be int32 [B]")
    B = kv_lens.shape[0]
    _flat(kv_lens, "kv_lens", torch.int32, (B,), dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}, pages]")
    _flat(block_table, "block_table", torch.int32, block_table.shape, dev)
    if cu_q is not None:
        _flat(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    if out is None:
        out, out_step = _empty(q), Hq * D
    else:
        out_step = _rows(out, "out", dtype, shape, dev)
    if lse is not None:
        _flat(lse, "lse", torch.float32, (T, Hq), dev)
    stream = _stream(dev)
    if not 0 <= max_q <= _LONGEST:
        max_q = _LONGEST if max_q > 0 else 0
    if not -1 <= window <= _LONGEST:
        window = _LONGEST if window > 0 else -1
    if ws is None:
        ws, ws_bytes = attn_kv4_workspace(layout, Hq, max_q, dev, stream)
    else:
        if not isinstance(ws, torch.Tensor) or ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on {dev}")
        ws_bytes = ws.numel() * ws.element_size()
    _call("wq_attn_kv4", dev, q.data_ptr(), q_step, Hq, None if cu_q is None else cu_q.data_ptr(), B, T, max_q,
          pages.data_ptr(), layout[1], block_table.data_ptr(), block_table.shape[1], kv_lens.data_ptr(),
          D ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(), out_step,
          None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), ws_bytes, stream)
    return out
