"""ctypes binding of the operators around 8-bit projections (include/wq.h): norm with the
residual's addition, quantiser of activations, block-scaled product, gated product.
Argument checks and marshalling only; the work is in libwq.so.

8-bit activations are a pair: codes float8_e4m3fn [T, K] and fp32 scales [ceil(K / 128), T].
"""
from __future__ import annotations

import torch

from ._attn import _DTYPES, _call, _flat, _stream

_E4M3 = torch.float8_e4m3fn
_F32 = torch.float32
_empty, _empty_like, _Tensor = torch.empty, torch.empty_like, torch.Tensor


# A decode step's calls are bound by the host, so a tensor's common form is tested in one expression and told apart
# only where that fails (a call of wq_add_rms_norm that makes its outputs: 13.6 us with a check for each property).

def _step(t, name, dtype, shape, device):
    """The elements from row to row of a [T, H] tensor (any stride) of this type, shape and device."""
    if not isinstance(t, _Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1]
    step, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the values of a token must be contiguous")
    return step if shape[0] > 1 else shape[1]


def _rows(x):
    """(elements from row to row, shape, type, its code, device) of 16-bit activations x [T, H]."""
    if not isinstance(x, _Tensor) or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    shape, dtype, dev = x.shape, x.dtype, x.device
    if len(shape) != 2:
        raise ValueError(f"x must be [tokens, values], got {tuple(shape)}")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"16-bit values must be float16 or bfloat16, got {dtype}")
    return shape[1] if x.is_contiguous() else _step(x, "x", dtype, shape, dev), shape, dtype, code, dev


def _type(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"16-bit values must be float16 or bfloat16, got {dtype}")
    return code


def _codes(t, name, device=None):
    """A contiguous e4m3 matrix (float8_e4m3fn, or its bytes as uint8)."""
    if not isinstance(t, _Tensor) or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a tensor on {device if device is not None else 'a CUDA device'}")
    if t.dtype is not _E4M3 and t.dtype is not torch.uint8:
        raise ValueError(f"{name} must have dtype float8_e4m3fn or uint8, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix")
    return shape


def _pair(codes, scales, T, K, device):
    """The two outputs of 8-bit activations, made where none are given."""
    blocks = -(-K // 128)
    if codes is None:
        codes = _empty((T, K), dtype=_E4M3, device=device)
    elif _codes(codes, "codes", device) != (T, K):
        raise ValueError(f"codes must have shape {(T, K)}, got {tuple(codes.shape)}")
    if scales is None:
        scales = _empty((blocks, T), dtype=_F32, device=device)
    else:
        _flat(scales, "scales", _F32, (blocks, T), device)
    return codes, scales


# ------------------------------------------------------------------ norm, quantiser

def _sum_of(residual, sum_out, x, shape, dtype, dev):
    """(residual's pointer, its step, the sum, the sum's pointer, its step)."""
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out without a residual: there is no sum")
        return None, 0, None, None, 0
    step = _step(residual, "residual", dtype, shape, dev)
    if sum_out is None:
        sum_out = _empty_like(x) if x.is_contiguous() else _empty(shape, dtype=dtype, device=dev)
        return residual.data_ptr(), step, sum_out, sum_out.data_ptr(), shape[1]
    s_step = _step(sum_out, "sum_out", dtype, shape, dev)
    return residual.data_ptr(), step, sum_out, sum_out.data_ptr(), s_step


def wq_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor = None, eps: float = 1e-6,
                    sum_out: torch.Tensor = None, out: torch.Tensor = None):
    """Norm of the rows of x + residual (x where there is none) [T, H] -> (out, sum; None without a residual).

    out = s * rsqrt(mean(s^2) + eps) * weight of the fp32 sum s; sum is s rounded, the new residual.  sum_out may
    be residual (or x), out may be x (or residual): in place."""
    x_step, shape, dtype, code, dev = _rows(x)
    T, H = shape
    _flat(weight, "weight", dtype, (H,), dev)
    r, r_step, total, s, s_step = _sum_of(residual, sum_out, x, shape, dtype, dev)
    if out is None:
        out, o_step = _empty_like(x) if x_step == H else _empty(shape, dtype=dtype, device=dev), H
    else:
        o_step = _step(out, "out", dtype, shape, dev)
    _call("wq_add_rms_norm", dev, x.data_ptr(), x_step, r, r_step, code, T, H, weight.data_ptr(), eps, s, s_step,
          out.data_ptr(), o_step, _stream(dev))
    return out, total


def wq_add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor = None, eps: float = 1e-6,
                        sum_out: torch.Tensor = None, codes: torch.Tensor = None, scales: torch.Tensor = None):
    """wq_add_rms_norm with its output in 8 bits -> (codes, scales, sum; None without a residual)."""
    x_step, shape, dtype, code, dev = _rows(x)
    T, H = shape
    _flat(weight, "weight", dtype, (H,), dev)
    r, r_step, total, s, s_step = _sum_of(residual, sum_out, x, shape, dtype, dev)
    codes, scales = _pair(codes, scales, T, H, dev)
    _call("wq_add_rms_norm_fp8", dev, x.data_ptr(), x_step, r, r_step, code, T, H, weight.data_ptr(), eps, s, s_step,
          codes.data_ptr(), scales.data_ptr(), _stream(dev))
    return codes, scales, total


def wq_quantize_fp8(x: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None):
    """16-bit activations x [T, K] -> (codes float8_e4m3fn [T, K], scales fp32 [ceil(K / 128), T])."""
    x_step, (T, K), _, code, dev = _rows(x)
    codes, scales = _pair(codes, scales, T, K, dev)
    _call("wq_quantize_fp8", dev, x.data_ptr(), x_step, code, T, K, codes.data_ptr(), scales.data_ptr(), _stream(dev))
    return codes, scales


# ------------------------------------------------------------------ products

def wq_gemm_w8a8_fp8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                     dtype: torch.dtype = torch.bfloat16, bias: torch.Tensor = None,
                     out: torch.Tensor = None) -> torch.Tensor:
    """out[M, N] = a . w^T (+ bias), both e4m3: a [M, K] with scales [ceil(K / 128), M], w [N, K] with scales
    [ceil(N / 128), ceil(K / 128)]; out in `dtype` (that of `out` where it is given)."""
    M, K = _codes(a, "a")
    dev = a.device
    N, K2 = _codes(w, "w", dev)
    if K2 != K:
        raise ValueError(f"w must be [N, {K}], got {(N, K2)}")
    blocks = -(-K // 128)
    _flat(a_scale, "a_scale", torch.float32, (blocks, M), dev)
    _flat(w_scale, "w_scale", torch.float32, (-(-N // 128), blocks), dev)
    if out is None:
        code = _type(dtype)
        out = torch.empty((M, N), dtype=dtype, device=dev)
    else:
        dtype = out.dtype if isinstance(out, torch.Tensor) else dtype
        code = _type(dtype)
        _flat(out, "out", dtype, (M, N), dev)
    if bias is not None:
        _flat(bias, "bias", dtype, (N,), dev)
    _call("wq_gemm_w8a8_fp8", dev, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
          None if bias is None else bias.data_ptr(), M, N, K, code, out.data_ptr(), _stream(dev))
    return out


def wq_gemm_w8a8_fp8_gated(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                           dtype: torch.dtype = None, codes: torch.Tensor = None, scales: torch.Tensor = None,
                           out: torch.Tensor = None):
    """silu(a . gate^T) * (a . up^T) -> (codes [M, F], scales [ceil(F / 128), M]); with dtype (or out) a 16-bit
    tensor [M, F] instead.

    w e4m3 [2 F, K]: the gate's rows, then those of up; w_scale fp32 [2, ceil(F / 128), ceil(K / 128)]."""
    M, K = _codes(a, "a")
    dev = a.device
    rows, K2 = _codes(w, "w", dev)
    F = rows // 2
    if K2 != K or rows % 2 != 0:
        raise ValueError(f"w must be [2 F, {K}], got {(rows, K2)}")
    blocks = -(-K // 128)
    _flat(a_scale, "a_scale", torch.float32, (blocks, M), dev)
    _flat(w_scale, "w_scale", torch.float32, (2, -(-F // 128), blocks), dev)
    if dtype is None and out is None:
        codes, scales = _pair(codes, scales, M, F, dev)
        _call("wq_gemm_w8a8_fp8_gated", dev, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), M, F, K,
              0, None, codes.data_ptr(), scales.data_ptr(), _stream(dev))
        return codes, scales
    if codes is not None or scales is not None:
        raise ValueError("either codes and scales, or a 16-bit output")
    if out is None:
        code = _type(dtype)
        out = torch.empty((M, F), dtype=dtype, device=dev)
    else:
        if isinstance(out, torch.Tensor) and dtype is None:
            dtype = out.dtype
        code = _type(dtype)
        _flat(out, "out", dtype, (M, F), dev)
    _call("wq_gemm_w8a8_fp8_gated", dev, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), M, F, K,
          code, out.data_ptr(), None, None, _stream(dev))
    return out
