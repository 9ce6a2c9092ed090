"""Host-side checks of the entry points around 8-bit projections, without a GPU: bad arguments refused before
anything touches the device, by the library and by its binding."""
import pytest
import torch

import weight_only_quantized_tma_gb300 as wq
from test_attn_binding_host import Stub, machine  # noqa: F401
from weight_only_quantized_tma_gb300 import _fp8

OK, NULL, SHAPE, GROUP, MISALIGNED, DTYPE = range(6)
P = 0x10000     # a 16-byte-aligned fake device address: validation never dereferences it


@pytest.fixture(scope="module")
def L():
    return wq.lib()


@pytest.mark.parametrize("quant", [False, True])
def test_norm_refusals(L, quant):
    def f(x=P, xs=256, r=P, rs=256, dt=0, T=4, H=256, w=P, eps=1e-6, s=P, ss=256, out=P, os_=256, codes=P, scales=P):
        if quant:
            return L.wq_add_rms_norm_fp8(x, xs, r, rs, dt, T, H, w, eps, s, ss, codes, scales, None)
        return L.wq_add_rms_norm(x, xs, r, rs, dt, T, H, w, eps, s, ss, out, os_, None)
    for kw in (dict(x=None), dict(w=None), dict(s=None), dict(codes=None) if quant else dict(out=None)):
        assert f(**kw) == NULL, kw
    if quant:
        assert f(scales=None) == NULL and f(H=24, xs=24, rs=24, ss=24) == SHAPE
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=252), dict(H=32784, xs=32784, rs=32784, ss=32784, os_=32784),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(xs=248), dict(xs=260), dict(rs=0),
               dict(ss=255)) + (() if quant else (dict(os_=252),)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2) == DTYPE
    for kw in (dict(x=P + 8), dict(r=P + 2), dict(w=P + 4), dict(s=P + 8)) + \
            ((dict(codes=P + 8), dict(scales=P + 2)) if quant else (dict(out=P + 8),)):
        assert f(**kw) == MISALIGNED, kw
    assert f(T=0, x=None, w=None) == OK


def test_quantize_refusals(L):
    def f(x=P, xs=256, dt=0, T=4, K=256, codes=P, scales=P):
        return L.wq_quantize_fp8(x, xs, dt, T, K, codes, scales, None)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None)):
        assert f(**kw) == NULL
    for kw in (dict(T=-1), dict(T=1 << 31), dict(K=0), dict(K=8), dict(K=264), dict(xs=128), dict(xs=260),
               dict(T=(1 << 31) - 1, K=1 << 20, xs=1 << 20)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=7) == DTYPE
    for kw in (dict(x=P + 8), dict(codes=P + 4), dict(scales=P + 2)):
        assert f(**kw) == MISALIGNED
    assert f(T=0, x=None) == OK


def test_product_refusals(L):
    def f(a=P, sa=P, w=P, sw=P, bias=None, M=4, N=256, K=256, dt=0, out=P):
        return L.wq_gemm_w8a8_fp8(a, sa, w, sw, bias, M, N, K, dt, out, None)
    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None)):
        assert f(**kw) == NULL
    for kw in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=4), dict(N=260), dict(N=(1 << 29) + 8), dict(K=0), dict(K=8),
               dict(K=264), dict(K=(1 << 30) + 16), dict(N=1 << 20, K=1 << 20), dict(M=1 << 30, N=1 << 16)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2) == DTYPE
    for kw in (dict(a=P + 8), dict(w=P + 8), dict(out=P + 8), dict(sa=P + 2), dict(sw=P + 1), dict(bias=P + 1)):
        assert f(**kw) == MISALIGNED
    assert f(M=0, a=None) == OK


def test_gated_refusals(L):
    def f(a=P, sa=P, w=P, sw=P, M=4, F=256, K=256, dt=0, out=None, codes=P, scales=P):
        return L.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, M, F, K, dt, out, codes, scales, None)
    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(codes=None), dict(scales=None), dict(out=P)):
        assert f(**kw) == NULL, kw
    for kw in (dict(M=-1), dict(F=0), dict(F=8), dict(F=264), dict(K=24)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2, out=P, codes=None, scales=None) == DTYPE
    for kw in (dict(codes=P + 8), dict(scales=P + 2), dict(out=P + 8, codes=None, scales=None), dict(w=P + 4)):
        assert f(**kw) == MISALIGNED
    assert f(M=0, a=None) == OK


H, E, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


def _calls(device):
    def t(shape, dtype=H):
        return Stub(shape, dtype, device)
    a, sa, w, sw = t((4, 256), E), t((2, 4), F32), t((512, 256), E), t((4, 2), F32)
    return {
        "wq_add_rms_norm": lambda: wq.wq_add_rms_norm(t((4, 256)), t((256,)), residual=t((4, 256)), sum_out=t((4, 256)),
                                                      out=t((4, 256))),
        "wq_add_rms_norm_fp8": lambda: wq.wq_add_rms_norm_fp8(t((4, 256)), t((256,)), codes=a, scales=sa),
        "wq_quantize_fp8": lambda: wq.wq_quantize_fp8(t((4, 256)), codes=a, scales=sa),
        "wq_gemm_w8a8_fp8": lambda: wq.wq_gemm_w8a8_fp8(a, sa, w, sw, out=t((4, 512))),
        "wq_gemm_w8a8_fp8_gated": lambda: wq.wq_gemm_w8a8_fp8_gated(a, sa, w, t((2, 2, 2), F32), codes=a, scales=sa),
    }


@pytest.mark.parametrize("name", sorted(_calls("cuda:0")))
@pytest.mark.parametrize("own", [0, 1, 3])
def test_the_library_runs_on_the_tensors_device(machine, monkeypatch, name, own):  # noqa: F811
    monkeypatch.setattr(_fp8, "_stream", lambda device: 40 + device.index)
    _calls(f"cuda:{own}")[name]()
    assert [c[:2] for c in machine.calls] == [(name, own)] and machine.calls[0][2][-1] == 40 + own
    assert machine.device == 0


def test_binding_refusals(machine, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_fp8, "_stream", lambda device: 40)

    def t(shape, dtype=H, device="cuda:0"):
        return Stub(shape, dtype, device)
    x, w = t((4, 256)), t((256,))
    a, sa, wt, sw = t((4, 256), E), t((2, 4), F32), t((512, 256), E), t((4, 2), F32)
    for call in (
        lambda: wq.wq_add_rms_norm(t((4, 2, 128)), w), lambda: wq.wq_add_rms_norm(t((4, 256), F32), t((256,), F32)),
        lambda: wq.wq_add_rms_norm(x, t((128,))), lambda: wq.wq_add_rms_norm(x, t((256,), torch.float16)),
        lambda: wq.wq_add_rms_norm(x, w, residual=t((3, 256))), lambda: wq.wq_add_rms_norm(x, w, residual=t((4, 256), torch.float16)),
        lambda: wq.wq_add_rms_norm(x, w, residual=t((4, 256), H, "cuda:1")), lambda: wq.wq_add_rms_norm(x, w, sum_out=x),
        lambda: wq.wq_add_rms_norm(x, w, out=t((4, 128))), lambda: wq.wq_add_rms_norm(x, w, residual=x, sum_out=t((4, 128))),
        lambda: wq.wq_add_rms_norm(torch.empty(4, 256, dtype=H), w),
        lambda: wq.wq_add_rms_norm_fp8(x, w, codes=t((4, 128), E), scales=sa), lambda: wq.wq_add_rms_norm_fp8(x, w, codes=a, scales=t((4, 2), F32)),
        lambda: wq.wq_quantize_fp8(t((4, 256), F32), codes=a, scales=sa), lambda: wq.wq_quantize_fp8(x, codes=t((4, 256), torch.int8), scales=sa),
        lambda: wq.wq_gemm_w8a8_fp8(a, t((4, 2), F32), wt, sw), lambda: wq.wq_gemm_w8a8_fp8(a, sa, t((512, 128), E), sw),
        lambda: wq.wq_gemm_w8a8_fp8(a, sa, wt, t((2, 4), F32)), lambda: wq.wq_gemm_w8a8_fp8(t((4, 256)), sa, wt, sw),
        lambda: wq.wq_gemm_w8a8_fp8(a, sa, wt, sw, dtype=F32), lambda: wq.wq_gemm_w8a8_fp8(a, sa, wt, sw, out=t((4, 256))),
        lambda: wq.wq_gemm_w8a8_fp8(a, sa, wt, sw, out=t((4, 512)), bias=t((512,), torch.float16)),
        lambda: wq.wq_gemm_w8a8_fp8(a, sa, t((512, 256), E, "cuda:1"), sw),
        lambda: wq.wq_gemm_w8a8_fp8_gated(a, sa, t((511, 256), E), sw), lambda: wq.wq_gemm_w8a8_fp8_gated(a, sa, wt, sw),
        lambda: wq.wq_gemm_w8a8_fp8_gated(a, sa, wt, t((2, 2, 2), F32), dtype=H, codes=a),
        lambda: wq.wq_gemm_w8a8_fp8_gated(a, sa, wt, t((2, 2, 2), F32), out=t((4, 512))),
    ):
        with pytest.raises(ValueError):
            call()
    assert not machine.calls


def test_one_buffer_for_sum_and_output_is_refused(L):
    def f(s, out, r=P):
        return L.wq_add_rms_norm(P, 256, r, 256, 0, 4, 256, P, 1e-6, s, 256, out, 256, None)
    Q = P + 0x10000
    assert f(Q, Q) == SHAPE and f(P, P) == SHAPE
    if not torch.cuda.is_available():      # (what is allowed gets as far as the device)
        assert f(P, Q) not in (SHAPE, NULL, MISALIGNED) and f(Q, P) not in (SHAPE, NULL, MISALIGNED)
