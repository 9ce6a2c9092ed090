"""The GEMMs' binding refuses tensors of a device that is not the current one (host only: stand-ins for
tensors, devices and the library)."""
import pytest
import torch

import weight_only_quantized_tma_gb300 as wq
from test_attn_binding_host import Stub, machine  # noqa: F401

H, U8, F32 = torch.float16, torch.uint8, torch.float32
N, K, G, M = 128, 256, 64, 4


def _calls(device):
    def t(shape, dtype):
        return Stub(shape, dtype, device)
    A, out, ws = t((M, K), H), t((M, N), H), t((1 << 20,), U8)
    bf, bf_out = t((M, K), torch.bfloat16), t((M, N), torch.bfloat16)
    w, s = t((N * K // 2,), U8), t((N * K // G,), H)
    return {
        "wq_gemm_w4a16": lambda: wq.wq_gemm_w4a16(A, w, s, N, K, G, out=out, ws=ws),
        "wq_gemm_w4a16_zp": lambda: wq.wq_gemm_w4a16_zp(A, w, s, t((K,), U8), N, K, G, out=out, ws=ws),
        "wq_gemm_w4a16_lut": lambda: wq.wq_gemm_w4a16_lut(A, w, s, t((16,), H), N, K, G, out=out, ws=ws),
        "wq_gemm_w4a16_noalloc": lambda: wq.wq_gemm_w4a16_noalloc(A, w, s, N, K, G, out=out),
        "wq_gemm_w2a16": lambda: wq.wq_gemm_w2a16(A, t((N, K // 4), U8), s, N, K, G, out=out, ws=ws),
        "wq_gemm_w8a16_fp8": lambda: wq.wq_gemm_w8a16_fp8(A, t((N, K), U8), t((1,), F32), out=out, ws=ws),
        "wq_gemm_bf16_fp4": lambda: wq.wq_gemm_bf16_fp4(bf, t((N, K // 2), U8), t((N * K // 16,), U8), t((1,), F32),
                                                        out=bf_out, ws=ws),
    }


@pytest.mark.parametrize("name", sorted(_calls("cuda:0")))
def test_tensors_of_another_device_are_refused(machine, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 7}))
    with pytest.raises(ValueError, match="current"):
        _calls("cuda:1")[name]()
    assert name not in [c[0] for c in machine.calls]
    _calls("cuda:0")[name]()
    assert machine.calls[-1][0] == name and machine.calls[-1][1] == 0
    with torch.cuda.device(1):
        _calls("cuda:1")[name]()
    assert machine.calls[-1][0] == name and machine.calls[-1][1] == 1
