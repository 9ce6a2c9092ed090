"""wq_gemm_w8a8_fp8_gated where exp(-gate) comes near the end of fp32: silu(gate) is as small as 2^-121 there, and an up of
2^100 and more still makes an ordinary number of it."""
import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu
GATES = [-60.0, -80.0, -84.0, -87.0, -87.5, -88.0, -88.25, -88.5]


# (tokens, F) of each kernel: up to 16 tokens, up to 32, tiles of a block's own, of a pair
@pytest.mark.parametrize("M,F", [(3, 256), (32, 256), (70, 256), (1600, 1664)])
def test_silu_far_below_zero(M, F):
    K = 128
    gate = torch.tensor(GATES, device="cuda", dtype=torch.float64).repeat(F)[:F]
    gate[128:] = gate[128:].clamp(max=-87.0)          # (a block of small numbers alone: their codes are not zero)
    parts = torch.zeros(2, F, K, device="cuda", dtype=torch.float64)
    parts[0, :, 0] = torch.trunc(gate / 8) * 8        # a multiple of 8 and the rest: two e4m3 numbers
    parts[0, :, 1] = gate - parts[0, :, 0]
    parts[1, :, 0] = 1
    assert torch.equal(parts.to(ref.E4M3).double(), parts)
    a = torch.zeros(M, K, device="cuda", dtype=torch.float64)
    a[:, :2] = 1
    sw = torch.ones(2, F // 128, 1, device="cuda")
    sw[1] = 2.0 ** 108
    args = a.to(ref.E4M3), torch.ones(1, M, device="cuda"), parts.view(2 * F, K).to(ref.E4M3), sw
    h = (gate / (1 + torch.exp(-gate)) * 2.0 ** 108).expand(M, F)
    # the exponential's argument, up to 128, is off by a rounding of its own and one of log2 e, 2^-17 each at most, so the
    # exponential by 2^-17 of itself and 2^-22 of its own; a few roundings more
    err = h.abs() * 2.0 ** -16
    out = wq.wq_gemm_w8a8_fp8_gated(*args, dtype=torch.bfloat16)
    assert ((out.double() - h).abs() <= ref.to16(h, "bf16") + err).all()
    ref.check_pair(*wq.wq_gemm_w8a8_fp8_gated(*args), h, err)
