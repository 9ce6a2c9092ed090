"""wq_add_rms_norm at the ends of fp32: rows of the least numbers without an eps, of the largest, eps of any size."""
import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu


def _check(x, r, w, eps):
    """Both outputs.  fp32: additions of positive numbers, halved by the root, and the roundings of the sum, the root,
    its argument and three products; what is subnormal on the way would show as far more."""
    y, _ = ref.norm(x.double(), None if r is None else r.double(), w.double(), eps)
    err = 70 * ref.EPS32 * y.abs()
    out, _ = wq.wq_add_rms_norm(x, w, residual=r, eps=eps)
    assert ((out.double() - y).abs() <= ref.to16(y, "bf16") + err).all()
    codes, scales, _ = wq.wq_add_rms_norm_fp8(x, w, residual=r, eps=eps)
    ref.check_pair(codes, scales, y, err)


@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("H", [16, 256, 4096, 8208, 16384, 32768])
@pytest.mark.parametrize("step", [2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -115])
def test_rows_of_least_numbers(step, H, add):
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randint(-9, 10, (4, H), device="cuda", generator=g).double()
    x[1] = 0
    x[1, 3] = 1          # one number alone: the root is its size over that of H
    x[2, 1:] = 0
    x[2, 0] = -7
    x = (x * step).bfloat16()
    r = (torch.randint(-9, 10, (4, H), device="cuda", generator=g).double() * step).bfloat16() if add else None
    if add:
        r[1:3] = 0
    w = (1 + 0.3 * torch.randn(H, device="cuda", generator=g)).bfloat16()
    assert (x != 0).any()
    _check(x, r, w, 0.0)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e30, 3e38, 3.4e38])
@pytest.mark.parametrize("size", [2.0 ** 127, 2.0 ** 126, 1.8e19, 1e19, 6e18, 1.0])
@pytest.mark.parametrize("H", [16, 4096, 32768])
def test_large_rows_and_any_eps(H, size, eps):
    g = torch.Generator(device="cuda").manual_seed(H)
    x = ((0.5 + 0.4 * torch.rand(3, H, device="cuda", generator=g).double()) * size).bfloat16()
    x[:, ::2] *= -1
    w = (1 + 0.3 * torch.randn(H, device="cuda", generator=g)).bfloat16()
    _check(x, None, w, eps)
    _check(x, (x * 0.0625).flip(0).contiguous(), w, eps)
