"""8-bit activations to the bit: a block's scale is max|y| / 448 rounded once (at least 2^-96), a code the e4m3 number
nearest to the fp32 quotient y / scale (ties to the even code), whichever kernel makes it."""
import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu
BITS = {"bf16": 7, "f16": 10}


def _pair(y):
    """codes' bytes [T, K] and scales of fp32 values y [T, K], whole blocks: every step one IEEE operation (divisors are
    tensors: a number's reciprocal might be multiplied with instead)."""
    T, K = y.shape
    blocks = y.view(T, K // 128, 128)
    scale = torch.clamp(blocks.abs().amax(-1) / torch.full((), 448.0, device=y.device), min=ref.LEAST)
    codes = (blocks / scale.unsqueeze(-1)).clamp(-448, 448).view(T, K).to(ref.E4M3)
    return codes.view(torch.uint8), scale.t().contiguous()


def _same(codes, scales, y):
    want, want_scales = _pair(y)
    assert torch.equal(scales, want_scales)
    codes = codes.view(torch.uint8)
    off = codes != want
    assert not off.any(), (int(off.sum()), off.nonzero()[:4].tolist(), codes[off][:4].tolist(), want[off][:4].tolist())


def _all_quotients(dtype, exponent):
    """Blocks of 16-bit values, each one largest value and 127 others: every mantissa of the largest (a row each, times
    2^exponent) with every mantissa of the others, from the largest's own power of two down to where codes are zero."""
    n = 1 << BITS[dtype]
    mantissa = 1 + torch.arange(n, device="cuda", dtype=torch.float64) / n
    powers = torch.tensor([2.0 ** -i for i in range(21)], device="cuda", dtype=torch.float64)
    rest = (mantissa[None] * powers[:, None]).flatten()
    blocks = -(-rest.numel() // 127)
    others = torch.zeros(blocks * 127, device="cuda", dtype=torch.float64)
    others[: rest.numel()] = rest
    others[1::2] *= -1
    y = torch.zeros(n, blocks, 128, device="cuda", dtype=torch.float32)
    y[:, :, 0] = mantissa[:, None].float()
    y[:, :, 1:] = others.view(1, blocks, 127).float()
    y[:, :, 1:] *= y[:, :, 1:].abs() <= y[:, :, :1]
    return (y.view(n, -1).double() * 2.0 ** exponent).to(ref.TYPES[dtype])


@pytest.mark.parametrize("dtype,exponent", [("bf16", 0), ("bf16", 127), ("bf16", -86), ("bf16", -87), ("bf16", -95), ("f16", 0),
                                            ("f16", 15), ("f16", -8)])
def test_every_quotient_of_16_bit_values(dtype, exponent):
    x = _all_quotients(dtype, exponent)
    _same(*wq.wq_quantize_fp8(x), x.float())


def test_exact_ties():
    """Largest values whose scale is exact (49 / 448 = 7 / 64), others exactly in the middle between two codes."""
    for most in (49.0, 91.0, 105.0):
        scale = most / 448
        middles = torch.cat([(torch.arange(8, dtype=torch.float64) + 0.5) * 2.0 ** -9] +
                            [(8.5 + torch.arange(8, dtype=torch.float64)) * 2.0 ** (e - 3) for e in range(-6, 8)])
        for dtype in ("bf16", "f16"):
            y = (middles * scale).to(ref.TYPES[dtype])
            y = y[y.double() == middles * scale]          # those that 16 bits hold
            assert y.numel() >= 8
            x = torch.zeros(2, 128, dtype=ref.TYPES[dtype])
            x[:, 0] = most
            x[0, 1: 1 + y.numel()], x[1, 1: 1 + y.numel()] = y, -y
            codes, scales = wq.wq_quantize_fp8(x.cuda())
            assert (scales == scale).all()
            _same(codes, scales, x.cuda().float())
            assert (codes.view(torch.uint8)[:, 1: 1 + y.numel()] & 1 == 0).all()


def test_zeros_keep_their_sign():
    x = torch.zeros(2, 128, device="cuda").bfloat16()
    x[0, 1::2] = -0.0
    x[1, 0], x[1, 1::2] = 3.0, -0.0
    codes, scales = wq.wq_quantize_fp8(x)
    _same(codes, scales, x.float())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("H", [4096, 8192, 16384, 32768])
def test_norm_codes(H, add, dtype):
    """Rows whose mean square is 1 (no eps): the normed values are the weights, times the row's signs."""
    w = _all_quotients(dtype, 0)
    sign = torch.where(torch.rand(3, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(H)) < 0.5, -1.0, 1.0)
    x = (sign * (0.5 if add else 1.0)).to(ref.TYPES[dtype])
    for at in range(0, w.shape[0], 1 if dtype == "bf16" else 16):
        row = w[at].repeat(-(-H // w.shape[1]))[:H].contiguous()
        codes, scales, _ = wq.wq_add_rms_norm_fp8(x, row, residual=x if add else None, eps=0.0)
        _same(codes, scales, sign * row.float())


# (tokens, F) of each kernel: up to 16 tokens, up to 32, tiles of a block's own, of a pair
@pytest.mark.parametrize("M,F", [(3, 1024), (16, 256), (20, 1024), (32, 256), (70, 1024), (300, 256), (1600, 1664)])
def test_gated_codes(M, F):
    """A gate of 64 and above is its own silu (1 + exp(-64) is 1), whole numbers make every sum exact: the outputs are
    known to the bit, and with them scales and codes."""
    K = 128
    g = torch.Generator(device="cuda").manual_seed(M * 10007 + F)
    # up: 8-bit whole numbers times 2^-shift, from two e4m3 numbers of four bits each
    number = torch.randint(128, 256, (F,), device="cuda", generator=g)
    shift = torch.randint(1, 10, (F,), device="cuda", generator=g)
    shift[torch.arange(0, F, 128)] = 0
    number[torch.arange(0, F, 128)] = torch.tensor([196, 182, 210, 129, 255, 171, 128, 223], device="cuda").repeat(F)[: F // 128]
    step = torch.tensor([2.0 ** -i for i in range(10)], device="cuda", dtype=torch.float64)[shift]
    up = torch.zeros(F, K, device="cuda", dtype=torch.float64)
    up[:, 0], up[:, 1] = (number // 16 * 16) * step, (number % 16) * step
    assert torch.equal(up.to(ref.E4M3).double(), up)
    gate = torch.zeros(F, K, device="cuda", dtype=torch.float64)
    gate[:, 2] = 64
    w = torch.cat([gate, up]).to(ref.E4M3)
    sw = torch.ones(2, F // 128, 1, device="cuda")
    a = torch.zeros(M, K, device="cuda", dtype=torch.float64)
    a[:, :3] = torch.tensor([1.0, 1.0, 1.0], device="cuda", dtype=torch.float64)
    a[1::2, :2] *= -1
    token = torch.tensor([1.0, 2.0, 4.0], device="cuda", dtype=torch.float64)[torch.arange(M, device="cuda") % 3]
    y = 64 * token[:, None] * (a[:, :1] * token[:, None]) * (number * step)
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a.to(ref.E4M3), token.float()[None].contiguous(), w, sw)
    _same(codes, scales, y.float())
