"""64-bit references of the operators around 8-bit projections, and bounds on what fp32 kernels may be off by.
torch in float64, where the tensors lie."""
import torch

E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -96
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # what one rounding may be off by at most, relative to the value
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS32 = 2.0 ** -24


def norm(x, residual, weight, eps):
    """(y, s) of float64 tensors."""
    s = x if residual is None else x + residual
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * weight, s


def blocks_most(y):
    """[blocks, T]: largest magnitude of each block of 128 of y [T, K]."""
    return torch.stack([p.abs().amax(1) for p in y.split(128, 1)])


def check_pair(codes, scales, y, err):
    """8-bit activations against float64 values y [T, K], which the kernel held in fp32 to within err (a tensor like y, or
    a number): a scale is the block's largest over 448 (at least 2^-96) to within that and three roundings, and a code is
    nearest to the value over the scale: within half a step (2^-4 of the value, 2^-10 below the least normal 2^-6),
    where the value itself is off by err and the quotient by three roundings."""
    T, K = y.shape
    err = torch.as_tensor(err, dtype=torch.float64, device=y.device).expand(y.shape)
    assert codes.dtype is E4M3 and codes.shape == (T, K)
    assert scales.dtype is torch.float32 and scales.shape == (-(-K // 128), T)
    most = blocks_most(y)
    want = (most / 448).clamp(min=LEAST)
    s = scales.double()
    off = blocks_most(err) / 448 + 4 * EPS32 * want
    assert ((s - want).abs() <= off).all(), ((s - want).abs() / want).max()
    wide = s.t().repeat_interleave(128, 1)[:, :K]
    value = codes.double() * wide
    bound = 2.0 ** -4 * y.abs() + 2.0 ** -10 * wide + 1.1 * err + 4 * EPS32 * y.abs()
    # at the top: codes end at 448, and a value past 448 scales is past it by what the scale is off by
    assert ((value - y).abs() <= bound).all(), ((value - y).abs() - bound).max()


def values(codes, scales):
    """float64 values of 8-bit activations."""
    return codes.double() * scales.double().t().repeat_interleave(128, 1)[:, : codes.shape[1]]


def weight_values(codes, scales):
    N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def product(a, a_scale, w, w_scale):
    """(out, err) in float64: err bounds what fp32 sums may be off by.  A block's 128 products are exact, their sum is
    128 additions off by 2^-23 of the partial sums at most (the tensor cores may cut where others round); the blocks'
    sums are scaled (two products) and added with one rounding each."""
    A, W = values(a, a_scale), weight_values(w, w_scale)
    blocks = -(-a.shape[1] // 128)
    return A @ W.t(), (A.abs() @ W.abs().t()) * (128 * 2.0 ** -23 + (blocks + 4) * EPS32)


def gated(a, a_scale, w, w_scale):
    """(h, err): |silu'| is below 1.1, |silu(g)| at most |g|; silu and the product are off by 16 roundings at most
    (an exponential to 2^-21, a division to 2^-22, two products)."""
    F = w.shape[0] // 2
    g, eg = product(a, a_scale, w[:F], w_scale[0])
    u, eu = product(a, a_scale, w[F:], w_scale[1])
    silu = g * torch.sigmoid(g)
    h = silu * u
    # (the exponential's relative error grows with |g| where exp(-g) matters: 2^-23 |g| from rounding -g log2 e)
    return h, 1.1 * eg * u.abs() + (silu.abs() + 1.1 * eg) * eu + h.abs() * (16 + 2 * g.abs()) * EPS32 + 1e-37


def random_pair(gen, T, K, device="cuda"):
    """8-bit activations with blocks of very unequal scales."""
    codes = (torch.randn(T, K, device=device, generator=gen) * 60).clamp(-448, 448).to(E4M3)
    scales = torch.exp(torch.randn(-(-K // 128), T, device=device, generator=gen))
    return codes, scales * 0.01


def random_weight(gen, N, K, device="cuda"):
    codes = (torch.randn(N, K, device=device, generator=gen) * 60).clamp(-448, 448).to(E4M3)
    scales = torch.exp(0.5 * torch.randn(-(-N // 128), -(-K // 128), device=device, generator=gen))
    return codes, scales * 0.01 / K ** 0.5


def to16(want, dtype):
    """How far one rounding to dtype may take float64 values (fp16 below 2^-14 keeps steps of 2^-24)."""
    return HALF[dtype] * want.abs() + (2.0 ** -25 if dtype == "f16" else 1e-39)
