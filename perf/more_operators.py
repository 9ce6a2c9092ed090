"""The operators around 8-bit projections of a decoder layer, as cases to time and compare.

Four operators that a decoder layer runs when its projections take both operands in 8 bits (e4m3):

* "norm"   root-mean-square norm with the residual's addition, its output in 16 bits (wq_add_rms_norm) or in 8
           bits with scales (wq_add_rms_norm_fp8);
* "quant"  16-bit activations, such as attention's output, to 8 bits with scales (wq_quantize_fp8);
* "gemm"   the product of 8-bit activations and 8-bit weights (wq_gemm_w8a8_fp8);
* "gated"  the first half of a gated feed-forward block: gate and up projection in one product, silu(gate) * up,
           its output in 8 bits with scales for the projection back (wq_gemm_w8a8_fp8_gated).

8-bit activations are codes [T][K] with a 32-bit scale for each token and block of 128 along K, scales [K / 128][T]:
scale = (largest magnitude of the block) / 448, at least 2^-96, and a code is the e4m3 number nearest to value / scale.
8-bit weights are codes [N][K] with a 32-bit scale for each block of 128 x 128, scales [N / 128][K / 128]; those of a
gated block have the gate's F rows first, then the F of up, scales [2][F / 128][K / 128].
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -96


# ---------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of 16 sequences of the 4096-wide layer: latency
        dict(name="norm_decode", kind="norm", dtype="bf16", T=16, H=4096, residual=True, quant=False),
        # a prompt before an 8-bit projection
        dict(name="norm_prompt_8bit", kind="norm", dtype="bf16", T=8192, H=4096, residual=True, quant=True),
        # the first norm of a stack (nothing to add yet), an odd number of tokens, rows that end inside a block
        dict(name="norm_first", kind="norm", dtype="f16", T=4999, H=5200, residual=False, quant=False),
        # attention's output of a serving batch of 64 sequences
        dict(name="quant_batch", kind="quant", dtype="bf16", T=64, K=4096),
        # the wide side of a feed-forward block, a whole prompt
        dict(name="quant_prompt", kind="quant", dtype="f16", T=8192, K=11008),
        # one new token through the packed projection of queries, keys and values
        dict(name="gemm_one", kind="gemm", dtype="bf16", M=1, N=12288, K=4096),
        # a serving batch through the projection back of the feed-forward block
        dict(name="gemm_batch", kind="gemm", dtype="f16", M=64, N=4096, K=11008),
        # a short prompt of an odd length
        dict(name="gemm_short", kind="gemm", dtype="bf16", M=333, N=4096, K=4096),
        # a long prompt through the packed projection
        dict(name="gemm_prompt", kind="gemm", dtype="bf16", M=8192, N=12288, K=4096),
        # a decode step of 16 sequences through the feed-forward block
        dict(name="gated_decode", kind="gated", M=16, F=11008, K=4096),
        # a chunk of a prompt, a width that ends inside a block
        dict(name="gated_chunk", kind="gated", M=777, F=6928, K=2560),
        # a long prompt
        dict(name="gated_prompt", kind="gated", M=4096, F=11008, K=4096),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "quant", "gemm", "gemm", "gated"])
    dtype = rng.choice(["bf16", "f16"])
    if kind in ("norm", "quant"):
        T, width = _spread(rng, 1, 16384), 16 * _spread(rng, 16, 704)
        T = max(1, min(T, 90_000_000 // width))
        if kind == "quant":
            return dict(kind=kind, dtype=dtype, T=T, K=width)
        return dict(kind=kind, dtype=dtype, T=T, H=width, residual=rng.random() < 0.7, quant=rng.random() < 0.5)
    # tokens from one to a long prompt; widths whole blocks mostly, some that end inside one
    M = _spread(rng, 1, 8192)
    K = rng.choice([128 * _spread(rng, 4, 96), 128 * _spread(rng, 4, 96), 16 * _spread(rng, 32, 704)])
    N = rng.choice([128 * _spread(rng, 4, 96), 128 * _spread(rng, 4, 96), 16 * _spread(rng, 32, 704)])
    M = max(1, min(M, 400_000_000_000 // (N * K)))
    if kind == "gemm":
        return dict(kind=kind, dtype=dtype, M=M, N=N, K=K)
    return dict(kind=kind, M=max(1, M // 2), F=N, K=K)


# ---------------------------------------------------------------------------------------- inputs

def _activations(gen, T, width):
    """A residual stream's values in 32 bits: a few strong channels, tokens of unequal size."""
    x = torch.randn(T, width, device="cuda", generator=gen)
    gain = torch.ones(width, device="cuda")
    gain[:: max(1, width // 6)] = 12.0
    size = torch.exp(0.3 * torch.randn(T, 1, device="cuda", generator=gen))
    return x.mul_(gain).mul_(size)


def _quantise(y):
    """codes and scales [blocks][T] of 32-bit values [T][K]; every step a 32-bit operation."""
    T, K = y.shape
    blocks = -(-K // 128)
    g = torch.zeros(T, blocks * 128, device=y.device)
    g[:, :K] = y
    g = g.view(T, blocks, 128)
    scale = torch.clamp(g.abs().amax(-1) / torch.full((), 448.0, device=y.device), min=LEAST)
    codes = (g / scale.unsqueeze(-1)).clamp_(-448, 448).view(T, -1)[:, :K].to(E4M3)
    return codes, scale.t().contiguous()


def _weight(gen, N, K):
    """codes [N][K] and scales [N / 128][K / 128] of a random weight whose blocks are of unequal size."""
    nb, kb = -(-N // 128), -(-K // 128)
    size = torch.exp(0.4 * torch.randn(nb, kb, device="cuda", generator=gen)) * K ** -0.5
    w = torch.zeros(nb * 128, kb * 128, device="cuda")
    w[:N, :K] = torch.randn(N, K, device="cuda", generator=gen)
    blocks = w.view(nb, 128, kb, 128).mul_(size.view(nb, 1, kb, 1))
    scale = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / scale.view(nb, 1, kb, 1)).clamp_(-448, 448).view(nb * 128, kb * 128)[:N, :K].to(E4M3)
    return codes.contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind = case["kind"]
    s = dict(case=case, kind=kind)
    if kind in ("norm", "quant"):
        dtype, T = TYPES[case["dtype"]], case["T"]
        if kind == "quant":
            s["x"] = _activations(gen, T, case["K"]).to(dtype)
            return s
        H = case["H"]
        s["x"] = torch.randn(T, H, device="cuda", generator=gen).mul_(0.7).to(dtype)
        s["residual"] = _activations(gen, T, H).to(dtype) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype)
        return s
    M, K = case["M"], case["K"]
    s["a"], s["a_scale"] = _quantise(_activations(gen, M, K))
    if kind == "gemm":
        s["w"], s["w_scale"] = _weight(gen, case["N"], K)
        return s
    gate, up = _weight(gen, case["F"], K), _weight(gen, case["F"], K)
    s["w"], s["w_scale"] = torch.cat([gate[0], up[0]]), torch.stack([gate[1], up[1]])
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _values(codes, scale):
    """The 32-bit values [T][K] of 8-bit activations."""
    return codes.float() * scale.t().repeat_interleave(128, 1)[:, : codes.shape[1]]


def _weight_values(codes, scale):
    """The 32-bit values [N][K] of an 8-bit weight."""
    N, K = codes.shape
    return codes.float() * scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _plain(s):
    c, kind = s["case"], s["kind"]
    if kind == "norm":
        x = s["x"].float()
        if s["residual"] is not None:
            x = x + s["residual"].float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
        out = {}
        if s["residual"] is not None:
            out["sum"] = x.to(s["x"].dtype)
        if c["quant"]:
            out["codes"], out["scales"] = _quantise(y)
        else:
            out["out"] = y.to(s["x"].dtype)
        return out
    if kind == "quant":
        codes, scales = _quantise(s["x"].float())
        return {"codes": codes, "scales": scales}
    a = _values(s["a"], s["a_scale"])
    if kind == "gemm":
        return {"out": (a @ _weight_values(s["w"], s["w_scale"]).t()).to(TYPES[c["dtype"]])}
    F = c["F"]
    gate = a @ _weight_values(s["w"][:F], s["w_scale"][0]).t()
    up = a @ _weight_values(s["w"][F:], s["w_scale"][1]).t()
    codes, scales = _quantise(gate / (1 + torch.exp(-gate)) * up)
    return {"codes": codes, "scales": scales}


def run(s):
    if not own:
        return _plain(s)
    import weight_only_quantized_tma_gb300 as wq
    c, kind = s["case"], s["kind"]
    if kind == "norm":
        if c["quant"]:
            codes, scales, total = wq.wq_add_rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=1e-6)
            out = {"codes": codes, "scales": scales}
        else:
            y, total = wq.wq_add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6)
            out = {"out": y}
        if s["residual"] is not None:
            out["sum"] = total
        return out
    if kind == "quant":
        codes, scales = wq.wq_quantize_fp8(s["x"])
    elif kind == "gemm":
        return {"out": wq.wq_gemm_w8a8_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], dtype=TYPES[c["dtype"]])}
    else:
        codes, scales = wq.wq_gemm_w8a8_fp8_gated(s["a"], s["a_scale"], s["w"], s["w_scale"])
    return {"codes": codes, "scales": scales}


# ---------------------------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    blocks = lambda n: -(-n // 128)  # noqa: E731
    if kind == "norm":
        T, H = case["T"], case["H"]
        rows = 3 if case["residual"] else 1   # x in; with a residual that in and the sum out
        out = T * H + 4 * T * blocks(H) if case["quant"] else 2 * T * H
        return {"bytes": 2 * rows * T * H + out + 2 * H, "flops": 5 * T * H}
    if kind == "quant":
        T, K = case["T"], case["K"]
        return {"bytes": 3 * T * K + 4 * T * blocks(K), "flops": 3 * T * K}
    M, K = case["M"], case["K"]
    N = case["N"] if kind == "gemm" else 2 * case["F"]
    out = 2 * M * N if kind == "gemm" else M * case["F"] + 4 * M * blocks(case["F"])
    return {"bytes": M * K + N * K + 4 * blocks(K) * (M + blocks(N)) + out, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------------------- in 64 bits

def _exact_blocks(y):
    """value / scale and the scales [blocks][T] of 64-bit values, block by block."""
    codes, scales = [], []
    for at in range(0, y.shape[1], 128):
        part = y[:, at: at + 128]
        scale = (part.abs().max(1).values / 448.0).clamp(min=LEAST)
        codes.append(part / scale[:, None])
        scales.append(scale)
    return {"codes": torch.cat(codes, 1), "scales": torch.stack(scales)}


def _exact_product(a, a_scale, w, w_scale):
    out = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device=a.device)
    A = torch.cat([a[:, 128 * k: 128 * k + 128].double() * a_scale[k].double()[:, None] for k in range(a_scale.shape[0])], 1)
    for n in range(w_scale.shape[0]):
        rows = w[128 * n: 128 * n + 128].double()
        across = torch.arange(rows.shape[1], device=w.device) // 128
        out[:, 128 * n: 128 * n + 128] = A @ (rows * w_scale[n].double()[across]).T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        y = x / ((x * x).sum(-1, keepdim=True) / x.shape[1] + 1e-6).sqrt() * s["weight"].double()
        out = _exact_blocks(y) if case["quant"] else {"out": y}
        if s["residual"] is not None:
            out["sum"] = x
        return out
    if kind == "quant":
        return _exact_blocks(s["x"].double())
    if kind == "gemm":
        return {"out": _exact_product(s["a"], s["a_scale"], s["w"], s["w_scale"])}
    F = case["F"]
    gate = _exact_product(s["a"], s["a_scale"], s["w"][:F], s["w_scale"][0])
    up = _exact_product(s["a"], s["a_scale"], s["w"][F:], s["w_scale"][1])
    return _exact_blocks(gate * torch.sigmoid(gate) * up)
