"""A decoder layer whose projections take both operands in 8 bits, end to end:

    residual's addition + norm, to 8 bits            wq_add_rms_norm_fp8
    projection to queries, keys and values           wq_gemm_w8a8_fp8
    norms for each head + rotation by position       wq_qk_norm_rope   (in place)
    keys and values quantised into the paged cache   wq_kv4_write
    attention over the 4-bit cache                   wq_attn_kv4
    attention's output to 8 bits                     wq_quantize_fp8
    projection back                                  wq_gemm_w8a8_fp8
    residual's addition + norm, to 8 bits            wq_add_rms_norm_fp8
    silu(gate) * up, to 8 bits                       wq_gemm_w8a8_fp8_gated
    projection back                                  wq_gemm_w8a8_fp8

and, behind the last layer, the residual's addition + norm in 16 bits (wq_add_rms_norm).  Run some layers for a
prompt and some single-token steps of a batch (random weights):

    python examples/decoder_layer.py [--layers 4] [--seqs 4] [--prompt 1000] [--steps 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_tma_gb300 as wq  # noqa: E402
from attention_layer import PagedCache  # noqa: E402


def quantise_weight(w):
    """e4m3 codes [N, K] of a weight and a scale for each block of 128 x 128, fp32 [N / 128, K / 128] (offline, once)."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    full = torch.zeros(nb * 128, kb * 128, device=w.device)
    full[:n, :k] = w
    blocks = full.view(nb, 128, kb, 128)
    scale = (blocks.abs().amax((1, 3)) / 448).clamp(min=1e-30)
    codes = (blocks / scale.view(nb, 1, kb, 1)).clamp_(-448, 448).view(nb * 128, kb * 128)[:n, :k]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale


class DecoderLayer:
    def __init__(self, width=4096, heads=32, kv_heads=8, head_dim=128, ffn=11008, max_pos=65536, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.head_dim, self.dtype = width, heads, kv_heads, head_dim, dtype

        def weight(n, k):
            return quantise_weight(torch.randn(n, k, device=device, generator=gen) * k ** -0.5)

        def ones(n):
            return (1 + 0.1 * torch.randn(n, device=device, generator=gen)).to(dtype)

        self.qkv = weight((heads + 2 * kv_heads) * head_dim, width)
        self.out = weight(width, heads * head_dim)
        gate, up = weight(ffn, width), weight(ffn, width)
        self.gate_up = torch.cat([gate[0], up[0]]), torch.stack([gate[1], up[1]])
        self.down = weight(width, ffn)
        self.attn_norm, self.ffn_norm = ones(width), ones(width)
        self.q_weight, self.k_weight = ones(head_dim), ones(head_dim)
        angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] / 10000 ** (
            torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    def __call__(self, x, residual, cache, seq, position, cu_q=None, max_q=1):
        """x [T, width]: what the layer before adds to the residual stream [T, width] -> the same of this layer.

        The other arguments are AttentionLayer's (examples/attention_layer.py)."""
        h, kv, d, T = self.heads, self.kv_heads, self.head_dim, x.shape[0]
        codes, scales, residual = wq.wq_add_rms_norm_fp8(x, self.attn_norm, residual=residual)
        qkv = wq.wq_gemm_w8a8_fp8(codes, scales, *self.qkv, dtype=self.dtype)
        q, key = qkv[:, : h * d].view(T, h, d), qkv[:, h * d: (h + kv) * d].view(T, kv, d)
        value = qkv[:, (h + kv) * d:].view(T, kv, d)
        wq.wq_qk_norm_rope(q, key, position, self.cos_sin, self.q_weight, self.k_weight, q_out=q, k_out=key)
        wq.wq_kv4_write(key, value, cache.slots(seq, position), cache.pages, cache.group, cache.page_size)
        o = wq.wq_attn_kv4(q, cache.pages, cache.table, cache.lens, cache.group, cache.page_size, cu_q=cu_q, max_q=max_q)
        codes, scales = wq.wq_quantize_fp8(o.view(T, h * d))
        x = wq.wq_gemm_w8a8_fp8(codes, scales, *self.out, dtype=self.dtype)
        codes, scales, residual = wq.wq_add_rms_norm_fp8(x, self.ffn_norm, residual=residual)
        codes, scales = wq.wq_gemm_w8a8_fp8_gated(codes, scales, *self.gate_up)
        return wq.wq_gemm_w8a8_fp8(codes, scales, *self.down, dtype=self.dtype), residual


class Decoder:
    """Layers one behind the other, each with its own cache, and the last norm."""

    def __init__(self, layers, caches):
        self.layers, self.caches = layers, caches
        self.norm = torch.ones(layers[0].width, dtype=layers[0].dtype, device=layers[0].qkv[0].device)

    def __call__(self, x, seq, position, cu_q=None, max_q=1):
        add, residual = torch.zeros_like(x), x
        for layer, cache in zip(self.layers, self.caches):
            add, residual = layer(add, residual, cache, seq, position, cu_q=cu_q, max_q=max_q)
        return wq.wq_add_rms_norm(add, self.norm, residual=residual)[0]


def prompt_and_steps(model, x_prompt, x_steps):
    """The outputs of a prompt [seqs, prompt, width] and of single tokens [steps, seqs, width]."""
    seqs, n, width = x_prompt.shape
    dev = x_prompt.device
    seq = torch.arange(seqs, device=dev)
    for c in model.caches:
        c.lens.fill_(n)
    cu = torch.arange(seqs + 1, device=dev, dtype=torch.int32) * n
    first = model(x_prompt.reshape(seqs * n, width), seq.repeat_interleave(n), torch.arange(n, device=dev).repeat(seqs),
                  cu_q=cu, max_q=n)
    rest = []
    for i, x in enumerate(x_steps):
        for c in model.caches:
            c.lens.add_(1)
        rest.append(model(x, seq, torch.full((seqs,), n + i, device=dev)))
    return first.view(seqs, n, -1), rest


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--layers", type=int, default=4)
    a.add_argument("--seqs", type=int, default=4)
    a.add_argument("--prompt", type=int, default=1000)
    a.add_argument("--steps", type=int, default=32)
    a = a.parse_args()
    layers = [DecoderLayer(seed=i) for i in range(a.layers)]
    model = Decoder(layers, [PagedCache(a.seqs, a.prompt + a.steps, v.kv_heads, v.head_dim) for v in layers])
    x = torch.randn(a.seqs, a.prompt, layers[0].width, device="cuda").bfloat16()
    steps = torch.randn(a.steps, a.seqs, layers[0].width, device="cuda").bfloat16()
    prompt_and_steps(model, x, steps)
    torch.cuda.synchronize()
    t = time.perf_counter()
    first, rest = prompt_and_steps(model, x, steps)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.layers} layers, {a.seqs} sequences, prompt {a.prompt}, {a.steps} steps: {t * 1e3:.2f} ms; "
          f"finite {bool(torch.isfinite(first).all()) and all(bool(torch.isfinite(r).all()) for r in rest)}")


if __name__ == "__main__":
    main()
