"""The attention half of a decoder layer on the library's operators, end to end:

    W4A16 projection to queries, keys and values      wq_gemm_w4a16
    norms for each head + rotation by position        wq_qk_norm_rope   (in place)
    keys and values quantised into the paged cache    wq_kv4_write
    attention over the 4-bit cache                    wq_attn_kv4
    W4A16 projection back                             wq_gemm_w4a16

Run it for a prompt and some single-token steps of a batch (random weights, the 4096-wide layer's shapes):

    python examples/attention_layer.py [--seqs 4] [--prompt 1000] [--steps 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_tma_gb300 as wq  # noqa: E402


class PagedCache:
    """Pages of the 4-bit cache and which of them each sequence holds."""

    def __init__(self, seqs, tokens, kv_heads, head_dim, group=128, page_size=64, device="cuda"):
        self.group, self.page_size = group, page_size
        each = -(-tokens // page_size)
        self.pages = wq.wq_kv4_pages(seqs * each, kv_heads, head_dim, group, page_size, device)
        # a server hands pages out as sequences grow; here each sequence owns its own from the start
        self.table = torch.randperm(seqs * each, device=device).to(torch.int32).view(seqs, each).contiguous()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=device)

    def slots(self, seq, position):
        """int64 slots of tokens (seq and position int64, one entry for each token)."""
        page = self.table[seq, position // self.page_size].long()
        return page * self.page_size + position % self.page_size


class AttentionLayer:
    """Projections in prepacked INT4, group 128; queries and keys normed for each head and rotated."""

    def __init__(self, width=4096, heads=32, kv_heads=8, head_dim=128, max_pos=65536, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.head_dim = width, heads, kv_heads, head_dim

        def projection(n, k):
            w = (torch.randn(n, k, device=device, generator=gen) * k ** -0.5).half()
            codes, scales = wq.wq_quantize_int4(w, 128)
            return wq.wq_pack_int4(codes, scales, n, k, 128) + (n, k)

        self.qkv = projection((heads + 2 * kv_heads) * head_dim, width)
        self.out = projection(width, heads * head_dim)
        self.q_weight = (1 + 0.1 * torch.randn(head_dim, device=device, generator=gen)).to(dtype)
        self.k_weight = (1 + 0.1 * torch.randn(head_dim, device=device, generator=gen)).to(dtype)
        angle = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] / 10000 ** (
            torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    def __call__(self, x, cache, seq, position, cu_q=None, max_q=1):
        """x [T, width]: the new tokens of every sequence, seq and position int64 [T]; cache.lens already
        counts them.  cu_q int32 [B + 1]: each sequence's rows of x (None: one each)."""
        h, kv, d, T = self.heads, self.kv_heads, self.head_dim, x.shape[0]
        w, s, n, k = self.qkv
        qkv = wq.wq_gemm_w4a16(x, w, s, n, k, 128)
        q, key = qkv[:, : h * d].view(T, h, d), qkv[:, h * d: (h + kv) * d].view(T, kv, d)
        value = qkv[:, (h + kv) * d:].view(T, kv, d)
        wq.wq_qk_norm_rope(q, key, position, self.cos_sin, self.q_weight, self.k_weight, q_out=q, k_out=key)
        wq.wq_kv4_write(key, value, cache.slots(seq, position), cache.pages, cache.group, cache.page_size)
        o = wq.wq_attn_kv4(q, cache.pages, cache.table, cache.lens, cache.group, cache.page_size, cu_q=cu_q, max_q=max_q)
        w, s, n, k = self.out
        return wq.wq_gemm_w4a16(o.view(T, h * d), w, s, n, k, 128)


def prompt_and_steps(layer, x_prompt, x_steps, cache):
    """The outputs of a prompt [seqs, prompt, width] and of single tokens [steps, seqs, width]."""
    seqs, n, width = x_prompt.shape
    dev = x_prompt.device
    seq = torch.arange(seqs, device=dev)
    cache.lens.fill_(n)
    cu = torch.arange(seqs + 1, device=dev, dtype=torch.int32) * n
    first = layer(x_prompt.reshape(seqs * n, width), cache, seq.repeat_interleave(n),
                  torch.arange(n, device=dev).repeat(seqs), cu_q=cu, max_q=n)
    rest = []
    for i, x in enumerate(x_steps):
        cache.lens.add_(1)
        rest.append(layer(x, cache, seq, torch.full((seqs,), n + i, device=dev)))
    return first.view(seqs, n, -1), rest


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--seqs", type=int, default=4)
    a.add_argument("--prompt", type=int, default=1000)
    a.add_argument("--steps", type=int, default=32)
    a = a.parse_args()
    layer = AttentionLayer()
    cache = PagedCache(a.seqs, a.prompt + a.steps, layer.kv_heads, layer.head_dim)
    x = torch.randn(a.seqs, a.prompt, layer.width, device="cuda").bfloat16()
    steps = torch.randn(a.steps, a.seqs, layer.width, device="cuda").bfloat16()
    prompt_and_steps(layer, x, steps, cache)
    torch.cuda.synchronize()
    t = time.perf_counter()
    first, rest = prompt_and_steps(layer, x, steps, cache)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    kv16 = 2 * a.seqs * (a.prompt + a.steps) * layer.kv_heads * layer.head_dim * 2
    print(f"{a.seqs} sequences, prompt {a.prompt}, {a.steps} steps: {t * 1e3:.2f} ms; "
          f"cache {cache.pages.numel() / 1e6:.1f} MB (16-bit: {kv16 / 1e6:.1f} MB); "
          f"finite {bool(torch.isfinite(first).all()) and all(bool(torch.isfinite(r).all()) for r in rest)}")


if __name__ == "__main__":
    main()
