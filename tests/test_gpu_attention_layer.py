"""The example layer: projections, norm + rotation, 4-bit cache and attention together, against the same
steps in plain fp32 torch on the cache's read-back values."""
import importlib.util
import os

import pytest
import torch

import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(layer, cache, x, seq, position, lens):
    """The layer's output for tokens x, given the cache as it stands after they were written."""
    h, kv, d = layer.heads, layer.kv_heads, layer.head_dim

    def project(a, p):
        w, s, n, k = p
        return a.float() @ wq.wq_debug_dequant_int4(w, s, n, k, 128).T

    qkv = project(x, layer.qkv).to(x.dtype).float()
    q = qkv[:, : h * d].view(-1, h, d)
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * layer.q_weight.float()
    cs = layer.cos_sin[position][:, None]
    cos, sin, a, b = cs[..., : d // 2], cs[..., d // 2:], q[..., : d // 2], q[..., d // 2:]
    q = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype).float()
    out = torch.empty_like(q)
    for i in range(len(q)):
        t = torch.arange(int(position[i]) + 1, device=x.device)
        k, v = wq.wq_kv4_read(cache.pages, cache.slots(seq[i].expand_as(t), t), d, cache.group, cache.page_size, x.dtype)
        k, v = (y.float().repeat_interleave(h // kv, 1) for y in (k, v))
        p = (torch.einsum("hd,thd->ht", q[i], k) / d ** 0.5).softmax(-1)
        out[i] = torch.einsum("ht,thd->hd", p, v)
    return project(out.flatten(1).to(x.dtype), layer.out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_and_steps(ex, dtype):
    layer = ex.AttentionLayer(width=512, heads=8, kv_heads=2, head_dim=64, max_pos=256, dtype=dtype)
    seqs, n, steps = 3, 70, 3
    cache = ex.PagedCache(seqs, n + steps, 2, 64, group=32, page_size=16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(seqs, n, 512, device="cuda", generator=gen).to(dtype)
    xs = torch.randn(steps, seqs, 512, device="cuda", generator=gen).to(dtype)
    wq.wq_clear_device_status()
    first, rest = ex.prompt_and_steps(layer, x, xs, cache)
    assert wq.wq_device_status() == 0
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    seq = torch.arange(seqs, device="cuda")
    # Five roundings lie between the input and the output (projection, query, probabilities, attention, result), and
    # the tile kernels round the projection's operands: each of relative size u, on sums of independent terms.  In
    # norm over a row they stay within 8 u of it.
    for rows, pos, got in ((x[:, -1], n - 1, first[:, -1]), (x[:, 5], 5, first[:, 5]), (xs[-1], n + steps - 1, rest[-1])):
        want = _plain(layer, cache, rows, seq, torch.full((seqs,), pos, device="cuda"), None)
        err = (got.float() - want).norm(dim=-1) / want.norm(dim=-1)
        assert (err <= 8 * u).all(), err
