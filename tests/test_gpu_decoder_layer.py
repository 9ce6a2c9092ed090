"""The example decoder: norms, 8-bit projections, attention over the 4-bit cache and the gated block together, against
the same layers in plain fp32 torch without 8-bit activations, and step by step against the calls one by one."""
import importlib.util
import os

import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain(model, x):
    """x [seqs, n, width] -> the outputs in fp32: the weights' values, 16-bit keys and values, causal attention."""
    seqs, n, _ = x.shape
    pos = torch.arange(n, device=x.device)
    add, res = torch.zeros_like(x), x
    for v in model.layers:
        h, kv, d = v.heads, v.kv_heads, v.head_dim
        W = lambda w: ref.weight_values(*w).float()  # noqa: E731
        res = res + add
        qkv = _norm(res, v.attn_norm) @ W(v.qkv).T
        q, k, val = (t.unflatten(-1, (-1, d)) for t in qkv.split([h * d, kv * d, kv * d], -1))
        cs = v.cos_sin[pos][:, None]
        cos, sin = cs[..., : d // 2], cs[..., d // 2:]

        def turn(t, w):
            t = _norm(t, w)
            a, b = t[..., : d // 2], t[..., d // 2:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        q, k = turn(q, v.q_weight), turn(k, v.k_weight).repeat_interleave(h // kv, 2)
        s = torch.einsum("bnhd,bmhd->bhnm", q, k) / d ** 0.5
        s = s.masked_fill(pos[None, :] > pos[:, None], float("-inf"))
        o = torch.einsum("bhnm,bmhd->bnhd", s.softmax(-1), val.repeat_interleave(h // kv, 2))
        res = res + o.flatten(2) @ W(v.out).T
        y = _norm(res, v.ffn_norm)
        f = v.gate_up[0].shape[0] // 2
        gate, up = W((v.gate_up[0][:f], v.gate_up[1][0])), W((v.gate_up[0][f:], v.gate_up[1][1]))
        add = (torch.nn.functional.silu(y @ gate.T) * (y @ up.T)) @ W(v.down).T
    return _norm(res + add, model.norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_and_steps(ex, dtype):
    kv, d, seqs, n, steps = 2, 64, 3, 50, 4
    layers = [ex.DecoderLayer(width=512, heads=8, kv_heads=kv, head_dim=d, ffn=720, max_pos=256, dtype=dtype, seed=i)
              for i in range(2)]
    model = ex.Decoder(layers, [ex.PagedCache(seqs, n + steps, kv, d, group=32, page_size=16) for _ in layers])
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(seqs, n + steps, 512, device="cuda", generator=gen).to(dtype)
    wq.wq_clear_device_status()
    first, rest = ex.prompt_and_steps(model, x[:, :n], x[:, n:].transpose(0, 1).contiguous())
    assert wq.wq_device_status() == 0
    got = torch.cat([first, torch.stack(rest, 1)], 1).float()
    want = _plain(model, x.float())
    # What is summed over is rounded to 8 bits four times a layer and to 4 bits in the cache.  One rounding to e4m3 is
    # off by 2^-4 of the value at most, 2^-4 / 3^0.5 in the mean square, and a product's sum of independent terms by as
    # much; the cache's (a step is a fifteenth of 32 values' range of about 4 standard deviations, 4 / 15 / 12^0.5 =
    # 0.08) comes once a layer.  All of them in quadrature, as if each reached the output whole, for two layers:
    bound = (2 * (4 * (2 ** -4 / 3 ** 0.5) ** 2 + 0.08 ** 2)) ** 0.5
    off = (got - want).norm(dim=-1) / want.norm(dim=-1)
    assert off.mean() <= bound, (off.mean(), off.max(), bound)


def test_steps_in_a_graph(ex):
    """A decode step of a layer, captured once and replayed for token after token, gives the eager steps' bits."""
    kv, d, seqs, n, steps = 2, 64, 5, 30, 3
    layer = ex.DecoderLayer(width=512, heads=8, kv_heads=kv, head_dim=d, ffn=720, max_pos=256)
    make = lambda: ex.Decoder([layer], [ex.PagedCache(seqs, n + steps, kv, d, group=32, page_size=16)])  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(seqs, n, 512, device="cuda", generator=gen).bfloat16()
    xs = torch.randn(steps, seqs, 512, device="cuda", generator=gen).bfloat16()
    torch.manual_seed(3)
    a = make()
    _, want = ex.prompt_and_steps(a, x, xs)
    torch.manual_seed(3)
    b = make()
    ex.prompt_and_steps(b, x, xs[:0])
    seq, pos, token = torch.arange(seqs, device="cuda"), torch.full((seqs,), n, device="cuda"), xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = b(token, seq, pos)
    for i in range(steps):
        b.caches[0].lens.add_(1)
        pos.fill_(n + i)
        token.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
