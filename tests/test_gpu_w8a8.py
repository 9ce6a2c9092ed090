"""wq_gemm_w8a8_fp8 and wq_gemm_w8a8_fp8_gated against products in 64 bits."""
import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _gen(*seed):
    return torch.Generator(device="cuda").manual_seed(sum(s * 1009 ** i for i, s in enumerate(seed)) % (1 << 31))


def _case(M, N, K, halves=1):
    g = _gen(M, N, K)
    a, sa = ref.random_pair(g, M, K)
    parts = [ref.random_weight(g, N, K) for _ in range(halves)]
    if halves == 1:
        return a, sa, parts[0][0], parts[0][1]
    return a, sa, torch.cat([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _check(out, want, err, dtype):
    off = (out.double() - want).abs()
    bound = ref.to16(want, dtype) + err * (1 + ref.HALF[dtype])
    assert (off <= bound).all(), f"{(off - bound).max()} past the bound at {(off > bound).nonzero()[:4].tolist()}"


# tokens: every tile and its ends; widths and depths that end inside a block, a row tile, a copy
TOKENS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 513, 1024, 2100]
SHAPES = [(8, 16), (128, 128), (136, 144), (256, 2048), (1024, 1040), (1000, 512), (4096, 4096), (520, 11008), (2304, 400)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", TOKENS)
def test_product(M, N, K):
    dtype = "bf16" if (M + N // 8) % 2 else "f16"
    a, sa, w, sw = _case(M, N, K)
    out = wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=ref.TYPES[dtype])
    _check(out, *ref.product(a, sa, w, sw), dtype)


@pytest.mark.parametrize("F,K", [(16, 16), (128, 256), (144, 400), (1024, 2048), (1392, 1040), (688, 4096), (2560, 528)])
@pytest.mark.parametrize("M", TOKENS)
def test_gated(M, F, K):
    a, sa, w, sw = _case(M, F, K, halves=2)
    want, err = ref.gated(a, sa, w, sw)
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw)
    ref.check_pair(codes, scales, want, err)
    dtype = "bf16" if M % 2 else "f16"
    _check(wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, dtype=ref.TYPES[dtype]), want, err, dtype)


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1024), (5000, 2056, 640), (20000, 384, 256), (3, 40000, 256), (2048, 12288, 512)])
def test_larger(M, N, K):
    a, sa, w, sw = _case(M, N, K)
    _check(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=torch.float16), *ref.product(a, sa, w, sw), "f16")


@pytest.mark.parametrize("M,F,K", [(3000, 2064, 640), (4096, 4096, 512)])
def test_larger_gated(M, F, K):
    a, sa, w, sw = _case(M, F, K, halves=2)
    ref.check_pair(*wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw), *ref.gated(a, sa, w, sw))


@pytest.mark.parametrize("M,N,K", [(6000, 4096, 128), (6000, 2056, 16), (4500, 4112, 272), (9000, 2064, 1168)])
def test_many_tiles_of_few_blocks(M, N, K):
    """Several tiles for each pair of thread blocks, of an odd or even number of blocks of K, down to one: scales and
    buffers of sums go on from tile to tile."""
    a, sa, w, sw = _case(M, N, K)
    _check(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=torch.float16), *ref.product(a, sa, w, sw), "f16")


@pytest.mark.parametrize("M,F,K", [(6000, 2064, 128), (5000, 2816, 304), (9000, 1040, 528)])
def test_many_gated_tiles_of_few_blocks(M, F, K):
    a, sa, w, sw = _case(M, F, K, halves=2)
    ref.check_pair(*wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw), *ref.gated(a, sa, w, sw))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [5, 100, 700])
def test_bias(M, dtype):
    N, K = 648, 512
    a, sa, w, sw = _case(M, N, K)
    bias = torch.randn(N, device="cuda", generator=_gen(M)).to(ref.TYPES[dtype])
    want, err = ref.product(a, sa, w, sw)
    want = want + bias.double()
    _check(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=ref.TYPES[dtype], bias=bias), want, err + ref.EPS32 * want.abs(), dtype)


@pytest.mark.parametrize("M", [1, 16, 100, 600])
def test_whole_numbers_are_exact(M):
    """Small whole numbers, scales that are powers of two: every sum is exact, so any order gives the same bits."""
    N, K = 384, 1536
    g = _gen(M)
    a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).float().to(ref.E4M3)
    w = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float().to(ref.E4M3)
    sa = 2.0 ** torch.randint(-2, 3, (12, M), device="cuda", generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (3, 12), device="cuda", generator=g).float()
    want = ref.product(a, sa, w, sw)[0]
    assert torch.equal(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=torch.bfloat16), want.to(torch.bfloat16))
    assert torch.equal(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=torch.float16), want.to(torch.float16))


@pytest.mark.parametrize("M", [4, 70, 520])
def test_nan_stays_in_its_token_and_column(M):
    N, K = 272, 640
    a, sa, w, sw = _case(M, N, K)
    clean = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    a.view(torch.uint8)[1, 500] = 0x7F
    sa[4, 3] = NAN
    w.view(torch.uint8)[200, 0] = 0xFF
    got = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1], bad[3], bad[:, 200] = True, True, True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("M", [4, 70, 520])
def test_nan_of_a_gated_block(M):
    F, K = 272, 640
    a, sa, w, sw = _case(M, F, K, halves=2)
    clean = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw)
    sa[0, 2] = NAN
    w.view(torch.uint8)[F + 130, 9] = 0x7F      # a row of up, in the second block of 128
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw)
    bad = torch.zeros(3, M, dtype=torch.bool, device="cuda")
    bad[:, 2], bad[1] = True, True
    assert torch.equal(scales.isnan(), bad) and torch.equal(scales[~bad], clean[1][~bad])
    wide = bad.t().repeat_interleave(128, 1)[:, :F]
    assert torch.equal(codes.view(torch.uint8)[~wide], clean[0].view(torch.uint8)[~wide])
    assert (codes.view(torch.uint8)[wide] == 0).all()


@pytest.mark.parametrize("M", [3, 50, 300, 800])
def test_outputs_end_where_they_end(M):
    N, K = 328, 256
    a, sa, w, sw = _case(M, N, K)
    room = torch.full((M + 2, N), 7.0, device="cuda").half()
    wq.wq_gemm_w8a8_fp8(a, sa, w, sw, out=room[1: 1 + M])
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    assert torch.equal(room[1: 1 + M], wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=torch.float16))
    F = 336
    a, sa, w, sw = _case(M, F, K, halves=2)
    codes, scales = torch.full((M + 2, F), 7, dtype=torch.uint8, device="cuda"), torch.full((5, M), -1.0, device="cuda")
    wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, codes=codes[1: 1 + M], scales=scales[1: 4])
    assert (codes[0] == 7).all() and (codes[-1] == 7).all() and (scales[0] == -1).all() and (scales[4] == -1).all()


def test_empty():
    a, sa, w, sw = _case(1, 256, 256)
    assert wq.wq_gemm_w8a8_fp8(a[:0], sa[:, :0].contiguous(), w, sw).shape == (0, 256)
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a[:0], sa[:, :0].contiguous(), w, sw.view(2, 1, 2))
    assert codes.shape == (0, 128) and scales.shape == (1, 0)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 1024, 8192), (64, 512, 4096), (200, 2048, 2048), (1500, 1024, 1024)])
def test_same_bits_every_time_on_any_stream_and_in_graphs(M, N, K):
    a, sa, w, sw = _case(M, N, K)
    pair = sw.view(2, -1, sw.shape[1]).contiguous()
    first, first8 = wq.wq_gemm_w8a8_fp8(a, sa, w, sw), wq.wq_gemm_w8a8_fp8_gated(a, sa, w, pair)
    sides = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught, caught8 = wq.wq_gemm_w8a8_fp8(a, sa, w, sw), wq.wq_gemm_w8a8_fp8_gated(a, sa, w, pair)
    for _ in range(10):
        got = []
        for s in sides:     # two calls at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append((wq.wq_gemm_w8a8_fp8(a, sa, w, sw), wq.wq_gemm_w8a8_fp8_gated(a, sa, w, pair)))
        graph.replay()
        torch.cuda.synchronize()
        got.append((caught, caught8))
        for out, pair8 in got:
            assert torch.equal(out, first)
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(pair8, first8))


def test_back_to_back():
    """A layer's chain without anything waited for: each kernel reads what the one before it wrote."""
    T, H, F = 48, 1024, 1536
    g = _gen(11)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    r = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    weight = torch.ones(H, device="cuda").bfloat16()
    up = [ref.random_weight(g, F, H) for _ in range(2)]
    up = torch.cat([p[0] for p in up]), torch.stack([p[1] for p in up])
    down = ref.random_weight(g, H, F)

    def chain(wait):
        y, total = x, r
        for _ in range(6):
            codes, scales, total = wq.wq_add_rms_norm_fp8(y, weight, residual=total)
            wait()
            codes, scales = wq.wq_gemm_w8a8_fp8_gated(codes, scales, *up)
            wait()
            y = wq.wq_gemm_w8a8_fp8(codes, scales, *down)
            wait()
            codes, scales = wq.wq_quantize_fp8(y)
            wait()
        return y, total, scales
    slow = chain(torch.cuda.synchronize)
    for _ in range(20):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), slow))


def test_offsets_past_32_bits():
    """More than 2^31 outputs: the last rows are those of a call of their own."""
    M, N, K, n = 70_000, 32_768, 128, 256    # (the own call's tokens start a tile as they do in the large one)
    g = _gen(5)
    w, sw = ref.random_weight(g, N, K)
    a = torch.ones(M, K, device="cuda").to(ref.E4M3)
    sa = torch.ones(1, M, device="cuda")
    first = M // 256 * 256 - n
    tail, ts = ref.random_pair(g, M - first, K)
    a.view(torch.uint8)[first:] = tail.view(torch.uint8)
    sa[:, first:] = ts
    out = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    _check(out[first:], *ref.product(tail, ts, w, sw), "bf16")
    assert torch.equal(out[0], out[first - 1])
    del out
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, torch.cat([w, w]), torch.stack([sw, sw]))
    ref.check_pair(codes[first:].contiguous(), scales[:, first:].contiguous(), *ref.gated(tail, ts, torch.cat([w, w]), torch.stack([sw, sw])))


@pytest.mark.parametrize("M", [3, 40, 900])
def test_first_call_of_a_process_in_a_capture(M):
    """What the library asks of the device once is asked outside the stream: a first call may be a captured one."""
    import subprocess
    import sys
    code = f"""
import torch, weight_only_quantized_tma_gb300 as wq
E = torch.float8_e4m3fn
a, w = torch.ones({M}, 256, device="cuda").to(E), torch.ones(512, 256, device="cuda").to(E)
sa, sw = torch.ones(2, {M}, device="cuda"), torch.ones(4, 2, device="cuda")
x = torch.ones({M}, 256, device="cuda").half()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw.view(2, 2, 2))
    y, _ = wq.wq_add_rms_norm(x, x[0].clone())
    q, s = wq.wq_quantize_fp8(x)
g.replay()
torch.cuda.synchronize()
assert (out == 256).all() and (codes.double() == 448).all() and (scales == 65536 / 448).all()
assert (y == 1).all() and (q.double() == 448).all() and wq.wq_device_status() == 0
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("M", [7, 48, 600])
def test_padded_tokens_change_nothing(M):
    """Tokens are independent: those of a batch padded with rubbish get the bits that they get alone."""
    N, K = 512, 1024
    a, sa, w, sw = _case(M, N, K)
    alone = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[M // 2:] = 0x7F
    sa2[:, M // 2:] = NAN
    assert torch.equal(wq.wq_gemm_w8a8_fp8(a2, sa2, w, sw)[: M // 2], alone[: M // 2])
