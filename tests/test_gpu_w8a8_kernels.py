"""wq_gemm_w8a8_fp8 and wq_gemm_w8a8_fp8_gated: bias, NaN, ends of outputs, padding, repeats and captures at sizes that
each of the four kernels takes: up to 16 tokens, up to 32, tiles of 128 tokens of a block's own, tiles of 256 of a pair.
(The pair's: more tiles of a block's own than there are SMs, so that those would take a second round.)"""
import os
import subprocess
import sys

import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq
from test_gpu_w8a8 import _case, _check

pytestmark = pytest.mark.gpu
NAN = float("nan")
K = 640
PRODUCT = [(4, 264), (16, 264), (17, 264), (20, 2056), (32, 264), (70, 264), (1600, 2056), (2048, 2304)]
GATED = [(4, 272), (16, 272), (17, 272), (20, 2064), (32, 272), (70, 272), (1600, 1552), (2048, 1664)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", PRODUCT)
def test_bias(M, N, dtype):
    a, sa, w, sw = _case(M, N, K)
    bias = torch.randn(N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(M)).to(ref.TYPES[dtype])
    want, err = ref.product(a, sa, w, sw)
    want = want + bias.double()
    _check(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=ref.TYPES[dtype], bias=bias), want, err + ref.EPS32 * want.abs(), dtype)


@pytest.mark.parametrize("M,N", PRODUCT)
def test_whole_numbers_are_exact(M, N):
    """Small whole numbers, scales that are powers of two, a bias of whole numbers: every sum is exact."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).float().to(ref.E4M3)
    w = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float().to(ref.E4M3)
    sa = 2.0 ** torch.randint(-2, 3, (K // 128, M), device="cuda", generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (-(-N // 128), K // 128), device="cuda", generator=g).float()
    bias = torch.randint(-64, 65, (N,), device="cuda", generator=g).float()
    want = ref.product(a, sa, w, sw)[0] + bias.double()
    for t in ref.TYPES.values():
        assert torch.equal(wq.wq_gemm_w8a8_fp8(a, sa, w, sw, dtype=t, bias=bias.to(t)), want.to(t))


@pytest.mark.parametrize("M,N", PRODUCT)
def test_nan_stays_in_its_token_and_column(M, N):
    a, sa, w, sw = _case(M, N, K)
    clean = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    a.view(torch.uint8)[1, 500] = 0x7F
    sa[4, M - 1] = NAN
    w.view(torch.uint8)[N - 3, 0] = 0xFF
    got = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1], bad[M - 1], bad[:, N - 3] = True, True, True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("M,F", GATED)
def test_nan_of_a_gated_block(M, F):
    a, sa, w, sw = _case(M, F, K, halves=2)
    clean = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw)
    plain = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, dtype=torch.float16)
    sa[0, M - 1] = NAN
    w.view(torch.uint8)[F + 130, 9] = 0x7F      # a row of up, in the second block of 128
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw)
    bad = torch.zeros(-(-F // 128), M, dtype=torch.bool, device="cuda")
    bad[:, M - 1], bad[1] = True, True
    assert torch.equal(scales.isnan(), bad) and torch.equal(scales[~bad], clean[1][~bad])
    wide = bad.t().repeat_interleave(128, 1)[:, :F]
    assert torch.equal(codes.view(torch.uint8)[~wide], clean[0].view(torch.uint8)[~wide])
    assert (codes.view(torch.uint8)[wide] == 0).all()
    got = wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, dtype=torch.float16)
    one = torch.zeros(M, F, dtype=torch.bool, device="cuda")
    one[M - 1], one[:, 130] = True, True
    assert torch.equal(got.isnan(), one) and torch.equal(got[~one], plain[~one])


@pytest.mark.parametrize("i", range(len(PRODUCT)))
def test_outputs_end_where_they_end(i):
    M, N = PRODUCT[i]
    a, sa, w, sw = _case(M, N, K)
    room = torch.full((M + 2, N), 7.0, device="cuda").half()
    wq.wq_gemm_w8a8_fp8(a, sa, w, sw, out=room[1: 1 + M])
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    _check(room[1: 1 + M], *ref.product(a, sa, w, sw), "f16")
    M, F = GATED[i]
    a, sa, w, sw = _case(M, F, K, halves=2)
    blocks = -(-F // 128)
    codes, scales = torch.full((M + 2, F), 7, dtype=torch.uint8, device="cuda"), torch.full((blocks + 2, M), -1.0, device="cuda")
    wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, codes=codes[1: 1 + M], scales=scales[1: 1 + blocks])
    assert (codes[0] == 7).all() and (codes[-1] == 7).all() and (scales[0] == -1).all() and (scales[-1] == -1).all()
    room = torch.full((M + 2, F), 7.0, device="cuda").bfloat16()
    wq.wq_gemm_w8a8_fp8_gated(a, sa, w, sw, out=room[1: 1 + M])
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    want, err = ref.gated(a, sa, w, sw)
    _check(room[1: 1 + M], want, err, "bf16")
    ref.check_pair(codes[1: 1 + M].view(ref.E4M3), scales[1: 1 + blocks], want, err)


@pytest.mark.parametrize("i", range(len(PRODUCT)))
def test_padded_tokens_change_nothing(i):
    """Tokens are independent: those of a batch padded with rubbish get the bits that they get with others there."""
    for halves, (M, N) in ((1, PRODUCT[i]), (2, GATED[i])):
        a, sa, w, sw = _case(M, N, K, halves=halves)
        run = wq.wq_gemm_w8a8_fp8 if halves == 1 else lambda *t: wq.wq_gemm_w8a8_fp8_gated(*t, dtype=torch.bfloat16)
        alone = run(a, sa, w, sw)
        a.view(torch.uint8)[M // 2:] = 0x7F
        sa[:, M // 2:] = NAN
        assert torch.equal(run(a, sa, w, sw)[: M // 2], alone[: M // 2])


@pytest.mark.parametrize("i", range(len(PRODUCT)))
def test_same_bits_every_time_on_any_stream_and_in_graphs(i):
    (M, N), (_, F) = PRODUCT[i], GATED[i]
    a, sa, w, sw = _case(M, N, K)
    _, _, w2, sw2 = _case(M, F, K, halves=2)

    def both():
        return (wq.wq_gemm_w8a8_fp8(a, sa, w, sw),) + tuple(t.view(torch.uint8) for t in wq.wq_gemm_w8a8_fp8_gated(a, sa, w2, sw2))
    first = both()
    sides = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = both()
    for _ in range(10):
        got = []
        for s in sides:     # two calls at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(both())
        graph.replay()
        torch.cuda.synchronize()
        for g in got + [caught]:
            assert all(torch.equal(p, q) for p, q in zip(g, first))
    assert wq.wq_device_status() == 0


@pytest.mark.parametrize("i", [2, 4, 6])
def test_first_call_of_a_process_in_a_capture(i):
    (M, N), (_, F) = PRODUCT[i], GATED[i]
    code = f"""
import torch, weight_only_quantized_tma_gb300 as wq
E = torch.float8_e4m3fn
a, w, w2 = (torch.ones(n, 256, device="cuda").to(E) for n in ({M}, {N}, 2 * {F}))
sa, sw, sw2 = torch.ones(2, {M}, device="cuda"), torch.ones(-(-{N} // 128), 2, device="cuda"), torch.ones(2, -(-{F} // 128), 2, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = wq.wq_gemm_w8a8_fp8(a, sa, w, sw)
    codes, scales = wq.wq_gemm_w8a8_fp8_gated(a, sa, w2, sw2)
g.replay()
torch.cuda.synchronize()
assert (out == 256).all() and (codes.double() == 448).all() and (scales == 65536 / 448).all() and wq.wq_device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
