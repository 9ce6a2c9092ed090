"""wq_add_rms_norm, wq_add_rms_norm_fp8 and wq_quantize_fp8 against 64-bit references."""
import pytest
import torch

import fp8_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(T, H, dtype, add, seed=0, size=1.0):
    g = _gen(seed + T * 31 + H)
    t = ref.TYPES[dtype]
    x = (torch.randn(T, H, device="cuda", generator=g) * size).to(t)
    r = (torch.randn(T, H, device="cuda", generator=g) * 4 * size).to(t) if add else None
    w = (1 + 0.3 * torch.randn(H, device="cuda", generator=g)).to(t)
    return x, r, w


def _bound(y):
    # fp32: a row's sum of squares is at most 32 + 5 + 32 additions of positive numbers, halved by the root; the sum s,
    # the root, its argument and two products are a rounding or two each
    return 64 * ref.EPS32 * y.abs()


def _check16(out, total, x, r, w, eps, dtype):
    y, s = ref.norm(x.double(), None if r is None else r.double(), w.double(), eps)
    assert ((out.double() - y).abs() <= ref.to16(y, dtype) + _bound(y)).all()
    if r is None:
        assert total is None
    else:   # (fp32 first, then 16 bits)
        assert ((total.double() - s).abs() <= ref.to16(s, dtype) + ref.EPS32 * s.abs()).all()


SIZES = [(1, 8), (1, 4096), (3, 16), (7, 256), (5, 264), (33, 520), (64, 1024), (9, 2056), (130, 4096), (2, 5200), (17, 8192),
         (4, 11008), (3, 16384), (2, 20000), (2, 32768), (1000, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_norm(size, add, dtype):
    x, r, w = _inputs(*size, dtype, add)
    kept = [None if t is None else t.clone() for t in (x, r, w)]
    out, total = wq.wq_add_rms_norm(x, w, residual=r, eps=1e-5)
    _check16(out, total, x, r, w, 1e-5, dtype)
    for a, b in zip((x, r, w), kept):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("size", [s for s in SIZES if s[1] % 16 == 0] + [(40, 144), (5, 4016)])
def test_norm_8bit(size, add, dtype):
    x, r, w = _inputs(*size, dtype, add, seed=5)
    codes, scales, total = wq.wq_add_rms_norm_fp8(x, w, residual=r, eps=1e-5)
    y, s = ref.norm(x.double(), None if r is None else r.double(), w.double(), 1e-5)
    ref.check_pair(codes, scales, y, _bound(y))
    if add:
        assert torch.equal(total, wq.wq_add_rms_norm(x, w, residual=r, eps=1e-5)[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [(1, 16), (1, 4096), (15, 128), (16, 144), (17, 11008), (333, 4016), (2049, 1024), (100, 20000)])
def test_quantize(size, dtype):
    x, _, _ = _inputs(*size, dtype, False, seed=9)
    x[::3] *= 0.01
    codes, scales = wq.wq_quantize_fp8(x)
    ref.check_pair(codes, scales, x.double(), 0.0)


def test_strides_in_place_and_neighbours():
    """Rows inside wider rows; outputs over their own inputs; what lies around the outputs stays."""
    T, H = 37, 512
    wide = torch.randn(T, 3 * H, device="cuda").bfloat16()
    x, r = wide[:, H: 2 * H], wide[:, 2 * H:]
    w = torch.rand(H, device="cuda").bfloat16()
    want, total = wq.wq_add_rms_norm(x.contiguous(), w, residual=r.contiguous())
    pair = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    again = wq.wq_add_rms_norm_fp8(x.contiguous(), w, residual=r.contiguous())
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pair, again))
    plain = wq.wq_quantize_fp8(x)
    assert torch.equal(plain[0].view(torch.uint8), wq.wq_quantize_fp8(x.contiguous())[0].view(torch.uint8))
    left = wide[:, :H].clone()
    out, sum_out = wq.wq_add_rms_norm(x, w, residual=r, sum_out=r, out=x)
    assert out.data_ptr() == x.data_ptr() and sum_out.data_ptr() == r.data_ptr()
    assert torch.equal(wide[:, :H], left) and torch.equal(x, want) and torch.equal(r, total)


def test_outputs_end_where_they_end():
    T, H = 5, 400
    x, r, w = _inputs(T, H, "f16", True)
    codes, scales = torch.full((T + 2, H), 7, dtype=torch.uint8, device="cuda"), torch.full((6, T), -1.0, device="cuda")
    wq.wq_add_rms_norm_fp8(x, w, residual=r, codes=codes[1: 1 + T], scales=scales[1: 5])
    assert (codes[0] == 7).all() and (codes[-1] == 7).all() and (scales[0] == -1).all() and (scales[5] == -1).all()
    codes.fill_(7), scales.fill_(-1)
    wq.wq_quantize_fp8(x, codes=codes[1: 1 + T], scales=scales[1: 5])
    assert (codes[0] == 7).all() and (codes[-1] == 7).all() and (scales[0] == -1).all() and (scales[5] == -1).all()


def test_infinities_and_nan_stay_in_their_rows_and_blocks():
    T, H = 6, 512
    x, r, w = _inputs(T, H, "f16", True)
    clean = wq.wq_add_rms_norm(x, w, residual=r)
    clean8 = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    x[1, 300], r[2, 5], x[4, 0], r[4, 0] = NAN, INF, INF, -INF
    out, total = wq.wq_add_rms_norm(x, w, residual=r)
    for t in (0, 3, 5):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(total[t], clean[1][t])
    assert out[1].isnan().all() and out[4].isnan().all()
    # x / infinity is zero, infinity / infinity none
    assert out[2, 5].isnan() and (out[2, :5] == 0).all() and (out[2, 6:] == 0).all() and total[2, 5] == INF
    codes, scales, _ = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    for t in (0, 3, 5):
        assert torch.equal(codes[t].view(torch.uint8), clean8[0][t].view(torch.uint8)) and torch.equal(scales[:, t], clean8[1][:, t])
    assert scales[:, 1].isnan().all() and scales[:, 4].isnan().all() and (codes.view(torch.uint8)[1] == 0).all()
    assert scales[0, 2].isnan() and (scales[1:, 2] == 2.0 ** -96).all() and (codes.view(torch.uint8)[2] & 127 == 0).all()
    y = torch.ones(2, 400, device="cuda").half()
    y[0, 200], y[1, 399] = INF, NAN
    codes, scales = wq.wq_quantize_fp8(y)
    assert scales.isnan().tolist() == [[False, False], [True, False], [False, False], [False, True]]
    assert (codes.double()[0, :128] == 448).all() and (codes.view(torch.uint8)[0, 128: 256] == 0).all()


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 64, 2.0 ** -60, 2.0 ** -100, 3e37])
@pytest.mark.parametrize("H", [256, 4096])
def test_rows_whose_squares_leave_fp32(size, H):
    x, r, w = _inputs(5, H, "bf16", True, size=size / 8)
    for eps in (0.0, 1e-6):
        out, total = wq.wq_add_rms_norm(x, w, residual=r, eps=eps)
        y, s = ref.norm(x.double(), r.double(), w.double(), eps)
        assert ((out.double() - y).abs() <= ref.to16(y, "bf16") + 70 * ref.EPS32 * y.abs()).all()
        codes, scales, _ = wq.wq_add_rms_norm_fp8(x, w, residual=r, eps=eps)
        ref.check_pair(codes, scales, y, 70 * ref.EPS32 * y.abs())


def test_zeros_and_least_scale():
    x = torch.zeros(3, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda").bfloat16()
    out, _ = wq.wq_add_rms_norm(x, w)
    assert (out == 0).all()
    codes, scales, _ = wq.wq_add_rms_norm_fp8(x, w)
    assert (codes.view(torch.uint8) == 0).all() and (scales == 2.0 ** -96).all()
    x[1, 3] = 2.0 ** -100
    codes, scales = wq.wq_quantize_fp8(x)
    assert (scales == 2.0 ** -96).all() and codes.double()[1, 3] == 2.0 ** -4


def test_empty():
    w = torch.ones(256, device="cuda").half()
    x = torch.empty(0, 256, device="cuda").half()
    assert wq.wq_add_rms_norm(x, w, residual=x)[0].shape == (0, 256)
    codes, scales, total = wq.wq_add_rms_norm_fp8(x, w, residual=x)
    assert codes.shape == (0, 256) and scales.shape == (2, 0) and total.shape == (0, 256)
    assert wq.wq_quantize_fp8(x)[0].shape == (0, 256)


def test_side_stream_and_graph():
    x, r, w = _inputs(64, 4096, "bf16", True)
    want = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    x2 = x.clone()
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    after = wq.wq_add_rms_norm_fp8(x, w, residual=r)
    for a, b in ((want, got), (caught, after)):
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(caught, want))


def test_outputs_over_either_input():
    """sum over x and out over residual: every value is read before it is written, by the thread that writes it."""
    x, r, w = _inputs(50, 4096, "f16", True)
    want, total = wq.wq_add_rms_norm(x, w, residual=r)
    wq.wq_add_rms_norm(x, w, residual=r, sum_out=x, out=r)
    assert torch.equal(r, want) and torch.equal(x, total)


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows are those of a call of their own."""
    T, H, n = 530_000, 4096, 200
    x = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    tail, _, w = _inputs(n, H, "bf16", False)
    x[:-n].fill_(1.0)
    x[-n:] = tail
    out, _ = wq.wq_add_rms_norm(x, w)
    assert torch.equal(out[-n:], wq.wq_add_rms_norm(tail, w)[0]) and torch.equal(out[0], out[T - n - 1])
    del out
    for pair, own in ((wq.wq_quantize_fp8(x), wq.wq_quantize_fp8(tail)), (wq.wq_add_rms_norm_fp8(x, w), wq.wq_add_rms_norm_fp8(tail, w))):
        assert torch.equal(pair[0][-n:].view(torch.uint8), own[0].view(torch.uint8)) and torch.equal(pair[1][:, -n:], own[1])
