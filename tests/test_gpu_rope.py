"""wq_qk_norm_rope against a 64-bit reference, and what it refuses."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu


def _table(rng, most, rot):
    ang = rng.uniform(-200, 200, (most, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _bound(want, x, dtype):
    # one rounding of the result; fp32: a square root and a few products and sums of values no larger than the
    # row's largest (64 steps of 2^-24 are generous); fp16 results below 2^-14 keep steps of 2^-24
    top = np.abs(want).max(-1, keepdims=True)
    return ref.unit(dtype) * np.abs(want) + 64 * 2.0 ** -24 * top + 2.0 ** -25


CASES = [  # T, Hq, Hkv, D, rot
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 5, 1, 64, 32), (33, 14, 2, 128, 64), (130, 3, 3, 96, 96),
    (5, 2, 2, 80, 16), (9, 4, 2, 256, 128), (3, 2, 1, 256, 256), (17, 6, 6, 8, 8), (64, 32, 32, 128, 128),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", ["both", "q", "none"])
@pytest.mark.parametrize("case", CASES)
def test_matches_reference(case, weights, interleaved, dtype):
    T, Hq, Hkv, D, rot = case
    rng = np.random.default_rng(T * 1000 + D + rot)
    # a packed projection: q, k, v of a token in one row
    qkv = ref.random16(rng, (T, (Hq + 2 * Hkv) * D), dtype, 2.0)
    q, k = qkv[:, : Hq * D].reshape(T, Hq, D), qkv[:, Hq * D: (Hq + Hkv) * D].reshape(T, Hkv, D)
    cs = _table(rng, 300, rot)
    pos = rng.integers(0, 300, T)
    w = [ref.round16(1 + 0.3 * rng.standard_normal(D), dtype) for _ in range(2)]
    wq_, wk_ = (w[0] if weights != "none" else None), (w[1] if weights == "both" else None)
    dev = ref.on_gpu(qkv, dtype)
    dq, dk = dev[:, : Hq * D].view(T, Hq, D), dev[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
    before = dev.clone()
    oq, ok = wq.wq_qk_norm_rope(dq, dk, torch.from_numpy(pos).cuda(), torch.from_numpy(cs).cuda(),
                                None if wq_ is None else ref.on_gpu(wq_, dtype),
                                None if wk_ is None else ref.on_gpu(wk_, dtype), eps=1e-5, interleaved=interleaved)
    assert torch.equal(dev, before)
    for got, x, weight in ((oq, q, wq_), (ok, k, wk_)):
        want = ref.norm_rope(x, pos, cs.astype(np.float64), rot, interleaved, weight, 1e-5)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= _bound(want, x, dtype)).all(), err.max()


def test_in_place_and_side_stream():
    rng = np.random.default_rng(3)
    T, Hq, Hkv, D = 41, 8, 2, 128
    dev = ref.on_gpu(ref.random16(rng, (T, (Hq + 2 * Hkv) * D), "bf16"), "bf16")
    q, k = dev[:, : Hq * D].view(T, Hq, D), dev[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
    tail = dev[:, (Hq + Hkv) * D:].clone()
    pos = torch.arange(T, device="cuda")
    cs = torch.from_numpy(_table(rng, T, D)).cuda()
    want = wq.wq_qk_norm_rope(q, k, pos, cs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        oq, ok = wq.wq_qk_norm_rope(q, k, pos, cs, q_out=q, k_out=k)
    side.synchronize()
    assert oq.data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(dev[:, (Hq + Hkv) * D:], tail)


def test_zero_rows_and_infinities():
    """A row of zeros stays zero under the norm; an infinity spoils its own row only."""
    D = 64
    q = torch.randn(3, 2, D, device="cuda", dtype=torch.float16)
    k = torch.randn(3, 1, D, device="cuda", dtype=torch.float16)
    q[0, 0] = 0
    q[1, 1, 5] = float("inf")
    cs = torch.from_numpy(_table(np.random.default_rng(0), 4, D)).cuda()
    w = torch.ones(D, device="cuda", dtype=torch.float16)
    oq, ok = wq.wq_qk_norm_rope(q, k, torch.zeros(3, dtype=torch.int64, device="cuda"), cs, w, w)
    assert (oq[0, 0] == 0).all()
    assert not torch.isfinite(oq[1, 1, 5])
    good = torch.ones(3, 2, dtype=torch.bool, device="cuda")
    good[1, 1] = False
    assert torch.isfinite(oq[good]).all() and torch.isfinite(ok).all()


def test_position_out_of_range_is_reported_and_left_unwritten():
    D = 64
    q = torch.randn(3, 2, D, device="cuda", dtype=torch.float16)
    k = torch.randn(3, 1, D, device="cuda", dtype=torch.float16)
    cs = torch.from_numpy(_table(np.random.default_rng(0), 4, D)).cuda()
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    wq.wq_clear_device_status()
    wq.wq_qk_norm_rope(q, k, torch.tensor([1, 4, -1], device="cuda"), cs, q_out=qo, k_out=ko)
    assert wq.wq_device_status() == 1 << 6
    wq.wq_clear_device_status()
    assert (qo[1:] == 7).all() and (ko[1:] == 7).all() and not (qo[0] == 7).all()


def test_empty():
    q = torch.empty(0, 2, 64, device="cuda", dtype=torch.float16)
    oq, ok = wq.wq_qk_norm_rope(q, q, torch.empty(0, dtype=torch.int64, device="cuda"),
                                torch.empty(4, 64, device="cuda"))
    assert oq.shape == (0, 2, 64) and ok.shape == (0, 2, 64)


def test_refusals():
    T, D = 4, 64
    q = torch.randn(T, 2, D, device="cuda", dtype=torch.float16)
    k = torch.randn(T, 1, D, device="cuda", dtype=torch.float16)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    cs = torch.zeros(8, D, device="cuda")
    ok = dict(q=q, k=k, positions=pos, cos_sin=cs)
    bad = [dict(q=q.float()), dict(k=k.bfloat16()), dict(k=k[:3]), dict(positions=pos.int()), dict(positions=pos[:3]),
           dict(cos_sin=cs.half()), dict(cos_sin=cs[:, ::2]), dict(q_weight=torch.ones(D, device="cuda")),
           dict(k_weight=torch.ones(D - 1, device="cuda", dtype=torch.float16)), dict(q=q.transpose(0, 1)),
           dict(q_out=torch.empty_like(k)), dict(q=q.cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            wq.wq_qk_norm_rope(**{**ok, **b})
    for b in (dict(cos_sin=torch.zeros(8, D + 8, device="cuda")), dict(cos_sin=torch.zeros(8, 12, device="cuda")),
              dict(eps=-1.0)):
        with pytest.raises(wq.WQError):
            wq.wq_qk_norm_rope(**{**ok, **b})
