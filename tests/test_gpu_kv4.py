"""The 4-bit cache: wq_kv4_write and wq_kv4_read byte for byte and value for value against a
64-bit reference, on ordinary and on awkward values, and what they refuse."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu

LAYOUTS = [(D, G, P) for D in (64, 128) for G in (32, 64, 128) if G <= D for P in (16, 32, 64, 128)]


def _values(rng, shape, dtype, kind):
    if kind == "plain":
        return ref.random16(rng, shape, dtype)
    if kind == "coarse":     # few significant bits: quotients fall on ties
        return rng.integers(-8, 9, shape).astype(np.float64) / 2
    if kind == "wide":       # magnitudes over many binades
        lim = 12 if dtype == "f16" else 60
        return ref.round16(rng.standard_normal(shape) * np.exp2(rng.integers(-lim, lim, shape)), dtype)
    if kind == "tiny":       # subnormal steps
        return ref.round16(rng.standard_normal(shape) * (2.0 ** -22 if dtype == "f16" else 2.0 ** -130), dtype)
    if kind == "flat":       # one value in a group
        return np.broadcast_to(ref.random16(rng, shape[:-1] + (1,), dtype), shape).copy()
    raise ValueError(kind)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_write_bytes_and_read_values(layout, dtype):
    D, G, P = layout
    H, pages, T = 3, 4, 37
    rng = np.random.default_rng(D + G + P)
    cache = ref.Cache(pages, H, D, G, P, dtype)
    dev = wq.wq_kv4_pages(pages, H, D, G, P, "cuda")
    assert dev.shape == cache.bytes.shape
    slots = rng.permutation(pages * P)[:T]
    k, v = ref.random16(rng, (T, H, D), dtype), ref.random16(rng, (T, H, D), dtype, 3.0)
    for t in range(T):
        cache.put(slots[t], k[t], v[t])
    wq.wq_kv4_write(ref.on_gpu(k, dtype), ref.on_gpu(v, dtype), torch.from_numpy(slots).cuda(), dev, G, P)
    assert np.array_equal(dev.cpu().numpy(), cache.bytes)
    order = rng.permutation(T)
    rk, rv = wq.wq_kv4_read(dev, torch.from_numpy(slots[order]).cuda(), D, G, P, ref.TORCH[dtype])
    for i, t in enumerate(order):
        wk, wv = cache.get(slots[t])
        assert np.array_equal(rk[i].double().cpu().numpy(), wk) and np.array_equal(rv[i].double().cpu().numpy(), wv)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["coarse", "wide", "tiny", "flat"])
def test_awkward_values(kind, dtype):
    D, G, P, H, T = 128, 32, 16, 2, 48
    rng = np.random.default_rng(5)
    k, v = _values(rng, (T, H, D), dtype, kind), _values(rng, (T, H, D), dtype, kind)
    cache = ref.Cache(3, H, D, G, P, dtype)
    for t in range(T):
        cache.put(t, k[t], v[t])
    dev = wq.wq_kv4_pages(3, H, D, G, P, "cuda")
    slots = torch.arange(T, device="cuda")
    wq.wq_kv4_write(ref.on_gpu(k, dtype), ref.on_gpu(v, dtype), slots, dev, G, P)
    rk, rv = wq.wq_kv4_read(dev, slots, D, G, P, ref.TORCH[dtype])
    for got, x, which in ((rk, k, 0), (rv, v, 1)):
        got = got.double().cpu().numpy()
        want = np.stack([cache.get(t)[which] for t in range(T)])
        if kind != "wide":
            assert np.array_equal(got, want)
        # a value stays within half a step of its code, a step's own rounding (15 of them), and one rounding
        g = x.reshape(T, H, -1, G)
        step = (g.max(-1) - g.min(-1)) / 15
        p, qmin = ref.FORMATS[dtype]
        slack = 0.5 * step + 15.5 * np.maximum(step * 2.0 ** -p, 2.0 ** (qmin - 1))
        tol = np.repeat(slack, G, -1).reshape(x.shape) + ref.unit(dtype) * np.abs(want) + 2.0 ** (qmin - 1)
        assert (np.abs(got - x) <= tol * (1 + 1e-6)).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_largest_values(dtype):
    D, G, P = 64, 64, 16
    top = 65504.0 if dtype == "f16" else 1e38
    k = torch.zeros(2, 1, D, device="cuda", dtype=ref.TORCH[dtype])
    k[0, 0, 0], k[0, 0, 1] = top, -top
    k[1, 0, :] = top
    dev = wq.wq_kv4_pages(1, 1, D, G, P, "cuda")
    slots = torch.arange(2, device="cuda")
    wq.wq_kv4_write(k, k, slots, dev, G, P)
    rk, rv = wq.wq_kv4_read(dev, slots, D, G, P, ref.TORCH[dtype])
    assert torch.isfinite(rk).all() and torch.equal(rk, rv)
    assert torch.equal(rk[1], k[1]) and rk[0, 0, 1] == k[0, 0, 1]
    # half a step of 2 top / 15, and 15 roundings of the step
    assert (rk[0].double() - k[0].double()).abs().max() <= top / 15 * 1.001 + 2 * top * ref.unit(dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_spoils_its_group_only(dtype, bad):
    D, G, P, H = 128, 32, 16, 2
    k = torch.randn(3, H, D, device="cuda").to(ref.TORCH[dtype])
    k[1, 1, 40] = bad
    v = torch.randn(3, H, D, device="cuda").to(ref.TORCH[dtype])
    dev = wq.wq_kv4_pages(2, H, D, G, P, "cuda")
    slots = torch.tensor([5, 6, 7], device="cuda")
    wq.wq_kv4_write(k, v, slots, dev, G, P)
    rk, rv = wq.wq_kv4_read(dev, slots, D, G, P, ref.TORCH[dtype])
    assert torch.isnan(rk[1, 1, 32:64]).all()
    rk[1, 1, 32:64] = 0
    assert torch.isfinite(rk).all() and torch.isfinite(rv).all()


def test_slots_skipped_and_out_of_range():
    D, G, P, H = 64, 32, 16, 1
    k = torch.randn(4, H, D, device="cuda", dtype=torch.float16)
    dev = wq.wq_kv4_pages(2, H, D, G, P, "cuda")
    wq.wq_clear_device_status()
    wq.wq_kv4_write(k[:2], k[:2], torch.tensor([-1, 3], device="cuda"), dev, G, P)
    assert wq.wq_device_status() == 0
    kept = dev.clone()
    wq.wq_kv4_write(k[2:], k[2:], torch.tensor([-5, 32], device="cuda"), dev, G, P)
    assert wq.wq_device_status() == 1 << 6 and torch.equal(dev, kept)
    wq.wq_clear_device_status()
    rk, rv = wq.wq_kv4_read(dev, torch.tensor([-1, 3, 31, 32], device="cuda"), D, G, P, torch.float16)
    assert wq.wq_device_status() == 1 << 6
    wq.wq_clear_device_status()
    assert (rk[0] == 0).all() and (rv[0] == 0).all() and (rk[3] == 0).all() and (rk[1] != 0).any()


def test_strides_and_side_stream():
    """Keys and values inside a packed projection, read back into strided outputs, on another stream."""
    D, G, P, H, T = 128, 64, 32, 4, 29
    qkv = torch.randn(T, 10 * D, device="cuda").bfloat16()
    k, v = qkv[:, 2 * D: 6 * D].view(T, H, D), qkv[:, 6 * D:].view(T, H, D)
    slots = torch.randperm(64, device="cuda")[:T]
    a, b = wq.wq_kv4_pages(2, H, D, G, P, "cuda"), wq.wq_kv4_pages(2, H, D, G, P, "cuda")
    wq.wq_kv4_write(k.contiguous(), v.contiguous(), slots, a, G, P)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full((T, 3, H, D), 9.0, device="cuda", dtype=torch.bfloat16)
    with torch.cuda.stream(side):
        wq.wq_kv4_write(k, v, slots, b, G, P)
        side_k, side_v = wq.wq_kv4_read(b, slots, D, G, P, torch.bfloat16, k=out[:, 0], v=out[:, 2])
    side.synchronize()
    assert torch.equal(a, b) and (out[:, 1] == 9).all()
    rk, rv = wq.wq_kv4_read(a, slots, D, G, P, torch.bfloat16)
    assert torch.equal(rk, out[:, 0]) and torch.equal(rv, out[:, 2])


def test_writing_again_what_was_read_changes_nothing_much():
    """Read values are on their group's grid: quantised again they come back within a step's rounding."""
    D, G, P, H, T = 128, 128, 64, 2, 64
    k = torch.randn(T, H, D, device="cuda", dtype=torch.float16)
    dev = wq.wq_kv4_pages(1, H, D, G, P, "cuda")
    slots = torch.arange(T, device="cuda")
    wq.wq_kv4_write(k, k, slots, dev, G, P)
    k1, _ = wq.wq_kv4_read(dev, slots, D, G, P, torch.float16)
    wq.wq_kv4_write(k1, k1, slots, dev, G, P)
    k2, _ = wq.wq_kv4_read(dev, slots, D, G, P, torch.float16)
    # the second step differs from the first by its rounding, at most 2^-11 of it and of the ends (|x| < 8)
    assert (k1.double() - k2.double()).abs().max() <= 15 * 2.0 ** -10 + 2 * 2.0 ** -8


def test_offsets_past_32_bits():
    D, G, P, H = 128, 128, 128, 8
    block = P * (D + 8)
    n = (1 << 32) // (block * H) + 5
    pages = torch.empty(n, H, block, dtype=torch.uint8, device="cuda")
    pages[0].zero_()
    k = torch.randn(3, H, D, device="cuda").bfloat16()
    slots = torch.tensor([n * P - 1, 1, (n - 2) * P + 64], device="cuda")
    wq.wq_kv4_write(k, k, slots, pages, G, P)
    small = wq.wq_kv4_pages(1, H, D, G, P, "cuda")
    three = torch.arange(3, device="cuda")
    wq.wq_kv4_write(k, k, three, small, G, P)
    want = wq.wq_kv4_read(small, three, D, G, P, torch.bfloat16)
    got = wq.wq_kv4_read(pages, slots, D, G, P, torch.bfloat16)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_and_refusals():
    D, G, P, H = 64, 32, 16, 2
    dev = wq.wq_kv4_pages(2, H, D, G, P, "cuda")
    e = torch.empty(0, H, D, device="cuda", dtype=torch.float16)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    wq.wq_kv4_write(e, e, none, dev, G, P)
    assert wq.wq_kv4_read(dev, none, D, G, P, torch.float16)[0].shape == (0, H, D)
    k = torch.randn(3, H, D, device="cuda", dtype=torch.float16)
    s = torch.arange(3, device="cuda")
    ok = dict(k=k, v=k, slots=s, pages=dev, group=G, page_size=P)
    for b in (dict(k=k.float()), dict(v=k[:2]), dict(v=k.bfloat16()), dict(slots=s.int()), dict(slots=s[:2]), dict(group=64),
              dict(page_size=32), dict(pages=dev.int()), dict(pages=dev[:, :1].contiguous()), dict(pages=dev.cpu()),
              dict(k=k.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            wq.wq_kv4_write(**{**ok, **b})
    odd = torch.randn(3, H * D + 4, device="cuda", dtype=torch.float16)[:, : H * D].unflatten(1, (H, D))
    with pytest.raises(wq.WQError):      # rows off their 16-byte alignment
        wq.wq_kv4_write(**{**ok, "k": odd})
    with pytest.raises(wq.WQError):
        wq.wq_kv4_page_bytes(H, 96, 32, 16)
    with pytest.raises(wq.WQError):
        wq.wq_kv4_page_bytes(H, 64, 128, 16)
