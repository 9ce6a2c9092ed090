"""Norm + rotation and the cache at a prompt's sizes, where a group of lanes takes several heads: every number of
heads that the launch rules choose, with head counts that it does not divide."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ norm + rotation

def _tokens(per, Hq, Hkv, D):
    """The fewest tokens for which a group of lanes takes `per` heads: two blocks of 256 threads for each SM."""
    lanes = 8 if D <= 64 else 16 if D <= 128 else 32
    want = _sms() * 2 * (256 // lanes)

    def groups(n):
        return -(-Hq // n) + -(-Hkv // n)
    T = -(-want // groups(per))
    assert per == 16 or T * groups(2 * per) < want
    return T


def _table(rng, most, rot):
    ang = rng.uniform(-200, 200, (most, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _groups(per, heads):
    return sum(-(-n // per) for n in heads)


SHAPES = [(128, 128, False), (64, 32, True), (256, 64, False), (96, 96, True)]   # D, rotated values, neighbours
HEADS = [(14, 2), (5, 1), (33, 3), (19, 17)]
# (where twice the heads make no fewer groups, they are taken)
CASES = [(*s, per, h) for s in SHAPES for h in HEADS for per in (4, 8, 16)
         if per == 16 or _groups(per, h) > _groups(2 * per, h)]
CASES = [(*c, ("both", "k", "none")[i % 3], ("f16", "bf16")[i // 2 % 2]) for i, c in enumerate(CASES)]


@pytest.mark.parametrize("D,rot,interleaved,per,heads,weights,dtype", CASES)
def test_rotation_of_several_heads_for_each_group(D, rot, interleaved, per, heads, weights, dtype):
    Hq, Hkv = heads
    T = _tokens(per, Hq, Hkv, D)
    rng = np.random.default_rng(per * 1000 + Hq + D)
    qkv = ref.random16(rng, (T, (Hq + 2 * Hkv) * D), dtype, 2.0)
    q, k = qkv[:, : Hq * D].reshape(T, Hq, D), qkv[:, Hq * D: (Hq + Hkv) * D].reshape(T, Hkv, D)
    cs = _table(rng, 300, rot)
    pos = rng.integers(0, 300, T)
    w = [ref.round16(1 + 0.3 * rng.standard_normal(D), dtype) for _ in range(2)]
    wq_, wk_ = (w[0] if weights == "both" else None), (w[1] if weights != "none" else None)
    dev = ref.on_gpu(qkv, dtype)
    dq, dk = dev[:, : Hq * D].view(T, Hq, D), dev[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
    tail = dev[:, (Hq + Hkv) * D:].clone()
    call = dict(positions=torch.from_numpy(pos).cuda(), cos_sin=torch.from_numpy(cs).cuda(),
                q_weight=None if wq_ is None else ref.on_gpu(wq_, dtype),
                k_weight=None if wk_ is None else ref.on_gpu(wk_, dtype), eps=1e-5, interleaved=interleaved)
    oq, ok = wq.wq_qk_norm_rope(dq, dk, **call)
    # one rounding of the result; fp32: a square root and a few products and sums of values no larger than the row's
    # largest (64 steps of 2^-24 are generous); fp16 results below 2^-14 keep steps of 2^-24
    for got, x, weight in ((oq, q, wq_), (ok, k, wk_)):
        want = ref.norm_rope(x, pos, cs.astype(np.float64), rot, interleaved, weight, 1e-5)
        tol = ref.unit(dtype) * np.abs(want) + 64 * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True) + 2.0 ** -25
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    # in place, inside the packed projection
    wq.wq_qk_norm_rope(dq, dk, **call, q_out=dq, k_out=dk)
    assert torch.equal(dq, oq) and torch.equal(dk, ok) and torch.equal(dev[:, (Hq + Hkv) * D:], tail)


# ------------------------------------------------------------------ the cache

def _pair_tokens(H, D):
    """The fewest tokens for which a group of lanes takes two heads."""
    return -(-_sms() * 2 * 256 // (-(-H // 2) * (D // 8)))


def _bytes(cache, slots, k, v):
    """The reference cache with the tokens k, v [T][H][D] in their slots."""
    page, place = slots // cache.P, slots % cache.P
    c, r = cache.D // 2, 4 * (cache.D // cache.G)
    for which, x in ((0, k), (1, v)):
        q, s, lo = ref.quantise(x, cache.G, cache.dtype)
        pairs = ref.to_bits(np.stack([s, lo], -1), cache.dtype).reshape(x.shape[:2] + (-1,)).view(np.uint8)
        code = ((which * cache.P + place) * c)[:, None] + np.arange(c)
        pair = (cache.P * cache.D + (which * cache.P + place) * r)[:, None] + np.arange(r)
        for h in range(cache.H):
            cache.bytes[page[:, None], h, code] = q[:, h, 0::2] | (q[:, h, 1::2] << 4)
            cache.bytes[page[:, None], h, pair] = pairs[:, h]


@pytest.mark.parametrize("D,G,P,H,dtype", [(128, 128, 16, 2, "bf16"), (128, 128, 64, 9, "f16"), (128, 64, 128, 3, "f16"),
                                           (128, 64, 32, 8, "bf16"), (128, 32, 64, 3, "bf16"), (128, 32, 16, 2, "f16"),
                                           (64, 64, 32, 9, "bf16"), (64, 64, 16, 4, "f16"), (64, 32, 128, 3, "f16"),
                                           (64, 32, 16, 8, "bf16")])
def test_two_heads_for_each_group_write_and_read(D, G, P, H, dtype):
    T = _pair_tokens(H, D) + 3
    rng = np.random.default_rng(D + G + P + H)
    pages = -(-T // P) + 2
    cache = ref.Cache(pages, H, D, G, P, dtype)
    slots = rng.permutation(pages * P)[:T]
    k, v = ref.random16(rng, (T, H, D), dtype), ref.random16(rng, (T, H, D), dtype, 3.0)
    k[::7] = rng.integers(-8, 9, k[::7].shape) / 2      # quotients on ties
    v[::5] = v[::5, :, :1]                              # one value in a group
    _bytes(cache, slots, k, v)
    dev = wq.wq_kv4_pages(pages, H, D, G, P, "cuda")
    given = slots.copy()
    spare = sorted(set(range(pages * P)) - set(slots.tolist()))[0]
    given[11], given[T - 1] = -1, -9                    # skipped: their slots stay as they are
    for t in (11, T - 1):
        page, place = divmod(int(slots[t]), P)
        for which in (0, 1):
            for at in cache._at(which, place):
                cache.bytes[page, :, at] = 0
    # keys and values as slices of one packed row
    packed = ref.on_gpu(np.concatenate([k.reshape(T, -1), v.reshape(T, -1)], 1), dtype)
    dk, dv = packed[:, : H * D].view(T, H, D), packed[:, H * D:].view(T, H, D)
    wq.wq_kv4_write(dk, dv, torch.from_numpy(given).cuda(), dev, G, P)
    assert np.array_equal(dev.cpu().numpy(), cache.bytes)
    order = rng.permutation(T)
    asked = slots[order].copy()
    asked[0], asked[1] = -1, spare
    rk, rv = wq.wq_kv4_read(dev, torch.from_numpy(asked).cuda(), D, G, P, ref.TORCH[dtype])
    for which, (got, x) in enumerate(((rk, k), (rv, v))):
        want = ref.values(*ref.quantise(x, G, dtype), dtype)[order]
        skipped = np.isin(order, (11, T - 1))
        want[skipped] = 0
        want[:2] = 0
        assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["wide", "tiny", "bad"])
@pytest.mark.parametrize("H", [3, 4])
def test_two_heads_for_each_group_awkward_values(H, kind, dtype):
    """The bytes that calls of a few tokens, one head for each group of lanes, write of the same values."""
    D, G, P = 128, 32, 32
    T = _pair_tokens(H, D) + 5
    gen = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(2, T, H, D, device="cuda", generator=gen)
    if kind == "wide":
        e = 12 if dtype == "f16" else 60
        x *= torch.randint(-e, e, x.shape, device="cuda", generator=gen).float().exp2()
    elif kind == "tiny":
        x *= 2.0 ** -22 if dtype == "f16" else 2.0 ** -127
    else:
        at = torch.randint(0, 400, x.shape, device="cuda", generator=gen)
        x = x.where(at != 0, float("nan")).where(at != 1, float("inf")).where(at != 2, -float("inf"))
    k, v = x.to(ref.TORCH[dtype])
    pages = -(-T // P)
    slots = torch.randperm(pages * P, device="cuda", generator=gen)[:T]
    a, b = (wq.wq_kv4_pages(pages, H, D, G, P, "cuda") for _ in range(2))
    wq.wq_kv4_write(k, v, slots, a, G, P)
    step = _pair_tokens(H, D) // 4
    for t in range(0, T, step):
        wq.wq_kv4_write(k[t: t + step], v[t: t + step], slots[t: t + step], b, G, P)
    assert torch.equal(a, b)
