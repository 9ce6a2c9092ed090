"""wq_attn_kv4 over caches and scales far from one: keys, values and scales of any size that the types hold
give what the cache's values give in 64 bits, to a bound that is relative to them."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu


class Sequence:
    """One sequence over a shuffled cache: k, v float64 [L][Hkv][D], already numbers of the type."""

    def __init__(self, k, v, G, P, dtype, seed=0):
        L, H, self.D = k.shape
        self.G, self.P, self.dtype, self.L = G, P, dtype, L
        each = -(-L // P)
        cache = ref.Cache(each + 1, H, self.D, G, P, dtype)
        table = np.random.default_rng(seed).permutation(each + 1)[:each].astype(np.int32)
        self.K, self.V = np.zeros_like(k), np.zeros_like(v)
        for t in range(L):
            slot = int(table[t // P]) * P + t % P
            cache.put(slot, k[t], v[t])
            self.K[t], self.V[t] = cache.get(slot)
        self.pages = cache.pages()
        self.table = torch.from_numpy(table)[None].cuda()

    def check(self, q, scale=None, causal=True):
        n, Hq = q.shape[:2]
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([self.L], dtype=torch.int32, device="cuda")
        lse = torch.empty(n, Hq, device="cuda")
        out = wq.wq_attn_kv4(ref.on_gpu(q, self.dtype), self.pages, self.table, lens, self.G, self.P, cu_q=cu, max_q=n,
                             scale=scale, causal=causal, lse=lse).double().cpu().numpy()
        sc = 1 / np.sqrt(self.D) if scale is None else scale
        want, wl, A = ref.attention(q, self.K, self.V, sc, n, causal)
        # one rounding of the result and one of each probability, a quarter more for the fp32 scores and sums; fp16:
        # probabilities below 2^-14 keep steps of 2^-24, and so do results
        tol = 2.5 * ref.unit(self.dtype) * A
        if self.dtype == "f16":
            tol += self.L * 2.0 ** -25 * np.abs(self.V).max() + 2.0 ** -25
        err = np.abs(out - want)
        assert (err <= tol).all(), (np.isnan(out).sum(), float((err / np.maximum(tol, 1e-300)).max()))
        S = max(1.0, float(np.abs(q).sum(-1).max() * np.abs(self.K).max() * abs(sc)))
        lse = lse.double().cpu().numpy()
        empty = np.isneginf(wl)     # more queries than tokens: the first ones see nothing
        assert np.isneginf(lse[empty]).all()
        assert (np.abs(lse[~empty] - wl[~empty]) <= 2 * self.D * 2.0 ** -24 * S + 2e-6).all()


# new tokens with 4 query heads for each key head: 4, 12, 20 rows (few rows), 240 (many)
NEWS = [1, 3, 5, 60]
POWERS = [("bf16", e) for e in (-90, -60, -47, -45, -31, -29, 60, 73, 76, 78, 100, 121)] + [("f16", -10), ("f16", 10)]


def _numbers(rng, shape, dtype, e=0):
    return ref.round16(rng.standard_normal(shape), dtype) * 2.0 ** e


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("dtype,e", POWERS)
@pytest.mark.parametrize("D,G,P", [(128, 128, 16), (64, 32, 64)])
def test_sizes_of_values(D, G, P, dtype, e, n):
    rng = np.random.default_rng(e + 200)
    k, v = _numbers(rng, (150, 2, D), dtype), _numbers(rng, (150, 2, D), dtype, e)
    Sequence(k, v, G, P, dtype).check(_numbers(rng, (n, 8, D), dtype))


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("dtype,e", POWERS)
def test_sizes_of_keys(dtype, e, n):
    """Keys of one size and queries of the other: scores of ordinary size."""
    rng = np.random.default_rng(e + 300)
    k, v = _numbers(rng, (150, 2, 64), dtype, e), _numbers(rng, (150, 2, 64), dtype)
    q = ref.round16(_numbers(rng, (n, 8, 64), dtype, -e), dtype)
    Sequence(k, v, 64, 16, dtype).check(q)


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("e", [-100, -40, 79, 110])
def test_one_token_of_another_size(e, causal, n):
    """A token among ordinary ones whose keys or values are very small, or so large that its low score
    makes it count as the others do."""
    rng = np.random.default_rng(e + 400)
    k, v = _numbers(rng, (300, 2, 64), "bf16"), _numbers(rng, (300, 2, 64), "bf16")
    q = np.abs(_numbers(rng, (n, 8, 64), "bf16")) + 0.25
    q = ref.round16(q, "bf16")
    for t in (140, 190):
        v[t] *= 2.0 ** e
        if e < 0:
            k[t] *= 2.0 ** e
        else:   # q . k / 8 below -2 |k|: the weight is some 2^-e of the others'
            k[t] = ref.round16(np.full((2, 64), -e * np.log(2) / (8 * q.mean() + 1e-9)), "bf16")
    Sequence(k, v, 32, 32, "bf16").check(q, causal=causal)


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("e", [-110, 45, 60, 100, 118])
def test_sizes_of_scales(e, n):
    """A scale of one size, keys and queries of the other."""
    rng = np.random.default_rng(e + 500)
    a, b = -(e // 2), -(e - e // 2)
    k, v = _numbers(rng, (150, 1, 64), "bf16", a), _numbers(rng, (150, 1, 64), "bf16")
    Sequence(k, v, 64, 32, "bf16").check(_numbers(rng, (n, 4, 64), "bf16", b), scale=2.0 ** (e - 3))


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rising", [False, True])
def test_largest_values(rising, dtype, n):
    """Values at the type's end, of one sign: no sum of them passes what it is divided by."""
    rng = np.random.default_rng(800)
    # a few steps of the type short of its end, so that the roundings of probabilities stay below it
    top = 64000.0 if dtype == "f16" else 2.0 ** 127 * 1.953125
    k, v = _numbers(rng, (500, 1, 64), dtype), np.full((500, 1, 64), top)
    v[::3, :, ::5] *= 0.5
    if rising:      # the running maximum follows late
        k = ref.round16(k + np.linspace(0, 12, 500)[:, None, None], dtype)
    q = ref.round16(np.abs(_numbers(rng, (n, 4, 64), dtype)), dtype)
    Sequence(k, v, 64, 32, dtype).check(q)


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("e", [-103, -120])
def test_small_scales_of_large_scores(e, n):
    rng = np.random.default_rng(e + 600)
    k, v = _numbers(rng, (150, 1, 64), "bf16", -e - 20), _numbers(rng, (150, 1, 64), "bf16")
    Sequence(k, v, 64, 32, "bf16").check(_numbers(rng, (n, 4, 64), "bf16", 17), scale=2.0 ** e)


@pytest.mark.parametrize("n", NEWS)
def test_zero_scale_of_large_scores(n):
    """Every visible token counts the same, however large its score."""
    rng = np.random.default_rng(700)
    k, v = _numbers(rng, (150, 1, 64), "bf16", 100), _numbers(rng, (150, 1, 64), "bf16")
    Sequence(k, v, 64, 32, "bf16").check(_numbers(rng, (n, 4, 64), "bf16", 10), scale=0.0)


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("e", [0, -60, 90])
@pytest.mark.parametrize("D,G", [(128, 32), (64, 32)])
def test_columns_of_zeros(D, G, e, n):
    """Heads padded with zeros: the padding's results are zero, the others as without it."""
    rng = np.random.default_rng(e + 900)
    k, v = _numbers(rng, (150, 2, D), "bf16"), _numbers(rng, (150, 2, D), "bf16", e)
    k[..., D - 32:], v[..., D - 32:] = 0, 0
    Sequence(k, v, G, 16, "bf16").check(_numbers(rng, (n, 8, D), "bf16"))


@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("L", [1, 2, 3, 17])
@pytest.mark.parametrize("e", [-70, 0, 80])
def test_a_few_tokens(e, L, n):
    rng = np.random.default_rng(e + 1000 + L)
    k, v = _numbers(rng, (L, 2, 64), "bf16"), _numbers(rng, (L, 2, 64), "bf16", e)
    Sequence(k, v, 64, 16, "bf16").check(_numbers(rng, (n, 8, 64), "bf16"))


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("e", [-70, 0, 80])
@pytest.mark.parametrize("P", [16, 64])
def test_pages_before_the_window_are_not_touched(P, e, n):
    """Their table entries may be anything, and what lies in the seen pages outside the window too."""
    L, window = 400, 100
    rng = np.random.default_rng(e + 1100)
    k, v = _numbers(rng, (L, 2, 64), "bf16"), _numbers(rng, (L, 2, 64), "bf16", e)
    gone = (L - n + 1 - window) // P * P          # tokens of pages that nobody sees
    s = Sequence(k, v, 32, P, "bf16")
    q = _numbers(rng, (n, 8, 64), "bf16")
    call = dict(cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n, window=window)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    wq.wq_clear_device_status()
    a = wq.wq_attn_kv4(ref.on_gpu(q, "bf16"), s.pages, s.table, lens, 32, P, **call)
    table = s.table.clone()
    table[0, : gone // P] = torch.tensor([-5, 10 ** 6] * (gone // P), dtype=torch.int32, device="cuda")[: gone // P]
    b = wq.wq_attn_kv4(ref.on_gpu(q, "bf16"), s.pages, table, lens, 32, P, **call)
    assert wq.wq_device_status() == 0 and torch.equal(a, b)
    want, _, A = ref.attention(q, s.K, s.V, 64 ** -0.5, n, True, window)
    assert (np.abs(a.double().cpu().numpy() - want) <= 2.5 * ref.unit("bf16") * A).all()


@pytest.mark.parametrize("n", NEWS)
@pytest.mark.parametrize("e", [0, -60, 90])
def test_sums_that_cancel(e, n):
    """Values of opposite sign under equal scores: results of exactly zero, beside values of another size."""
    rng = np.random.default_rng(e + 1200)
    k = np.broadcast_to(_numbers(rng, (1, 2, 64), "bf16"), (128, 2, 64)).copy()
    v = np.ones((128, 2, 64))
    v[:, :, ::3] = -1
    v[1::2] *= -1
    v[..., 32:] = _numbers(rng, (128, 2, 32), "bf16", e)
    Sequence(k, v, 32, 16, "bf16").check(_numbers(rng, (n, 8, 64), "bf16"), causal=False)
