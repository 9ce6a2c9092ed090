"""wq_attn_kv4 against 64-bit attention over the cache's values: head layouts, types, lengths and masks
where it can go wrong, what pages hold past a sequence's end, streams, graphs, determinism, refusals."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import weight_only_quantized_tma_gb300 as wq

pytestmark = pytest.mark.gpu


class Problem:
    """Sequences of given lengths and new tokens over a shuffled cache; values in 64 bits beside it."""

    def __init__(self, lens, news, Hq, Hkv, D, G, P, dtype, seed=0, qscale=1.0, poison=True):
        rng = np.random.default_rng(seed)
        self.lens, self.news, self.Hq, self.Hkv, self.D, self.G, self.P, self.dtype = lens, news, Hq, Hkv, D, G, P, dtype
        need = [-(-L // P) for L in lens]
        width = max(1, max(need))
        total = sum(need) + 2
        cache = ref.Cache(total, Hkv, D, G, P, dtype)
        place = rng.permutation(total - 1) + 1
        table = np.zeros((len(lens), width), dtype=np.int32)
        at, self.KV = 0, []
        for b, L in enumerate(lens):
            table[b, : need[b]] = place[at: at + need[b]]
            at += need[b]
            k = ref.random16(rng, (L, Hkv, D), dtype) + 0.25
            k, v = ref.round16(k, dtype), ref.random16(rng, (L, Hkv, D), dtype)
            kv = np.zeros((2, L, Hkv, D))
            for t in range(L):
                slot = int(table[b, t // P]) * P + t % P
                cache.put(slot, k[t], v[t])
                kv[:, t] = cache.get(slot)
            self.KV.append(kv)
        if poison:   # what lies past each sequence's end, and in pages of no sequence, is NaN
            bad = np.full((Hkv, D), np.nan)
            for b, L in enumerate(lens):
                for t in range(L, need[b] * P):
                    cache.put(int(table[b, t // P]) * P + t % P, bad, bad)
            for page in set(range(total)) - set(table[table > 0].tolist()):
                for t in range(P):
                    cache.put(page * P + t, bad, bad)
        self.q = ref.random16(rng, (sum(news), Hq, D), dtype, qscale)
        self.pages = cache.pages()
        self.table = torch.from_numpy(table).cuda()
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
        self.dq = ref.on_gpu(self.q, dtype)

    def run(self, single=False, **kw):
        lse = torch.full((self.q.shape[0], self.Hq), 5.0, device="cuda")
        kw.setdefault("lse", lse)
        kw.setdefault("max_q", max(self.news))
        out = wq.wq_attn_kv4(kw.pop("q", self.dq), self.pages, self.table, self.kv_lens, self.G, self.P,
                             cu_q=None if single else self.cu, **kw)
        return out, kw["lse"]

    def check(self, causal=True, window=0, scale=None, **kw):
        wq.wq_clear_device_status()
        out, lse = self.run(causal=causal, window=window, scale=scale, **kw)
        assert wq.wq_device_status() == 0
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        sc = 1 / np.sqrt(self.D) if scale is None else scale
        first = 0
        for b, (L, n) in enumerate(zip(self.lens, self.news)):
            q = self.q[first: first + n]
            K, V = self.KV[b]
            want, wl, A = ref.attention(q, K, V, sc, n, causal, window)
            got, gl = out[first: first + n], lse[first: first + n]
            first += n
            if n == 0:
                continue
            tol = ref.attention_bound(self.dtype, A, L, np.abs(V).max() if L else 0.0)
            err = np.abs(got - want)
            assert (err <= tol).all(), (b, L, n, float((err / tol).max()))
            empty = np.isneginf(wl)
            assert (got[empty] == 0).all() and np.isneginf(gl[empty]).all()
            # fp32 scores: products and sums of |q k| scale, 2 D roundings of 2^-24 at most
            S = max(1.0, float(np.abs(q).sum(-1).max() * np.abs(K).max() * sc)) if L else 1.0
            assert (np.abs(gl[~empty] - wl[~empty]) <= 2 * self.D * 2.0 ** -24 * S + 2e-6).all()


LENS = [1, 0, 2, 15, 16, 17, 31, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 300]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G,P", [(128, 128, 16), (128, 64, 32), (128, 32, 64), (64, 64, 16), (64, 32, 128), (128, 128, 128)])
def test_single_tokens(D, G, P, dtype):
    p = Problem(LENS, [1] * len(LENS), 8, 2, D, G, P, dtype, seed=1)
    p.check(single=True)


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (4, 2), (6, 2), (5, 1), (14, 2), (8, 1), (16, 1), (24, 2), (32, 1), (40, 1)])
def test_head_layouts(heads):
    Hq, Hkv = heads
    Problem([70, 3, 130], [1, 1, 1], Hq, Hkv, 128, 128, 16, "bf16", seed=2).check(single=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (7, 1), (6, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_drafts(D, heads, dtype):
    """A few new tokens of each sequence, more than a sequence has among them, some sequences with none."""
    lens = [70, 5, 1, 64, 33, 129, 20, 0]
    news = [4, 5, 3, 1, 0, 7, 20, 2]
    Problem(lens, news, heads[0], heads[1], D, 32, 32, dtype, seed=3).check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G,P", [(128, 128, 64), (64, 32, 16), (128, 32, 128), (64, 64, 32)])
@pytest.mark.parametrize("heads", [(2, 1), (3, 1), (2, 2)])
def test_prompts(heads, D, G, P, dtype):
    """Chunks of prompts: more rows than a tile, ends inside tiles and pages."""
    lens, news = [200, 131, 300, 40], [150, 131, 70, 33]
    Problem(lens, news, heads[0], heads[1], D, G, P, dtype, seed=4).check()


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 8, 2, 16], [100, 130, 41, 66]])
@pytest.mark.parametrize("window", [1, 5, 64, 100])
def test_window(news, window):
    Problem([200, 130, 41, 66], news, 4, 2, 64, 64, 16, "f16", seed=5).check(window=window)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 8, 2, 16], [100, 130, 50, 66]])
def test_not_causal(news):
    Problem([200, 130, 41, 0], news, 4, 2, 128, 64, 32, "bf16", seed=6).check(causal=False)


@pytest.mark.parametrize("n", [1, 4, 100])
@pytest.mark.parametrize("scale", [0.0, 0.5, -0.3, 3.0])
def test_scales(scale, n):
    """No scores, steep and negative ones: the running maximum moves late and often."""
    Problem([300, 150], [n, n], 2, 1, 64, 32, 16, "f16", seed=7).check(scale=scale)


@pytest.mark.parametrize("n", [1, 130])
def test_rising_scores(n):
    """Scores that rise along the sequence by far more than the accumulators' slack."""
    p = Problem([520], [n], 4, 1, 64, 64, 64, "bf16", seed=8, qscale=0.02, poison=False)
    c = ref.Cache(p.pages.shape[0], 1, 64, 64, 64, "bf16")
    table = p.table.cpu().numpy()
    rng = np.random.default_rng(9)
    for t in range(520):
        slot = int(table[0, t // 64]) * 64 + t % 64
        k = ref.round16(np.full((1, 64), t / 4.0) + rng.standard_normal((1, 64)), "bf16")
        c.put(slot, k, ref.random16(rng, (1, 64), "bf16"))
        p.KV[0][:, t] = c.get(slot)
    p.pages = c.pages()
    p.q = ref.round16(np.abs(p.q), "bf16")
    p.dq = ref.on_gpu(p.q, "bf16")
    p.check()


@pytest.mark.parametrize("n", [1, 7, 130])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_that_some_rows_see(n, which):
    """A NaN key or value makes the rows that see it NaN (a value: at least where it stands) and no others,
    those of the same tile that are masked from it among them."""
    at = 196 if n < 100 else 100    # seen by the queries at `at` and later; key head 1 of sequence 0
    p = Problem([200, 190], [n, n], 4, 2, 64, 64, 16, "f16", seed=10)
    page = int(p.table[0, at // 16])
    pair = 16 * 64 + which * 16 * 4 + (at % 16) * 4
    p.pages[page, 1, pair: pair + 4] = torch.tensor([0, 0x7E, 0, 0x7E], dtype=torch.uint8, device="cuda")
    clean = Problem([200, 190], [n, n], 4, 2, 64, 64, 16, "f16", seed=10)
    a, b = clean.run()[0], p.run()[0]
    pos = torch.arange(200 - n, 200, device="cuda")
    hit = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
    hit[:n, 2:] = (pos >= at)[:, None]
    assert torch.isnan(b[hit]).all()
    assert torch.equal(a[~hit], b[~hit])


@pytest.mark.parametrize("n", [1, 6, 100])
def test_strided_queries_and_outputs(n):
    p = Problem([130, 257], [n, n], 6, 3, 128, 128, 16, "bf16", seed=11)
    want, wl = p.run()
    T = 2 * n
    packed = torch.zeros(T, 12 * 128, device="cuda", dtype=torch.bfloat16)
    q = packed[:, : 6 * 128].view(T, 6, 128)
    q.copy_(p.dq)
    buf = torch.full((T, 2, 6, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    got, gl = p.run(q=q, out=buf[:, 1])
    assert torch.equal(got, want) and torch.equal(gl, wl) and (buf[:, 0] == 3).all()
    assert torch.equal(p.run(lse=None)[0], want)


@pytest.mark.parametrize("news", [[1] * 5, [2, 7, 1, 5, 4], [64, 200, 130, 33, 90]])
def test_same_results_every_time_and_on_other_streams(news):
    p = Problem([900, 200, 513, 64, 1100], news, 8, 2, 128, 64, 64, "bf16", seed=12)
    want, wl = p.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        out, lse = p.run()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out, lse = p.run()
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("case", [  # new tokens, length, query heads, key heads, D, G, P, type, sequences
    (9, 40000, 8, 2, 128, 128, 64, torch.bfloat16, 1), (200, 5000, 8, 2, 64, 32, 16, torch.float16, 2),
    (192, 5000, 8, 2, 64, 64, 64, torch.bfloat16, 2), (256, 5000, 8, 2, 64, 64, 64, torch.float16, 1),
    (1, 9000, 8, 2, 128, 64, 32, torch.bfloat16, 7), (25, 20000, 8, 2, 64, 64, 64, torch.float16, 1)])
def test_many_runs_agree(case):
    """Waits that end a phase early show as rare differences: many runs of calls that split items over
    blocks, mix full and part-filled row tiles and move their maxima."""
    n, L, Hq, H, D, G, P, dt, B = case
    gen = torch.Generator(device="cuda").manual_seed(n)
    each = -(-L // P)
    pages = wq.wq_kv4_pages(each * B, H, D, G, P, "cuda")
    table = torch.randperm(each * B, device="cuda", generator=gen).to(torch.int32).view(B, each).contiguous()
    t = torch.arange(L, device="cuda")
    for b in range(B):
        kv = torch.randn(2, L, H, D, device="cuda", generator=gen).to(dt)
        wq.wq_kv4_write(kv[0], kv[1], table[b].long()[t // P] * P + t % P, pages, G, P)
    q = torch.randn(n * B, Hq, D, device="cuda", generator=gen).to(dt)
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    runs = [wq.wq_attn_kv4(q, pages, table, lens, G, P, cu_q=cu, max_q=n) for _ in range(120)]
    assert torch.stack([(r != runs[0]).any() for r in runs]).sum() == 0


@pytest.mark.parametrize("n", [1, 5, 80])
def test_graph_replays_with_new_lengths(n):
    p = Problem([300, 150, 220], [n, n, n], 4, 2, 64, 32, 16, "f16", seed=13, poison=False)
    p.run()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = wq.wq_attn_kv4(p.dq, p.pages, p.table, p.kv_lens, p.G, p.P, cu_q=p.cu, max_q=n)
    for lens in ([300, 150, 220], [90, 100, 80], [300, 81, 200]):
        p.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, p.run()[0])


def test_many_sequences():
    """More sequences than a warp has lanes and than the grid has blocks."""
    rng = np.random.default_rng(14)
    lens = rng.integers(0, 40, 700).tolist()
    Problem(lens, [1] * 700, 2, 1, 64, 64, 16, "f16", seed=15).check(single=True)


def test_many_sequences_of_unequal_news():
    rng = np.random.default_rng(16)
    lens = rng.integers(0, 60, 90).tolist()
    Problem(lens, rng.integers(0, 9, 90).tolist(), 3, 1, 64, 32, 16, "bf16", seed=17).check()


@pytest.mark.parametrize("n", [1, 9, 300])
def test_long_context_against_plain_torch(n):
    """Thousands of tokens split over the whole GPU, against fp64 torch on the read-back cache."""
    H, Hq, D, G, P, L = 2, 8, 128, 128, 64, 40000
    gen = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn(L, H, D, device="cuda", generator=gen).bfloat16()
    v = torch.randn(L, H, D, device="cuda", generator=gen).bfloat16()
    npages = -(-L // P)
    pages = wq.wq_kv4_pages(npages, H, D, G, P, "cuda")
    table = torch.randperm(npages, device="cuda", generator=gen).to(torch.int32)[None].contiguous()
    t = torch.arange(L, device="cuda")
    slots = table[0].long()[t // P] * P + t % P
    wq.wq_kv4_write(k, v, slots, pages, G, P)
    K, V = (x.double() for x in wq.wq_kv4_read(pages, slots, D, G, P, torch.bfloat16))
    q = torch.randn(n, Hq, D, device="cuda", generator=gen).bfloat16()
    out = wq.wq_attn_kv4(q, pages, table, torch.tensor([L], dtype=torch.int32, device="cuda"), G, P,
                         cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_q=n)
    hide = t[None] > torch.arange(L - n, L, device="cuda")[:, None]
    for h in range(Hq):
        s = (q[:, h].double() @ K[:, h // 4].T / D ** 0.5).masked_fill(hide, -float("inf"))
        pr = s.softmax(-1)
        want, A = pr @ V[:, h // 4], pr @ V[:, h // 4].abs()
        assert ((out[:, h].double() - want).abs() <= 2.5 * ref.unit("bf16") * A).all()


def test_offsets_past_32_bits():
    """Pages that lie more than 4 GB into the cache."""
    D, G, P, H = 128, 128, 128, 8
    block = P * (D + 8)
    n = (1 << 32) // (block * H) + 6
    pages = torch.empty(n, H, block, dtype=torch.uint8, device="cuda")
    small = wq.wq_kv4_pages(3, H, D, G, P, "cuda")
    k = torch.randn(300, H, D, device="cuda").bfloat16()
    v = torch.randn(300, H, D, device="cuda").bfloat16()
    wq.wq_kv4_write(k, v, torch.arange(300, device="cuda"), small, G, P)
    far = torch.tensor([[n - 1, n - 3, n - 2]], dtype=torch.int32, device="cuda")
    pages[far[0].long()] = small
    near = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    L = torch.tensor([300], dtype=torch.int32, device="cuda")
    for m in (1, 40):
        q = torch.randn(m, 16, D, device="cuda").bfloat16()
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        a = wq.wq_attn_kv4(q, small, near, L, G, P, cu_q=cu, max_q=m)
        b = wq.wq_attn_kv4(q, pages, far, L, G, P, cu_q=cu, max_q=m)
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 70])
def test_lengths_and_pages_out_of_range_are_reported(n):
    p = Problem([100, 90], [n, n], 2, 1, 64, 64, 16, "f16", seed=18, poison=False)
    want = p.run()[0]
    wq.wq_clear_device_status()
    # past the table: cut to its width (7 pages of 16), as the length itself would be
    p.kv_lens[0] = 5000
    a = p.run()[0]
    assert wq.wq_device_status() == 1 << 6
    wq.wq_clear_device_status()
    p.kv_lens[0] = 7 * 16
    assert torch.equal(a, p.run()[0]) and wq.wq_device_status() == 0
    p.kv_lens[0] = 100
    p.table[0, 2] = 10 ** 6
    p.table[0, 3] = -7
    b = p.run()[0]
    assert wq.wq_device_status() == 1 << 6
    wq.wq_clear_device_status()
    assert torch.equal(b[n:], want[n:]) and torch.isfinite(b).all()
    p.kv_lens[1] = -3       # a negative length is an empty sequence
    assert (p.run()[0][n:] == 0).all()
    wq.wq_clear_device_status()


def test_empty_and_refusals():
    p = Problem([30, 20], [1, 1], 4, 2, 64, 32, 16, "f16", seed=19)
    e = wq.wq_attn_kv4(p.dq[:0], p.pages, p.table[:0], p.kv_lens[:0], 32, 16)
    assert e.shape == (0, 4, 64)
    ok = dict(q=p.dq, pages=p.pages, block_table=p.table, kv_lens=p.kv_lens, group=32, page_size=16)
    for b in (dict(q=p.dq.float()), dict(q=p.dq[0]), dict(pages=p.pages[..., :-1]), dict(group=64), dict(page_size=32),
              dict(block_table=p.table[0]), dict(block_table=p.table.long()), dict(kv_lens=p.kv_lens.long()),
              dict(kv_lens=p.kv_lens[:1]), dict(cu_q=p.cu.long()), dict(cu_q=p.cu[:2]), dict(out=p.dq[:1]),
              dict(lse=torch.empty(2, 4, device="cuda", dtype=torch.float64)), dict(q=p.dq.cpu())):
        with pytest.raises(ValueError):
            wq.wq_attn_kv4(**{**ok, **b})
    for b in (dict(q=p.dq[:, :3].contiguous()), dict(window=-1), dict(window=4, causal=False), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(max_q=0), dict(q=p.dq[:1]),
              dict(ws=torch.zeros(64, dtype=torch.uint8, device="cuda")[1:17])):
        with pytest.raises(wq.WQError):
            wq.wq_attn_kv4(**{**ok, **b})


def test_foreign_workspaces_are_refused():
    p = Problem([30, 20], [1, 1], 4, 2, 64, 32, 16, "f16", seed=20)
    call = dict(q=p.dq, pages=p.pages, block_table=p.table, kv_lens=p.kv_lens, group=32, page_size=16)
    for ws in (torch.zeros(1 << 26, dtype=torch.uint8), torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")[::2], 0):
        with pytest.raises(ValueError):
            wq.wq_attn_kv4(**call, ws=ws)


@pytest.mark.parametrize("news", [[1, 1], [100, 200], [9, 210], [350, 12]])   # more queries than tokens, too
def test_windows_beyond_every_length(news):
    p = Problem([300, 200], news, 4, 2, 64, 32, 16, "bf16", seed=21)
    call = dict(q=p.dq, pages=p.pages, block_table=p.table, kv_lens=p.kv_lens, group=32, page_size=16, cu_q=p.cu,
                max_q=max(news))
    whole = wq.wq_attn_kv4(**call)
    for window in (300, (1 << 31) - 1, 1 << 31, (1 << 32) + 5):
        assert torch.equal(wq.wq_attn_kv4(**call, window=window), whole)
