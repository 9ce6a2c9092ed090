"""The operators between the projections of an attention layer, as cases to time and compare.

Three operators that a decoder layer runs between its weight-only quantized projections:

* "rope"   norms of queries and keys for each head, and their rotation by position, in one pass
           (wq_qk_norm_rope);
* "cache"  keys and values quantised to 4 bits as they are written into a paged cache, and read back
           (wq_kv4_write, wq_kv4_read); "read" cases only read back;
* "attn"   attention of the queries over that cache (wq_attn_kv4): single tokens, short drafts, long
           prompts, one length for each sequence.

A cache is a uint8 tensor [pages][kv heads][bytes], one block for each page of P tokens and each head:
key codes [P][D / 2], value codes [P][D / 2] (even d in the low nibble), then for keys and for values the
pairs (s, lo) [P][D / G][2] in the 16-bit type of the keys.  A code q stands for lo + q s, rounded to that
type; lo is the least value of its group of G and s the 16-bit number nearest to the range / 15.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of 16 sequences, grouped heads: latency
        dict(name="rope_decode", kind="rope", dtype="bf16", T=16, Hq=32, Hkv=8, D=128, rot=128, inter=False, norm=True),
        # a prompt at the 4096-wide layer's 32 + 32 heads, read out of the packed 12288-wide projection
        dict(name="rope_prompt", kind="rope", dtype="f16", T=8192, Hq=32, Hkv=32, D=128, rot=128, inter=False, norm=True),
        # half of each head rotated, neighbouring pairs, no norm, an odd number of tokens
        dict(name="rope_part", kind="rope", dtype="bf16", T=1777, Hq=14, Hkv=2, D=64, rot=32, inter=True, norm=False),
        # one new token of each of 64 sequences goes into the cache
        dict(name="cache_decode", kind="cache", dtype="bf16", T=64, Hkv=8, D=128, G=128, P=16),
        # a whole prompt goes into the cache, all 32 heads, finer groups
        dict(name="cache_prompt", kind="cache", dtype="f16", T=16384, Hkv=32, D=128, G=64, P=64),
        # a stored prefix is read back for a path that wants 16-bit keys and values
        dict(name="read_prefix", kind="read", dtype="bf16", T=50001, Hkv=8, D=128, G=32, P=32),
        # the first steps of a single conversation: latency
        dict(name="attn_one_short", kind="attn", dtype="bf16", B=1, n=1, Lmin=777, Lmax=777, Hq=32, Hkv=8, D=128, G=128, P=16, window=0),
        # a serving batch of 64 sequences of unequal lengths
        dict(name="attn_batch", kind="attn", dtype="bf16", B=64, n=1, Lmin=300, Lmax=16384, Hq=32, Hkv=8, D=128, G=128, P=64, window=0),
        # the 4096-wide layer: every query head has its own keys
        dict(name="attn_heads", kind="attn", dtype="f16", B=16, n=1, Lmin=4096, Lmax=4096, Hq=32, Hkv=32, D=128, G=64, P=32, window=0),
        # one very long context
        dict(name="attn_long", kind="attn", dtype="bf16", B=1, n=1, Lmin=131072, Lmax=131072, Hq=32, Hkv=8, D=128, G=128, P=128, window=0),
        # drafts of 5 tokens checked at once, narrow heads, a sliding window
        dict(name="attn_draft", kind="attn", dtype="f16", B=24, n=5, Lmin=33, Lmax=6001, Hq=28, Hkv=4, D=64, G=32, P=16, window=4096),
        # a chunk of a long prompt
        dict(name="attn_prompt", kind="attn", dtype="bf16", B=1, n=4096, Lmin=16384, Lmax=16384, Hq=32, Hkv=8, D=128, G=128, P=64, window=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "read", "attn", "attn", "attn"])
    D = rng.choice([64, 128, 128])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "f16"]))
    if kind == "rope":
        Hkv = rng.choice([1, 2, 4, 8, 16, 32])
        rot = rng.choice([D, D, D // 2, D // 4])
        return dict(c, T=_spread(rng, 1, 8192), Hq=Hkv * rng.randint(1, max(1, 32 // Hkv)), Hkv=Hkv, D=D, rot=rot,
                    inter=rng.random() < 0.4, norm=rng.random() < 0.7)
    G = rng.choice([g for g in (32, 64, 128) if g <= D])
    P = rng.choice([16, 32, 64, 128])
    if kind in ("cache", "read"):
        return dict(c, T=_spread(rng, 1, 16384), Hkv=rng.choice([1, 2, 4, 8, 16, 32]), D=D, G=G, P=P)
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * Hkv <= 32])
    form = rng.choice(["one", "batch", "draft", "prompt"])
    if form == "one":
        B, n, Lmax = 1, 1, _spread(rng, 1, 100000)
    elif form == "batch":
        B, n = _spread(rng, 2, 64), 1
        Lmax = _spread(rng, 16, min(16384, 500000 // B))
    elif form == "draft":
        B, n = _spread(rng, 1, 32), rng.randint(2, 16)
        Lmax = _spread(rng, 64, min(16384, 200000 // B))
    else:
        B, n = rng.randint(1, 3), _spread(rng, 33, 1300)
        Lmax = n + _spread(rng, 1, 12000)
    Lmin = max(1, int(Lmax * rng.uniform(0.1, 1.0)))
    window = _spread(rng, 16, 4096) if rng.random() < 0.25 else 0
    return dict(c, B=B, n=n, Lmin=Lmin, Lmax=Lmax, Hq=Hq, Hkv=Hkv, D=D, G=G, P=P, window=window)


def _lens(case):
    """Each sequence's length, spread from Lmin to Lmax in no order."""
    B, lo, hi = case["B"], case["Lmin"], case["Lmax"]
    return [hi - (hi - lo) * ((b * 7919) % B) // max(1, B - 1) for b in range(B)]


def _news(case):
    """Each sequence's new tokens: single tokens and chunks of one prompt alike, else unequal."""
    B, n = case["B"], case["n"]
    return [n if B == 1 or n == 1 else max(1, n - (b % 3)) for b in range(B)]


# ---------------------------------------------------------------------------------------- inputs

def _block_bytes(P, D, G):
    return P * D + 8 * P * (D // G)


def _keys_and_values(gen, T, Hkv, D, dtype):
    """Keys with a few strong channels and a bias for each channel, as trained layers have them; plain values."""
    gain = torch.ones(Hkv, D, device="cuda")
    gain[:, :: max(1, D // 4)] = 4.0
    bias = torch.randn(Hkv, D, device="cuda", generator=gen) * 0.5
    k = torch.randn(T, Hkv, D, device="cuda", generator=gen).mul_(gain).add_(bias).to(dtype)
    v = torch.randn(T, Hkv, D, device="cuda", generator=gen).to(dtype)
    return k, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    s = dict(case=case, kind=kind)
    if kind == "rope":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        # the packed projection: queries, keys and values of a token in one row
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda", generator=gen).mul_(1.5).to(dtype)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        most = 2 * T + 64
        s["positions"] = torch.randint(0, most, (T,), device="cuda", generator=gen)
        inv = 1.0 / 10000.0 ** (torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        ang = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["wq"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).to(dtype) if case["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).to(dtype) if case["norm"] else None
        return s
    G, P = case["G"], case["P"]
    if kind in ("cache", "read"):
        T = case["T"]
        pages = -(-T // P) + 3
        s["pages"] = torch.zeros(pages, Hkv, _block_bytes(P, D, G), dtype=torch.uint8, device="cuda")
        # a prompt's tokens follow one another inside pages that lie anywhere; a decode batch's lie apart
        place = torch.randperm(pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        if T <= pages:
            s["slots"] = place[t] * P + torch.randint(0, P, (T,), device="cuda", generator=gen)
        else:
            s["slots"] = place[t // P] * P + t % P
        s["k"], s["v"] = _keys_and_values(gen, T, Hkv, D, dtype)
        if kind == "read":
            _store(s["pages"], s["slots"], s.pop("k"), s.pop("v"), G, P)
        return s
    lens, news = _lens(case), _news(case)
    B, Hq = case["B"], case["Hq"]
    need = [max(1, -(-x // P)) for x in lens]
    place = torch.randperm(sum(need) + 2, device="cuda", generator=gen).to(torch.int32)
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, : need[b]] = place[at: at + need[b]]
        at += need[b]
    s["pages"] = torch.zeros(sum(need) + 2, Hkv, _block_bytes(P, D, G), dtype=torch.uint8, device="cuda")
    for b in range(B):
        t = torch.arange(lens[b], device="cuda")
        k, v = _keys_and_values(gen, lens[b], Hkv, D, dtype)
        _store(s["pages"], table[b].long()[t // P] * P + t % P, k, v, G, P)
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([0] + [sum(news[: b + 1]) for b in range(B)], dtype=torch.int32, device="cuda")
    s["max_q"] = max(news)
    s["q"] = torch.randn(sum(news), Hq, D, device="cuda", generator=gen).to(dtype)
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _quantise(x, G):
    """codes, s and lo of groups of G along the last axis; every step a 32-bit operation."""
    g = x.float().unflatten(-1, (-1, G))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / torch.full_like(lo, 15.0)).to(x.dtype)
    step = s.float().unsqueeze(-1)
    q = torch.where(step > 0, ((g - lo.unsqueeze(-1)) / step).round(), torch.zeros_like(g)).clamp_(0, 15)
    return q.flatten(-2).to(torch.uint8), s, lo.to(x.dtype)


def _regions(pages, D, G, P, dtype):
    """Views of a cache: codes of keys and of values [pages][heads][P][D / 2], then (s, lo) [..][P][D / G][2]."""
    n, h = pages.shape[:2]
    c, r = P * D // 2, 4 * P * (D // G)
    kc, vc = pages[:, :, :c].unflatten(-1, (P, D // 2)), pages[:, :, c: 2 * c].unflatten(-1, (P, D // 2))
    par = pages[:, :, 2 * c:].view(dtype).unflatten(-1, (2, P, D // G, 2))
    return kc, vc, par[:, :, 0], par[:, :, 1]


def _store(pages, slots, k, v, G, P):
    """Quantises k and v [T][heads][D] into their slots."""
    D = k.shape[-1]
    page, off = slots // P, slots % P
    kc, vc, kp, vp = _regions(pages, D, G, P, k.dtype)
    for x, codes, pairs in ((k, kc, kp), (v, vc, vp)):
        q, s, lo = _quantise(x, G)
        codes[page, :, off] = q[..., 0::2] | (q[..., 1::2] << 4)
        pairs[page, :, off] = torch.stack([s, lo], -1)


def _values(codes, pairs):
    """The 32-bit values [...][D] of packed codes [...][D / 2] and their (s, lo) [...][D / G][2], rounded to the pairs' type."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    s, lo = pairs.float().unbind(-1)
    G = q.shape[-1] // s.shape[-1]
    return (q.unflatten(-1, (-1, G)) * s.unsqueeze(-1) + lo.unsqueeze(-1)).flatten(-2).to(pairs.dtype).float()


def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    cs = s["cos_sin"][s["positions"]].unsqueeze(1)
    cos, sin = cs[..., :half], cs[..., half:]

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["inter"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _plain_read(s):
    c = s["case"]
    dtype = TYPES[c["dtype"]]
    page, off = s["slots"] // c["P"], s["slots"] % c["P"]
    kc, vc, kp, vp = _regions(s["pages"], c["D"], c["G"], c["P"], dtype)
    return {"k": _values(kc[page, :, off], kp[page, :, off]).to(dtype),
            "v": _values(vc[page, :, off], vp[page, :, off]).to(dtype)}


def _plain_attn(s):
    c = s["case"]
    D, Hq, Hkv, dtype = c["D"], c["Hq"], c["Hkv"], TYPES[c["dtype"]]
    q, table, lens, cu = s["q"], s["table"].long(), s["lens"].long(), s["cu_q"].long()
    B, N, T = len(lens), s["max_q"], len(q)
    kc, vc, kp, vp = _regions(s["pages"], D, c["G"], c["P"], dtype)

    def all_tokens(codes, pairs):   # [B][heads][table's tokens][D]
        return _values(codes[table], pairs[table]).transpose(1, 2).flatten(2, 3)

    # queries padded to the most new tokens: [B][kv heads][N x group][D]
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    padded = torch.zeros(B, N, Hq, D, device=q.device)
    padded[b, i] = q.float()
    rows = padded.view(B, N, Hkv, Hq // Hkv, D).transpose(1, 2).flatten(2, 3)
    score = rows @ all_tokens(kc, kp).transpose(-1, -2)
    score *= 1.0 / math.sqrt(D)
    j = torch.arange(score.shape[-1], device=q.device)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(N, device=q.device)   # [B][N]
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(B, 1, N, Hq // Hkv, len(j)).flatten(2, 3)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    o = score @ all_tokens(vc, vp)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.unflatten(2, (N, Hq // Hkv)).transpose(1, 2).flatten(2, 3)
    return {"out": o[b, i].to(dtype)}


def run(s):
    c, kind = s["case"], s["kind"]
    if not own:
        if kind == "cache":
            _store(s["pages"], s["slots"], s["k"], s["v"], c["G"], c["P"])
        return _plain_rope(s) if kind == "rope" else _plain_attn(s) if kind == "attn" else _plain_read(s)
    import weight_only_quantized_tma_gb300 as wq
    if kind == "rope":
        q, k = wq.wq_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"],
                                  eps=1e-6, interleaved=c["inter"])
        return {"q": q, "k": k}
    if kind == "attn":
        return {"out": wq.wq_attn_kv4(s["q"], s["pages"], s["table"], s["lens"], c["G"], c["P"], cu_q=s["cu_q"],
                                      max_q=s["max_q"], window=c["window"])}
    if kind == "cache":
        wq.wq_kv4_write(s["k"], s["v"], s["slots"], s["pages"], c["G"], c["P"])
    k, v = wq.wq_kv4_read(s["pages"], s["slots"], c["D"], c["G"], c["P"], TYPES[c["dtype"]])
    return {"k": k, "v": v}


# ---------------------------------------------------------------------------------------- work

def work(case):
    kind, D, Hkv = case["kind"], case["D"], case["Hkv"]
    if kind == "rope":
        T, heads = case["T"], case["Hq"] + Hkv
        # rows in and out, a position and its cos and sin for each token, the weights
        return {"bytes": T * heads * D * 4 + T * (8 + 4 * case["rot"]) + (4 * D if case["norm"] else 0),
                "flops": T * heads * D * (7 if case["norm"] else 3)}
    token = 2 * Hkv * (D // 2 + 4 * (D // case["G"]))   # a token's codes and pairs, keys and values
    if kind in ("cache", "read"):
        T, rows = case["T"], 4 * case["T"] * Hkv * D
        return {"bytes": T * (token + 8) + (2 * rows if kind == "cache" else rows),
                "flops": T * Hkv * D * (12 if kind == "cache" else 4)}
    pairs = seen = 0
    for L, n in zip(_lens(case), _news(case)):
        w = case["window"] or L
        first = max(0, L - n + 1 - w)   # the first token that the first new token sees
        seen += L - first
        for i in range(n):
            pairs += max(0, min(w, L - n + i + 1))
    T = sum(_news(case))
    return {"bytes": seen * token + T * case["Hq"] * D * 4 + 4 * sum(-(-x // case["P"]) for x in _lens(case)),
            "flops": 4 * D * case["Hq"] * pairs}


# ---------------------------------------------------------------------------------------- in 64 bits

def _exact_values(s, which, slots):
    """The values [len(slots)][heads][D] that the cache holds of keys (0) or values (1), from its bytes."""
    c = s["case"]
    D, G, P, dtype = c["D"], c["G"], c["P"], TYPES[c["dtype"]]
    block = s["pages"][slots // P]                                     # [T][heads][bytes]
    T, H, size = block.shape
    off = (slots % P).view(T, 1, 1)
    d = torch.arange(D, device=block.device).view(1, 1, D)
    byte = block.gather(2, (which * (P * D // 2) + off * (D // 2) + d // 2).expand(T, H, D)).to(torch.int32)
    q = torch.where(d % 2 == 0, byte % 16, byte // 16).double()
    pair = block.view(torch.int16).view(dtype)                         # 16-bit words
    at = (P * D + which * 4 * P * (D // G)) // 2 + (off * (D // G) + d // G) * 2
    step = pair.gather(2, at.expand(T, H, D)).double()
    low = pair.gather(2, (at + 1).expand(T, H, D)).double()
    return (low + q * step).to(dtype).double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, D = case["kind"], case["D"]
    dtype = TYPES[case["dtype"]]
    if kind == "rope":
        rot, half = case["rot"], case["rot"] // 2
        turn = s["cos_sin"].double()[s["positions"]]
        z = torch.complex(turn[:, :half], turn[:, half:])[:, None]
        out = {}
        for name in ("q", "k"):
            x, w = s[name].double(), s["w" + name]
            if w is not None:
                x = x / ((x * x).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            p = x[..., :rot].unflatten(-1, (half, 2)) if case["inter"] else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(p.contiguous()) * z)
            y = y.flatten(-2) if case["inter"] else y.transpose(-1, -2).flatten(-2)
            out[name] = torch.cat([y, x[..., rot:]], -1)
        return out
    if kind == "read":
        return {"k": _exact_values(s, 0, s["slots"]), "v": _exact_values(s, 1, s["slots"])}
    if kind == "cache":
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            G = case["G"]
            parts = []
            for g in range(D // G):
                y = x[..., g * G: (g + 1) * G]
                low = y.min(-1, keepdim=True).values
                step = ((y.max(-1, keepdim=True).values - low) / 15.0).to(dtype).double()
                q = torch.floor((y - low) / step.clamp(min=1e-300) + 0.5)
                even = ((y - low) / step.clamp(min=1e-300) + 0.5 == q) & (q % 2 == 1)   # halves go to even
                q = torch.where(step > 0, (q - even.double()).clamp(0, 15), torch.zeros_like(q))
                parts.append((low + q * step).to(dtype).double())
            out[name] = torch.cat(parts, -1)
        return out
    lens, news = _lens(case), _news(case)
    if work(case)["flops"] > 3e12:
        return None
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["P"]
    group, out, first = Hq // Hkv, [], 0
    for b, (L, n) in enumerate(zip(lens, news)):
        t = torch.arange(L, device="cuda")
        slots = s["table"][b].long()[t // P] * P + t % P
        K, V = _exact_values(s, 0, slots), _exact_values(s, 1, slots)   # [L][Hkv][D]
        Q = s["q"][first: first + n].double()
        first += n
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        hide = (t > pos) | ((t <= pos - case["window"]) if case["window"] else torch.zeros_like(t > pos))
        o = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            a = (Q[:, h] @ K[:, h // group].T / math.sqrt(D)).masked_fill(hide, -math.inf)
            p = torch.exp(a - torch.logsumexp(a, -1, keepdim=True)).nan_to_num(0.0)
            o[:, h] = p @ V[:, h // group]
        out.append(o)
    return {"out": torch.cat(out)}
