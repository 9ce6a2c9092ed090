"""Plain 64-bit forms of the operators between the projections of an attention layer
(not collected as tests): norm + rotation, the 4-bit cache byte by byte, attention."""
import math

import numpy as np
import torch

# significant bits, exponent of the smallest step
FORMATS = {"f16": (11, -24), "bf16": (8, -133)}
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def unit(dtype):
    """Largest relative error of one rounding to the type."""
    return 2.0 ** -FORMATS[dtype][0]


def round16(x, dtype):
    """Round float64 to the type, half to even, in one rounding (no overflow handling)."""
    p, qmin = FORMATS[dtype]
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - p, qmin))
    return np.rint(x / step) * step


def to_bits(x, dtype):
    """float64 values that the type holds exactly -> their 16-bit patterns."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])
    return t.view(torch.int16).numpy()


def random16(rng, shape, dtype, scale=1.0):
    return round16(rng.standard_normal(shape) * scale, dtype)


def on_gpu(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype]).cuda()


# ------------------------------------------------------------------ norm + rotation

def norm_rope(x, pos, cos_sin, rot, interleaved, w=None, eps=1e-6):
    """x [T][H][D] float64; cos_sin [max_pos][rot] -> float64 [T][H][D]."""
    x = x.copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    cos, sin = cos_sin[pos, None, : rot // 2], cos_sin[pos, None, rot // 2:]
    a = x[..., 0:rot:2].copy() if interleaved else x[..., : rot // 2].copy()
    b = x[..., 1:rot:2].copy() if interleaved else x[..., rot // 2: rot].copy()
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = ra, rb
    else:
        x[..., : rot // 2], x[..., rot // 2: rot] = ra, rb
    return x


# ------------------------------------------------------------------ the cache

def quantise(x, G, dtype):
    """x float64 [..., D] -> codes uint8 [..., D], s, lo float64 [..., D / G]."""
    g = x.reshape(x.shape[:-1] + (-1, G))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        s = round16((hi - lo) / 15.0, dtype)
        ratio = np.where(s[..., None] > 0, (g - lo[..., None]) / np.where(s > 0, s, 1.0)[..., None], 0.0)
        q = np.clip(np.rint(ratio), 0, 15)
    bad = ~np.isfinite(g).all(-1)
    s, lo = np.where(bad, np.nan, s), np.where(bad, np.nan, lo)
    q = np.where(bad[..., None], 0, q)
    return q.reshape(x.shape).astype(np.uint8), s, lo


def values(q, s, lo, dtype):
    G = q.shape[-1] // s.shape[-1]
    q = q.reshape(q.shape[:-1] + (-1, G)).astype(np.float64)
    return round16(lo[..., None] + q * s[..., None], dtype).reshape(q.shape[:-2] + (-1,))


class Cache:
    """The cache as bytes, filled and read element by element in numpy."""

    def __init__(self, num_pages, H, D, G, P, dtype):
        self.H, self.D, self.G, self.P, self.dtype = H, D, G, P, dtype
        self.block = P * (D + 8 * (D // G))
        self.bytes = np.zeros((num_pages, H, self.block), dtype=np.uint8)

    def _at(self, which, place):
        c, r = self.D // 2, 4 * (self.D // self.G)
        code = (which * self.P + place) * c
        pair = self.P * self.D + (which * self.P + place) * r
        return slice(code, code + c), slice(pair, pair + r)

    def put(self, slot, k, v):
        """k, v float64 [H][D]."""
        page, place = divmod(int(slot), self.P)
        for which, x in ((0, k), (1, v)):
            q, s, lo = quantise(x, self.G, self.dtype)
            codes, pairs = self._at(which, place)
            self.bytes[page, :, codes] = q[:, 0::2] | (q[:, 1::2] << 4)
            self.bytes[page, :, pairs] = to_bits(np.stack([s, lo], -1), self.dtype).reshape(self.H, -1).view(np.uint8)

    def get(self, slot):
        page, place = divmod(int(slot), self.P)
        out = []
        for which in (0, 1):
            codes, pairs = self._at(which, place)
            b = self.bytes[page, :, codes]
            q = np.stack([b & 15, b >> 4], -1).reshape(self.H, self.D)
            pr = torch.from_numpy(self.bytes[page, :, pairs].copy()).view(TORCH[self.dtype]).double().numpy()
            pr = pr.reshape(self.H, -1, 2)
            out.append(values(q, pr[..., 0], pr[..., 1], self.dtype))
        return out

    def pages(self):
        return torch.from_numpy(self.bytes).cuda()


# ------------------------------------------------------------------ attention

def attention(q, K, V, scale, n, causal=True, window=0):
    """One sequence: q [n][Hq][D], K, V [L][Hkv][D] -> out, lse and A = sum softmax |v| (error bounds)."""
    Hq, D = q.shape[1:]
    L, Hkv = K.shape[:2]
    pos = np.arange(L - n, L)[:, None]
    j = np.arange(L)[None]
    see = (j <= pos) if causal else np.ones((n, L), bool)
    if window:
        see &= j > pos - window
    out, lse, A = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    if L == 0:
        return out, lse, A
    for h in range(Hq):
        k, v = K[:, h // (Hq // Hkv)], V[:, h // (Hq // Hkv)]
        for i in range(n):
            vis = see[i]
            if not vis.any():
                continue
            s = k[vis] @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            out[i, h] = p @ v[vis] / p.sum()
            A[i, h] = p @ np.abs(v[vis]) / p.sum()
            lse[i, h] = m + math.log(p.sum())
    return out, lse, A


def attention_bound(dtype, A, L, vmax):
    """|out - exact|: one rounding of the result and one of each probability (both relative u, each at most
    u A), a quarter more for the fp32 scores and sums; fp16 probabilities below 2^-14 keep steps of 2^-24."""
    return 2.5 * unit(dtype) * A + (L * 2.0 ** -25 * vmax if dtype == "f16" else 0.0) + 2.0 ** -24
