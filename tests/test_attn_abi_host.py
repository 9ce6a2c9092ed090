"""Host-side checks of the entry points between the projections, without a GPU: sizes, and bad arguments
refused before anything touches the device."""
import ctypes

import pytest

import weight_only_quantized_tma_gb300 as wq
from weight_only_quantized_tma_gb300._attn import Kv4Layout

OK, NULL, SHAPE, GROUP, MISALIGNED, DTYPE = range(6)
P = 0x10000     # a 16-byte-aligned fake device address: validation never dereferences it


@pytest.fixture(scope="module")
def L():
    return wq.lib()


def lay(**kw):
    d = dict(num_pages=10, kv_heads=2, head_dim=128, group=64, page_size=32, dtype=0)
    return ctypes.byref(Kv4Layout(*{**d, **kw}.values()))


BAD_LAYOUTS = [(dict(kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE), (dict(group=16), GROUP),
               (dict(head_dim=64, group=128), GROUP), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
               (dict(dtype=2), DTYPE), (dict(num_pages=-1), SHAPE)]


def test_page_bytes(L):
    b = ctypes.c_size_t()
    for D, G, page, H in ((128, 128, 16, 1), (128, 32, 64, 8), (64, 64, 128, 3)):
        assert L.wq_kv4_page_bytes(lay(kv_heads=H, head_dim=D, group=G, page_size=page), ctypes.byref(b)) == OK
        assert b.value == H * page * (D // 2 * 2 + D // G * 4 * 2)
    assert L.wq_kv4_page_bytes(None, ctypes.byref(b)) == NULL
    for kw, status in BAD_LAYOUTS:
        assert L.wq_kv4_page_bytes(lay(**kw), ctypes.byref(b)) == status


def test_rope_refusals(L):
    def f(q=P, qs=512, k=P, ks=256, dt=0, T=4, Hq=4, Hkv=2, D=128, wq_=None, wk=None, eps=1e-6, pos=P, cs=P, most=8,
          rot=128, inter=0, qo=P, qos=512, ko=P, kos=256):
        return L.wq_qk_norm_rope(q, qs, k, ks, dt, T, Hq, Hkv, D, wq_, wk, eps, pos, cs, most, rot, inter, qo, qos, ko,
                                 kos, None)
    for kw in (dict(q=None), dict(k=None), dict(pos=None), dict(cs=None), dict(qo=None), dict(ko=None)):
        assert f(**kw) == NULL
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=12), dict(D=264), dict(rot=4), dict(rot=136), dict(rot=12),
               dict(most=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qs=508), dict(ks=252),
               dict(qos=514), dict(kos=0)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2) == DTYPE
    for kw in (dict(q=P + 4), dict(k=P + 2), dict(qo=P + 4), dict(ko=P + 4), dict(wq_=P + 2), dict(wk=P + 4), dict(pos=P + 4),
               dict(cs=P + 8)):
        assert f(**kw) == MISALIGNED, kw
    assert f(T=0, q=None, k=None) == OK


@pytest.mark.parametrize("write", [True, False])
def test_cache_refusals(L, write):
    def f(k=P, ks=256, v=P, vs=256, slots=P, T=4, l=None, pages=P):
        l = lay() if l is None else l
        if write:
            return L.wq_kv4_write(k, ks, v, vs, slots, T, l, pages, None)
        return L.wq_kv4_read(pages, l, slots, T, k, ks, v, vs, None)
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(pages=None)):
        assert f(**kw) == NULL
    for kw in (dict(T=-1), dict(ks=255), dict(vs=248), dict(ks=260)):
        assert f(**kw) == SHAPE
    for kw in (dict(k=P + 8), dict(v=P + 2), dict(slots=P + 4), dict(pages=P + 8)):
        assert f(**kw) == MISALIGNED
    for kw, status in BAD_LAYOUTS:
        assert f(l=lay(**kw)) == status
    assert f(T=0, k=None) == OK


def test_attention_refusals(L):
    def f(q=P, qs=512, Hq=4, cu=P, B=2, T=4, mq=2, pages=P, l=None, table=P, ts=8, lens=P, scale=1.0, causal=1, window=0,
          out=P, os_=512, lse=None, ws=None, wb=0):
        return L.wq_attn_kv4(q, qs, Hq, cu, B, T, mq, pages, lay() if l is None else l, table, ts, lens, scale, causal,
                             window, out, os_, lse, ws, wb, None)
    for kw in (dict(q=None), dict(pages=None), dict(table=None), dict(lens=None), dict(out=None)):
        assert f(**kw) == NULL
    for kw in (dict(Hq=3), dict(Hq=0), dict(B=-1), dict(T=-1), dict(mq=0), dict(ts=-1), dict(window=-1),
               dict(window=5, causal=0), dict(scale=float("nan")), dict(cu=None), dict(qs=504), dict(qs=516),
               dict(os_=256)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=P + 8), dict(out=P + 8), dict(pages=P + 8), dict(cu=P + 2), dict(table=P + 2), dict(lens=P + 1),
               dict(lse=P + 2), dict(ws=P + 8)):
        assert f(**kw) == MISALIGNED, kw
    for kw, status in BAD_LAYOUTS:
        assert f(l=lay(**kw)) == status
    assert f(T=0, cu=None, B=0, q=None) == OK


def test_row_numbers_stay_within_31_bits(L):
    """Rows (a token's head) are counted in 32 bits on the device: more of them are refused, not wrapped."""
    T = 1 << 30     # two heads of each token: 2^31 rows
    assert L.wq_qk_norm_rope(P, 128, P, 128, 0, T, 1, 1, 128, None, None, 1e-6, P, P, 8, 128, 0, P, 128, P, 128, None) == SHAPE
    assert L.wq_kv4_write(P, 256, P, 256, P, T, lay(), P, None) == SHAPE
    assert L.wq_kv4_read(P, lay(), P, T, P, 256, P, 256, None) == SHAPE
    assert L.wq_attn_kv4(P, 512, 4, P, 2, T, T, P, lay(), P, 8, P, 1.0, 1, 0, P, 512, None, None, 0, None) == SHAPE


def test_scales_whose_logarithmic_form_overflows_are_refused(L):
    """The kernels work with scale * log2(e) in fp32."""
    def f(scale):   # (a misaligned out where the scale passes: nothing reaches the device)
        return L.wq_attn_kv4(P, 512, 4, P, 2, 4, 2, P, lay(), P, 8, P, scale, 1, 0, P + 8, 512, None, None, 0, None)
    for scale in (2.0 ** 127 * 1.001, -3e38, float("inf"), float("nan")):
        assert f(scale) == SHAPE
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0, 1e-45):
        assert f(scale) == MISALIGNED
