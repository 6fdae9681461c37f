"""Pins of the 64-bit reference of the cache, attention and verification (no GPU): worked values of the
two element types, ties, the exponent rule, the layout as a permutation, attention and verification
in cases with known answers; and the refusals of the C entry points, decided before any device work."""
import ctypes as C

import numpy as np
import pytest

import step_reference as ref
from step_reference import MXFP4, MXFP8


def block(values):
    x = np.zeros(32)
    x[:len(values)] = values
    return x


def test_e2m1_nearest_and_ties():
    # 6 fixes the exponent at 127; ties go to the even code
    x = block([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, -0.25, -5.1, -0.0])
    code, b = ref.encode(x, MXFP4)
    assert b[0] == 127
    assert code[:12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 1, 8, 15, 8]


def test_e4m3_nearest_and_ties():
    x = block([448, 432.0, 17.0, 19.0, 2.0 ** -10, 2.0 ** -9, 1.5 * 2.0 ** -9, -1.0])
    code, b = ref.encode(x, MXFP8)
    assert b[0] == 127
    assert ref.decode(code, b, MXFP8)[:8].tolist() == [448, 448, 16, 20, 0, 2.0 ** -9, 2.0 ** -8, -1.0]


@pytest.mark.parametrize("fmt,largest", [(MXFP8, 448.0), (MXFP4, 6.0)])
def test_exponent_rule(fmt, largest):
    assert ref.encode(block([largest]), fmt)[1][0] == 127
    assert ref.encode(block([np.nextafter(np.float32(largest), np.float32(1e9))]), fmt)[1][0] == 128
    assert ref.encode(block([largest / 2]), fmt)[1][0] == 126
    assert ref.encode(block([0.0]), fmt)[1][0] == 16
    assert ref.encode(block([1e-45]), fmt)[1][0] == 16
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 127, -2.0 ** 127.5):
        code, b = ref.encode(block([1.0, bad]), fmt)
        assert b[0] == 255 and not code.any() and np.isnan(ref.decode(code, b, fmt)).all()
    assert ref.encode(block([np.nextafter(np.float32(2.0 ** 127), np.float32(0))]), fmt)[1][0] != 255


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layout_uses_every_byte_once(fmt, dim):
    k, v, ek, ev = ref.places(fmt, dim)
    codes = np.sort(np.concatenate([k.ravel(), v.ravel()]))
    assert np.array_equal(codes, np.arange(64 * dim))
    exps = np.sort(np.concatenate([ek[:, ::32].ravel(), ev[:, ::32].ravel()]))
    first = codes.size if fmt == MXFP8 else codes.size // 2
    assert np.array_equal(exps, np.arange(first, ref.record_bytes(fmt, dim)))


def test_write_then_read_gives_the_rounded_numbers():
    rng = np.random.default_rng(3)
    for fmt in (MXFP8, MXFP4):
        c = ref.Cache(fmt, 2, 64, 32, 3, fill=0xFF)
        k, v = rng.normal(size=(2, 5, 2, 64))
        slots = [70, 3, -1, 96, 31]
        c.write(k, v, slots)
        rk, rv = c.read(slots)
        for x, r in ((k, rk), (v, rv)):
            want = ref.decode(*ref.encode(x, fmt), fmt)
            assert np.array_equal(r[[0, 1, 4]], want[[0, 1, 4]])
            assert not r[[2, 3]].any()
            step = 2.0 ** -4 if fmt == MXFP8 else 0.25
            assert np.abs(want - x).max() <= step * np.abs(x).max()


def test_attention_of_equal_scores_is_the_mean():
    c = ref.Cache(MXFP8, 1, 64, 32, 2)
    v = np.arange(1.0, 4.0)[:, None, None] * np.ones((3, 1, 64))
    c.write(np.zeros((3, 1, 64)), v, [0, 32, 33])
    q = np.ones((1, 2, 2, 64))
    out, lse, _, _, count = ref.attend(c, q, np.array([[1]]), [2], [0], 1, 0.125)
    assert count.tolist() == [[2, 3]]
    assert np.allclose(out[0, 0], 1.5) and np.allclose(out[0, 1], 2.0)
    assert np.allclose(lse[0, :, 0], np.log([2, 3]))


def test_verification_by_hand():
    p = np.array([[[0.5, 0.25, 0.25, 0.0], [0.0, 0.0, 0.25, 0.75]]], np.float32)
    q = np.array([[[0.25, 0.75, 0.0, 0.0]]], np.float32)

    def one(x, ua, us, q=q):
        t, a = ref.verify(p, q, np.array([[x]]), np.array([[ua]]), np.array([us]))
        return t[0].tolist(), int(a[0])
    assert one(0, 0.99, 0.2) == ([0, 2], 1)       # accepted, then p_1 by inversion
    assert one(0, 0.99, 0.25) == ([0, 3], 1)      # the sum has to pass, not reach
    assert one(1, 0.34, 0.0) == ([0, -1], 0)      # 0.34 * 0.75 > 0.25: refused; r = (0.25, 0, 0.25, 0)
    assert one(1, 0.34, 0.5) == ([2, -1], 0)
    assert one(1, 0.33, 0.0) == ([1, 2], 1)
    assert one(9, 0.0, 0.0) == ([0, -1], 0)       # not a token
    assert one(0, 0.6, 0.0, q=None) == ([1, -1], 0)
    assert one(0, 0.4, 0.0, q=None) == ([0, 2], 1)


# ---- refusals -----------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def pn():
    import block_quantized_weight_pn3t_amd as pn
    return pn


FAKE = 0x1000  # never dereferenced: every call fails its checks or is a no-op


def desc(pn, format=0, heads=4, dim=128, page=64, pages=8, data=FAKE):
    return pn.CacheDesc(format, heads, dim, page, pages, data)


def test_page_bytes(pn):
    assert pn.cache_page_bytes(MXFP8, 4, 256, 64) == 4 * 2 * 66 * 256
    assert pn.cache_page_bytes(MXFP4, 3, 64, 1024) == 3 * 32 * 34 * 64
    for bad in ((2, 4, 128, 64), (-1, 4, 128, 64), (0, 0, 128, 64), (0, 4, 96, 64), (0, 4, 512, 64),
                (0, 4, 128, 16), (0, 4, 128, 48), (0, 4, 128, 2048), (0, 4, 128, 0), (0, 4, 128, -64),
                (0, 65537, 128, 64)):
        assert pn.cache_page_bytes(*bad) == 0, bad


BAD_CACHES = [(dict(format=2), -9), (dict(heads=0), -2), (dict(dim=96), -2), (dict(page=16), -2),
              (dict(page=96), -2), (dict(pages=-1), -2), (dict(pages=1 << 40), -2), (dict(data=0), -4),
              (dict(data=FAKE + 8), -5)]


def test_cache_write_and_read_refusals(pn):
    L = pn.lib()

    def write(c=None, type=0, k=FAKE, v=FAKE, slots=FAKE, T=3):
        c = desc(pn) if c is None else c
        return L.pn_cache_write(C.byref(c) if c else None, type, k, 512, 128, v, 512, 128, slots, T, None)

    def read(c=None, type=0, k=FAKE, v=FAKE, slots=FAKE, T=3):
        c = desc(pn) if c is None else c
        return L.pn_cache_read(C.byref(c) if c else None, type, slots, T, k, v, None)
    for f in (write, read):
        for kw, st in BAD_CACHES:
            assert f(desc(pn, **kw)) == st, (f.__name__, kw)
        assert f(c=False) == -4
        assert f(type=3) == -9 and f(type=-1) == -9
        assert f(T=-1) == -2 and f(T=1 << 50) == -2
        assert f(T=0) == 0
        assert f(k=None) == -4 and f(v=None) == -4 and f(slots=None) == -4
        assert f(slots=FAKE + 4) == -5
    assert write(k=FAKE + 2) == -5 and write(type=1, v=FAKE + 1) == -5
    assert read(k=FAKE + 4) == -5 and read(type=1, v=FAKE + 4) == -5


def attend_args(pn, **kw):
    a = dict(type=1, B=2, Q=3, Hq=8, q=FAKE, q_seq_stride=3 * 1024, q_token_stride=1024, q_head_stride=128,
             scale=0.1, table=FAKE, table_stride=4, table_width=4, lens=FAKE, q_lens=None, prefix_table=FAKE,
             prefix_len=100, out=FAKE, lse=FAKE)
    a.update(kw)
    return pn.AttendArgs(**a)


def test_attend_refusals(pn):
    L = pn.lib()
    big = 1 << 40

    def call(c=None, ws=FAKE, ws_bytes=big, **kw):
        c = desc(pn) if c is None else c
        return L.pn_attend(C.byref(c), C.byref(attend_args(pn, **kw)), ws, ws_bytes, None)
    for kw, st in BAD_CACHES:
        assert call(desc(pn, **kw)) == st, kw
    assert L.pn_attend(None, C.byref(attend_args(pn)), FAKE, big, None) == -4
    assert L.pn_attend(C.byref(desc(pn)), None, FAKE, big, None) == -4
    assert call(type=3) == -9
    for kw in (dict(B=-1), dict(Q=-1), dict(Hq=0), dict(Hq=6), dict(table_width=-1), dict(prefix_len=-1),
               dict(prefix_len=1 << 31), dict(table_width=1 << 26), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(B=1 << 20, Q=1 << 10)):
        assert call(**kw) == -2, kw
    assert call(desc(pn, pages=0)) == -2
    assert call(B=0) == 0 and call(Q=0) == 0
    for name in ("q", "out", "lens", "table", "prefix_table"):
        assert call(**{name: None}) == -4, name
    assert call(q=FAKE + 1) == -5 and call(type=0, q=FAKE + 2) == -5 and call(out=FAKE + 8) == -5
    for name in ("lens", "table", "prefix_table", "q_lens", "lse"):
        assert call(**{name: FAKE + 2}) == -5, name
    need = L.pn_attend_workspace_bytes(C.byref(desc(pn)), C.byref(attend_args(pn)))
    assert need > 0
    assert call(ws_bytes=need - 1) == -10 and call(ws=None) == -4 and call(ws=FAKE + 8) == -5
    for kw in (dict(Hq=6), dict(B=0), dict(Q=0)):
        assert L.pn_attend_workspace_bytes(C.byref(desc(pn)), C.byref(attend_args(pn, **kw))) == 0
    assert L.pn_attend_workspace_bytes(C.byref(desc(pn)), None) == 0
    assert L.pn_attend_workspace_bytes(None, C.byref(attend_args(pn))) == 0
    for kw in (dict(table_width=0), dict(prefix_len=0), dict(table_width=0, prefix_len=0), dict(B=1, Q=1, Hq=4)):
        assert L.pn_attend_workspace_bytes(C.byref(desc(pn)), C.byref(attend_args(pn, **kw))) >= 0


def test_verify_refusals(pn):
    L = pn.lib()
    big = 1 << 40

    def call(type=0, p=FAKE, q=FAKE, draft=FAKE, n_draft=None, ua=FAKE, us=FAKE, B=2, K=3, V=1000, tokens=FAKE,
             accepted=FAKE, ws=FAKE, ws_bytes=big):
        return L.pn_verify(type, p, V, q, V, draft, n_draft, ua, us, B, K, V, tokens, accepted, ws, ws_bytes, None)
    assert call(type=3) == -9
    for kw in (dict(B=-1), dict(K=-1), dict(K=64), dict(V=0), dict(V=1 << 30), dict(B=1 << 30, V=1 << 20)):
        assert call(**kw) == -2, kw
    assert call(B=0) == 0
    for name in ("p", "draft", "ua", "us", "tokens", "accepted", "ws"):
        assert call(**{name: None}) == -4, name
    assert call(p=FAKE + 2) == -5 and call(type=2, q=FAKE + 1) == -5 and call(ws=FAKE + 8) == -5
    for name in ("draft", "n_draft", "ua", "us", "tokens", "accepted"):
        assert call(**{name: FAKE + 2}) == -5, name
    need = L.pn_verify_workspace_bytes(2, 1000)
    assert need > 0 and call(ws_bytes=need - 1) == -10
    assert L.pn_verify_workspace_bytes(-1, 10) == 0 and L.pn_verify_workspace_bytes(1, 0) == 0
    assert "workspace" in pn.status_string(-10) and "format" in pn.status_string(-9)


def test_binding_refuses_host_tensors_and_bad_caches(pn):
    import torch
    with pytest.raises(ValueError):
        pn.Cache(MXFP8, 4, 96, 64, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        pn.Cache(MXFP8, 4, 128, 64, torch.zeros(pn.cache_page_bytes(MXFP8, 4, 128, 64), dtype=torch.uint8))
