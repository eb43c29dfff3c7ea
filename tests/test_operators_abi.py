"""Host-side validation of the block-scaled products and the residual RMS norm
(no GPU): every bad argument is rejected with the documented status before any
CUDA call.  The addresses are made up and never dereferenced."""
import ctypes

import pytest

from test_abi import T, _lib

by = ctypes.byref
BASE = 1 << 40
G = 1 << 30


@pytest.fixture(scope="module")
def L():
    return _lib()


def codes(L, at, B, R, K, fp4=False, rs=None, bs=None):
    n = K // 2 if fp4 else K
    rs = n if rs is None else rs
    return T(L, at, B, R, K, R * rs if bs is None else bs, rs)


def bf16(L, at, B, R, C, rs=None):
    rs = C if rs is None else rs
    return T(L, at, B, R, C, R * rs, rs)


def test_mxfp8_matmul_validation(L):
    f = L.lib.mxfp8_matmul
    a, w, y = codes(L, BASE, 2, 8, 64), codes(L, BASE + G, 2, 24, 64), bf16(L, BASE + 2 * G, 2, 8, 24)
    sa, sw = BASE + 3 * G, BASE + 4 * G

    def st(a=a, sa=sa, w=w, sw=sw, y=y):
        return f(by(a) if a else None, sa, by(w) if w else None, sw, by(y) if y else None, None)

    assert st(a=None) == st(w=None) == st(y=None) == st(sa=None) == st(sw=None) == L.PWQ_ERR_NULL
    assert st(a=codes(L, None, 2, 8, 64)) == L.PWQ_ERR_NULL
    # K % 32, and every pair of extents that must agree
    assert st(a=codes(L, BASE, 2, 8, 48), w=codes(L, BASE + G, 2, 24, 48)) == L.PWQ_ERR_SHAPE
    assert st(w=codes(L, BASE + G, 2, 24, 96)) == L.PWQ_ERR_SHAPE
    assert st(w=codes(L, BASE + G, 1, 24, 64)) == L.PWQ_ERR_SHAPE
    assert st(y=bf16(L, BASE + 2 * G, 2, 9, 24)) == L.PWQ_ERR_SHAPE
    assert st(y=bf16(L, BASE + 2 * G, 2, 8, 25)) == L.PWQ_ERR_SHAPE
    assert st(a=codes(L, BASE, 2, -8, 64)) == L.PWQ_ERR_SHAPE
    # too many output tiles for one launch (code tensors of 2^30 rows of 32 bytes)
    many = codes(L, BASE, 1 << 20, 8, 32), codes(L, BASE + (1 << 33), 1 << 20, 1 << 10, 32)
    assert f(by(many[0]), BASE + (1 << 39), by(many[1]), BASE + (1 << 42), by(bf16(L, BASE + (1 << 44), 1 << 20, 8, 1 << 10)),
             None) == L.PWQ_ERR_SHAPE
    # alignment: code base, row and batch strides 16 bytes, scales 16 bytes, y 2 bytes
    assert st(a=codes(L, BASE + 8, 2, 8, 64)) == L.PWQ_ERR_ALIGN
    assert st(a=codes(L, BASE, 2, 8, 64, rs=72)) == L.PWQ_ERR_ALIGN
    assert st(w=codes(L, BASE + G, 2, 24, 64, bs=24 * 64 + 8)) == L.PWQ_ERR_ALIGN
    assert st(sa=sa + 8) == st(sw=sw + 4) == L.PWQ_ERR_ALIGN
    assert st(y=bf16(L, BASE + 2 * G + 1, 2, 8, 24)) == L.PWQ_ERR_ALIGN
    # strides
    assert st(a=codes(L, BASE, 2, 8, 64, rs=48)) == L.PWQ_ERR_STRIDE
    assert st(a=codes(L, BASE, 2, 8, 64, bs=256)) == L.PWQ_ERR_STRIDE
    assert st(y=bf16(L, BASE + 2 * G, 2, 8, 24, rs=23)) == L.PWQ_ERR_STRIDE
    # y over an operand or its scales (the padded tile of a_scale included)
    for at in (BASE, BASE + G + 16, sa + 1022, sw):
        assert st(y=bf16(L, at, 2, 8, 24)) == L.PWQ_ERR_OVERLAP
    # nothing to launch
    assert st(a=codes(L, None, 2, 0, 64), y=bf16(L, None, 2, 0, 24), sa=None) == L.PWQ_OK
    assert st(w=codes(L, None, 2, 0, 64), y=bf16(L, None, 2, 8, 0), sw=None) == L.PWQ_OK


def test_nvfp4_matmul_validation(L):
    f = L.lib.nvfp4_matmul
    a, w = codes(L, BASE, 1, 8, 64, True), codes(L, BASE + G, 1, 24, 64, True)
    y = bf16(L, BASE + 2 * G, 1, 8, 24)
    sa, sw, ga, gw = (BASE + i * G for i in (3, 4, 5, 6))

    def st(a=a, sa=sa, ga=ga, w=w, sw=sw, gw=gw, y=y):
        return f(by(a), sa, ga, by(w), sw, gw, by(y), None)

    assert st(ga=None) == st(gw=None) == st(sa=None) == L.PWQ_ERR_NULL
    assert st(ga=ga + 2) == st(gw=gw + 1) == L.PWQ_ERR_ALIGN
    assert st(a=codes(L, BASE, 1, 8, 40, True), w=codes(L, BASE + G, 1, 24, 40, True)) == L.PWQ_ERR_SHAPE
    # K = 48: 24-byte rows are refused, rows padded to 32 bytes would be taken
    assert st(a=codes(L, BASE, 1, 8, 48, True), w=codes(L, BASE + G, 1, 24, 48, True, rs=32)) == L.PWQ_ERR_ALIGN
    assert st(y=bf16(L, ga - 4, 1, 8, 24)) == L.PWQ_ERR_OVERLAP


@pytest.mark.parametrize("fmt", ("mxfp8", "nvfp4"))
@pytest.mark.parametrize("fake", (False, True), ids=("codes", "fake"))
def test_norm_validation(L, fmt, fake):
    fp4 = fmt == "nvfp4"
    D = 64
    x, r, h = (bf16(L, BASE + i * G, 2, 8, D) for i in range(3))
    q = bf16(L, BASE + 3 * G, 2, 8, D) if fake else codes(L, BASE + 3 * G, 2, 8, D, fp4)
    w, sc, gs, am, rs = (BASE + i * G for i in (4, 5, 6, 7, 8))
    f = getattr(L.lib, "rms_norm_%s%s" % (fmt, "_fake_quant" if fake else ""))

    def st(x=x, r=r, w=w, eps=1e-6, am=am, h=h, q=q, sc=sc, mma=1, gs=gs, rs=rs):
        ref = lambda t: by(t) if t is not None else None  # noqa: E731
        args = [ref(x), ref(r), w, eps] + ([am] if fp4 else []) + [ref(h), ref(q)]
        if not fake:
            args += [sc, mma] + ([gs] if fp4 else [])
        return f(*args, rs, None)

    assert st(x=None) == st(q=None) == st(w=None) == L.PWQ_ERR_NULL
    # h exactly with a residual; eps; the layout flag
    assert st(r=None) == st(h=None) == L.PWQ_ERR_ARG
    assert st(eps=0.0) == st(eps=-1.0) == st(eps=float("nan")) == st(eps=float("inf")) == st(eps=1e-17) == L.PWQ_ERR_ARG
    assert st(w=w + 8) == st(rs=rs + 2) == L.PWQ_ERR_ALIGN
    assert st(x=bf16(L, BASE + 8, 2, 8, D)) == L.PWQ_ERR_ALIGN
    assert st(r=bf16(L, BASE + G, 2, 8, D, rs=68)) == L.PWQ_ERR_ALIGN
    assert st(h=bf16(L, BASE + 2 * G, 2, 8, D, rs=56)) == L.PWQ_ERR_STRIDE
    assert st(r=bf16(L, BASE + G, 2, 9, D)) == L.PWQ_ERR_SHAPE
    bad = 72 if not fp4 else 56

    def out(at, D, B=2, M=8):
        return bf16(L, at, B, M, D) if fake else codes(L, at, B, M, D, fp4, rs=D)

    assert st(x=bf16(L, BASE, 2, 8, bad), r=None, h=None, q=out(BASE + 3 * G, bad)) == L.PWQ_ERR_SHAPE
    assert st(x=bf16(L, BASE, 1, 8, 32800), r=None, h=None, q=out(BASE + 3 * G, 32800, 1)) == L.PWQ_ERR_SHAPE
    assert st(q=out(BASE + 3 * G, D, 2, 7)) == L.PWQ_ERR_SHAPE
    # h in place is exact or refused; other outputs never over an input
    assert st(h=bf16(L, BASE + 16, 2, 8, D)) == L.PWQ_ERR_OVERLAP
    assert st(h=bf16(L, BASE + G + 2 * D, 2, 8, D)) == L.PWQ_ERR_OVERLAP
    assert st(q=out(BASE, D)) == st(q=out(BASE + G, D)) == st(rs=w) == st(rs=BASE + 2 * G) == L.PWQ_ERR_OVERLAP
    assert st(h=x, q=out(BASE, D)) == st(h=r, rs=BASE + G) == L.PWQ_ERR_OVERLAP
    if not fake:
        assert st(sc=None) == L.PWQ_ERR_NULL
        assert st(mma=2) == L.PWQ_ERR_ARG
        assert st(sc=sc + 2) == L.PWQ_ERR_ALIGN
        assert st(sc=BASE + 3 * G + 4) == L.PWQ_ERR_OVERLAP
        # the zero padding of the tile layout is an output too
        assert st(sc=rs - 4, mma=1) == L.PWQ_ERR_OVERLAP
    if fp4:
        assert st(am=None) == L.PWQ_ERR_NULL
        assert st(am=am + 1) == L.PWQ_ERR_ALIGN
        if not fake:
            assert st(gs=None) == L.PWQ_ERR_NULL
            assert st(gs=am + 4) == L.PWQ_ERR_OVERLAP
    assert st(x=bf16(L, None, 2, 0, D), r=None, h=None, q=out(None, D, 2, 0)) == L.PWQ_OK


def test_norm_backward_validation(L):
    f = L.lib.rms_norm_backward
    D = 64
    dy, dh, h, dx = (bf16(L, BASE + i * G, 1, 300, D) for i in range(4))
    w, rs, dw, ws = (BASE + i * G for i in (4, 5, 6, 7))
    big = 1 << 26

    def st(dy=dy, dh=dh, h=h, w=w, rs=rs, dx=dx, dw=dw, b=0, ws=ws, n=big):
        ref = lambda t: by(t) if t is not None else None  # noqa: E731
        return f(ref(dy), ref(dh), ref(h), w, rs, ref(dx), dw, b, ws, n, None)

    assert st(dy=None) == st(h=None) == st(dx=None) == st(w=None) == st(rs=None) == L.PWQ_ERR_NULL
    assert st(b=2) == L.PWQ_ERR_ARG
    assert st(w=w + 2) == st(rs=rs + 1) == st(dw=dw + 2) == st(dw=dw + 1, b=1) == L.PWQ_ERR_ALIGN
    assert st(dy=bf16(L, BASE, 1, 299, D)) == st(dx=bf16(L, BASE + 3 * G, 1, 300, 80)) == L.PWQ_ERR_SHAPE
    assert st(dh=bf16(L, BASE + G, 1, 300, 48)) == L.PWQ_ERR_SHAPE
    assert st(ws=None) == st(n=255) == st(ws=ws + 4) == L.PWQ_ERR_WORKSPACE
    for at in (BASE, BASE + G, BASE + 2 * G, w, rs):
        assert st(dx=bf16(L, at, 1, 300, D)) == L.PWQ_ERR_OVERLAP
    assert st(dw=ws + 128) == st(dw=BASE + 3 * G + 64) == st(ws=BASE + 16) == L.PWQ_ERR_OVERLAP
    assert L.lib.rms_norm_backward_workspace_size(None) == 0
    assert L.lib.rms_norm_backward_workspace_size(by(bf16(L, BASE, 1, 4, 40000))) == 0
    e = bf16(L, None, 1, 0, D)
    assert st(dy=e, dh=None, h=e, dx=e, dw=None, ws=None, n=0) == L.PWQ_OK
