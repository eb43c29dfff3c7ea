"""GPU tests of the residual RMS norm with block-scaled output and of its
backward pass.

Forward: y is defined as the BF16 nearest to h rstd weight with the sum of
squares exact, and codes, scales and fake-quantised values follow from y by
the formats' definitions; so everything is compared bit for bit with the CPU
oracle applied to a y made here in 64 bits (numpy).
Backward: against the formula in 64 bits, and against differences of the loss
along random directions; tolerances are derived beside each test.
"""
import numpy as np
import pytest
import torch

import guard
from oracle import oracle as O
import workloads as W

from test_gpu_matmul import Operand, exact_and_bound

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FORMATS = ("mxfp8", "nvfp4")


@pytest.fixture(scope="module")
def P():
    import precision_weight_quantization_b200 as P
    return P


def u8(t):
    return t.contiguous().cpu().view(torch.uint8).numpy()


def bf16_of_64(v):
    """BF16 bits of 64-bit values, rounded once (ties to even): significand
    of 8 bits by frexp, exponents below 2^-126 on the subnormal grid."""
    m, e = np.frexp(v)
    e = np.maximum(e, -125)
    step = np.exp2(e - 8.0)
    r = np.rint(v / step) * step
    return W.bits(torch.from_numpy(np.copysign(r, v).astype(np.float32)).bfloat16())


def f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def reference(x, weight, residual, eps):
    """(y bits, h bits, rstd) from BF16 tensors on the CPU."""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    h64 = h.double().numpy()
    with np.errstate(under="ignore"):
        rstd = 1 / np.sqrt((h64 * h64).sum(-1, keepdims=True) / h64.shape[-1] + eps)
        return bf16_of_64(h64 * weight.double().numpy() * rstd), W.bits(h), rstd[..., 0]


def inputs(shape, seed, std=1.0, residual=True):
    x = W.random_bf16(shape, seed=seed, std=std, device="cpu")
    r = W.random_bf16(shape, seed=seed + 1, std=2 * std, device="cpu") if residual else None
    g = torch.Generator().manual_seed(seed + 2)
    return x, (1 + 0.2 * torch.randn(shape[-1], generator=g)).bfloat16(), r


def quantised(fmt, y, amax):
    """Oracle codes, dense scales, global scale and dequantised bits of y [M, D]."""
    if fmt == "mxfp8":
        q, e = O.mxfp8_quant(y)
        return q, e, None, O.mxfp8_dequant(q, e)
    q, sb, gs = O.nvfp4_quant(y, np.float32(amax))
    return q, sb, gs, O.nvfp4_fake_quant(y, np.float32(amax))


def amax_of(y):
    """A static amax a little below the batch's own (the largest values saturate)."""
    return np.float32(np.abs(f64(y)).max() * 0.93)


def check_forward(P, fmt, x, weight, r, eps=1e-6):
    """Codes in both scale layouts and the fake-quantised form, bit for bit."""
    y, h, rstd = reference(x, weight, r, eps)
    slabs = y.reshape((-1,) + y.shape[-2:])
    am = np.array([amax_of(s) for s in slabs], np.float32)
    want = [quantised(fmt, s, a) for s, a in zip(slabs, am)]
    xg, wg, rg = x.to(DEV), weight.to(DEV), r.to(DEV) if r is not None else None
    amax = torch.from_numpy(am).to(DEV)
    for mma in (True, False):
        if fmt == "mxfp8":
            codes, scale, hh = P.rms_norm_mxfp8(xg, wg, rg, eps=eps, mma=mma)
        else:
            codes, scale, gs, hh = P.rms_norm_nvfp4(xg, wg, amax, rg, eps=eps, mma=mma)
            assert np.array_equal(gs.cpu().numpy(), np.array([w[2] for w in want], np.float32))
        assert np.array_equal(u8(codes).reshape(len(want), -1), np.stack([w[0] for w in want]).reshape(len(want), -1))
        dense = np.stack([w[1] for w in want])
        tiles = np.concatenate([O.mma_scale_layout(s).reshape(-1) for s in dense])
        assert np.array_equal(u8(scale).reshape(-1), tiles if mma else dense.reshape(-1)), mma
        assert np.array_equal(W.bits(hh), h)
    yq, hh, rs = P.rms_norm_fake_quant(xg, wg, rg, fmt, amax if fmt == "nvfp4" else None, eps)
    assert np.array_equal(W.bits(yq).reshape(slabs.shape), np.stack([w[3] for w in want]))
    assert np.array_equal(W.bits(hh), h)
    assert np.array_equal(rs.cpu().numpy(), rstd.astype(np.float32))


# ------------------------------------------------------------------ forward

SHAPES = [(1, 32), (1, 2560), (3, 64), (5, 96), (127, 1024), (128, 1056), (129, 160), (2, 4096), (40, 4128),
          (300, 2560), (7, 7168), (3, 16416), (2, 32768), (3, 130, 320), (2, 1, 2048)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("residual", (True, False), ids=("residual", "plain"))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_bits(P, fmt, residual, shape):
    check_forward(P, fmt, *inputs(shape, 31, residual=residual))


def test_nvfp4_odd_sixteens(P):
    for shape in ((3, 16), (130, 48), (4, 2064)):
        check_forward(P, "nvfp4", *inputs(shape, 37))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", (1e-36, 1e-20, 1e-4, 1e4, 1e18, 1e36), ids=str)
def test_forward_over_the_exponent_range(P, fmt, scale):
    """Rows whose squares leave the FP32 range, and rows far below eps."""
    x, w, r = inputs((6, 512), 41)
    check_forward(P, fmt, (x.double() * scale).bfloat16(), w, (r.double() * scale).bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
def test_products_of_weight_and_value_outside_fp32(P, fmt):
    """h weight overflows or underflows FP32 although y does not."""
    for hs, ws in ((1e30, 1e10), (1e-3, 1e-37), (1e-25, 1e-20)):
        x, w, _ = inputs((4, 256), 43, residual=False)
        check_forward(P, fmt, (x.double() * hs).bfloat16(), (w.double() * ws).bfloat16(), None)


@pytest.mark.parametrize("fmt", FORMATS)
def test_exact_ties(P, fmt):
    """Rows of threes and ones with mean square 4 (rstd = 1/2 exactly, eps below
    64-bit resolution): 3 * (odd / 128) has nine significant bits, a tie."""
    D = 256
    x = torch.ones(8, D)
    x.view(8, D // 8, 8)[:, :, :3] = 3.0
    x[1::2] *= -1
    g = torch.Generator().manual_seed(47)
    w = (1 + torch.randint(0, 128, (D,), generator=g) / 128).bfloat16()
    y, _, rstd = reference(x.bfloat16(), w, None, 1e-16)
    assert (rstd == 0.5).all()
    check_forward(P, fmt, x.bfloat16(), w, None, eps=1e-16)


@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_rows_and_zero_weights(P, fmt):
    x, w, r = inputs((5, 320), 53)
    x[1], r[1] = 0, 0
    r[3] = -x[3]
    w[::3] = 0
    check_forward(P, fmt, x, w, r)


def test_nvfp4_amax_of_zero(P):
    """amax 0: every scale and code is zero, with the signs of y."""
    x, w, _ = inputs((3, 64), 59, residual=False)
    codes, sb, gs, _ = P.rms_norm_nvfp4(x.to(DEV), w.to(DEV), torch.zeros(1, device=DEV), mma=False)
    q, s, g = O.nvfp4_quant(reference(x, w, None, 1e-6)[0], np.float32(0))
    assert np.array_equal(u8(codes), q) and np.array_equal(u8(sb), s) and float(gs) == 0.0


@pytest.mark.parametrize("fmt", FORMATS)
def test_strides_and_in_place(P, fmt):
    """Inputs inside wider rows, outputs given by the caller, h written over the
    residual or over x."""
    x, w, r = inputs((33, 288), 61)
    y, h, _ = reference(x, w, r, 1e-6)
    am = torch.tensor([float(amax_of(y))], device=DEV)
    want = quantised(fmt, y, amax_of(y))
    def wide(t, pad):
        buf = torch.full((33, 288 + pad), 9.0, dtype=torch.bfloat16, device=DEV)
        buf[:, :288] = t.to(DEV)
        return buf[:, :288]
    for target in ("new", "residual", "x"):
        xg, rg = wide(x, 8), wide(r, 24)
        hg = {"new": guard.empty((33, 288), torch.bfloat16, lead=8, pad=16), "residual": rg, "x": xg}[target]
        n = 288 if fmt == "mxfp8" else 144
        out = guard.empty((33, n), torch.uint8, lead=16, pad=8)
        if fmt == "mxfp8":
            q, s, hh = P.rms_norm_mxfp8(xg, w.to(DEV), rg, mma=False, out=out, h=hg)
        else:
            q, s, _, hh = P.rms_norm_nvfp4(xg, w.to(DEV), am, rg, mma=False, out=out, h=hg)
        assert hh is hg and q is out
        assert np.array_equal(u8(q), want[0]) and np.array_equal(u8(s), want[1]) and np.array_equal(W.bits(hh), h)
        for t in (xg, rg):
            assert bool((t._base[:, 288:] == 9).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", (5, 400))
def test_rows_that_are_not_finite_leave_the_others(P, fmt, M):
    """A padded batch may hold anything: NaN, infinities and sums that
    overflow in one row change nothing in another, forward and backward."""
    x, w, r = (t.to(DEV) for t in inputs((M, 320), 90))
    dy = W.random_bf16((M, 320), seed=91, std=0.5, device=DEV)
    amax = torch.tensor([3.0], device=DEV)
    bad, keep = [0, 2, 3], [1] + list(range(4, M))
    xb, rb = x.clone(), r.clone()
    xb[0, 5], xb[2], xb[3], rb[3] = float("nan"), float("-inf"), 3e38, 3e38

    def run(x, r):
        if fmt == "mxfp8":
            q, s, h = P.rms_norm_mxfp8(x, w, residual=r, mma=False)
        else:
            q, s, _, h = P.rms_norm_nvfp4(x, w, amax, residual=r, mma=False)
        y, _, rstd = P.rms_norm_fake_quant(x, w, r, fmt, None if fmt == "mxfp8" else amax)
        dx, _ = P.rms_norm_backward(dy, h, w, rstd)
        return q.view(torch.uint8), s.view(torch.uint8), h, y, dx

    for good, got in zip(run(x, r), run(xb, rb)):
        assert torch.equal(good[keep], got[keep])
    h = run(xb, rb)[2]
    assert bool(h[0].isnan()[5]) and bool(torch.isinf(h[2]).all()) and bool(torch.isinf(h[3]).all())
    assert len(bad) + len(keep) == M and P.device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,D", [(7, 320), (400, 2560), (7, 8224)])
def test_rows_that_are_not_finite_follow_the_definition(P, fmt, M, D):
    """rstd and y of the rows themselves: NaN in h makes the whole row NaN, an
    infinite h (from an input, or a sum that overflows BF16) makes rstd 0, y 0
    where h is finite and NaN where it is not.  NaN shows as E4M3 NaN codes, or
    as an NVFP4 block scale of NaN where the whole block is NaN; E2M1 codes have none."""
    x, w, r = (t.to(DEV) for t in inputs((M, D), 97))
    x[0, 5] = float("nan")                      # in the input
    x[1, 0], r[1, 0] = float("inf"), float("-inf")
    x[2], r[2] = 3e38, 3e38                     # every sum overflows
    x[3, 40], r[3, 40] = 3e38, 3e38             # one sum overflows
    x[4, :] = float("-inf")
    h = (x.float() + r.float()).bfloat16()
    rstd = 1 / torch.sqrt(h.double().square().sum(-1, keepdim=True) / D + 1e-6)
    y = (h.double() * w.double() * rstd)[:5]
    nan = y.isnan()
    assert bool(nan[0].all() and nan[1].all() and nan[2].all() and nan[4].all()) and int(nan[3].sum()) == 1
    amax = torch.tensor([3.0], device=DEV)
    yq, hq, got = P.rms_norm_fake_quant(x, w, r, fmt, None if fmt == "mxfp8" else amax)
    assert torch.equal(hq.nan_to_num(7.0), h.nan_to_num(7.0))
    assert bool(got[:2].isnan().all()) and bool((got[2:5] == 0).all())
    whole = [0, 1, 2, 4]
    assert bool(yq[whole].isnan().all()) and bool((yq[3][~nan[3]] == 0).all())
    if fmt == "mxfp8":
        assert bool(yq[3][nan[3]].isnan().all())
        q, s, _ = P.rms_norm_mxfp8(x, w, residual=r, mma=False)
        assert torch.equal(q.view(torch.uint8)[:5] & 0x7f == 0x7f, nan)
        assert bool((q.view(torch.uint8)[3][~nan[3]] & 0x7f == 0).all())
    else:
        q, s, _, _ = P.rms_norm_nvfp4(x, w, amax, residual=r, mma=False)
        assert bool((s.view(torch.uint8)[whole] == 0x7f).all()) and bool((s.view(torch.uint8)[3] == 0).all())
        assert bool((q[3] & 0x77 == 0).all())
    # the rows after them are finite, and the bad rows' gradients are NaN by the formula
    assert bool(got[5:].isfinite().all()) and bool(yq[5:].isfinite().all())
    dy = W.random_bf16((M, D), seed=98, std=0.5, device=DEV)
    dx, dw = P.rms_norm_backward(dy, hq, w, got)
    assert bool(dx[:5].isnan().all()) and bool(dx[5:].isfinite().all()) and bool(dw.isnan().all())


def test_rows_past_32_bits(P):
    """2^31 elements end inside x: the rows around them and the last ones are
    those of a call on these rows alone."""
    M, D = 300000, 7200
    x = torch.empty(M, D, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(92))
    w = W.random_bf16((1, D), seed=93, std=1.0, device=DEV)[0]
    at = 2 ** 31 // D
    rows = torch.tensor([0, at - 1, at, at + 1, at + 700, M - 1], device=DEV)
    few = x[rows].contiguous()
    q, s, _ = P.rms_norm_mxfp8(x, w, mma=False)
    q1, s1, _ = P.rms_norm_mxfp8(few, w, mma=False)
    assert torch.equal(q.view(torch.uint8)[rows], q1.view(torch.uint8)) and torch.equal(s[rows], s1)
    del q
    y, _, rstd = P.rms_norm_fake_quant(x, w)
    dx, _ = P.rms_norm_backward(y, x, w, rstd, need_dweight=False)
    y1, _, rstd1 = P.rms_norm_fake_quant(few, w)
    dx1, _ = P.rms_norm_backward(y1, few, w, rstd1, need_dweight=False)
    assert torch.equal(y[rows], y1) and torch.equal(rstd[rows], rstd1) and torch.equal(dx[rows], dx1)


def test_empty(P):
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    q, s, h = P.rms_norm_mxfp8(x, w, x)
    assert q.shape == (0, 64) and s.numel() == 0 and h.shape == (0, 64)
    dx, dw = P.rms_norm_backward(x, x, w, torch.empty(0, device=DEV))
    assert dx.shape == (0, 64) and bool((dw == 0).all())


# ------------------------------------------------------------------ norm and product as one layer uses them

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", (1, 20, 300))
def test_norm_then_product(P, fmt, M):
    x, w, r = inputs((M, 1056), 67)
    y, _, _ = reference(x, w, r, 1e-6)
    g = torch.Generator(device=DEV).manual_seed(68)
    lin = (torch.randn(500, 1056, generator=g, device=DEV) * 0.02).bfloat16()
    q, s, gs, _ = quantised(fmt, y, amax_of(y))
    if fmt == "mxfp8":
        (qw,), (sw,) = P.mxfp8_quant_grouped_mma([lin])
        codes, scale, _ = P.rms_norm_mxfp8(x.to(DEV), w.to(DEV), r.to(DEV))
        out = P.mxfp8_matmul(codes, scale, qw, sw)
        a = Operand(fmt, torch.from_numpy(q)[None], torch.from_numpy(s)[None])
        b = Operand(fmt, torch.from_numpy(u8(qw))[None], P.scales_from_mma(sw, (1, 500, 33)).cpu())
    else:
        o, sb, gw = P.nvfp4_quant_grouped_mma([[lin]])
        am = torch.tensor([float(amax_of(y))], device=DEV)
        packed, scale, ga, _ = P.rms_norm_nvfp4(x.to(DEV), w.to(DEV), am, r.to(DEV))
        out = P.nvfp4_matmul(packed, scale, ga, o[0][0], sb[0][0], gw[0])
        def nibbles(p):
            p = torch.as_tensor(p)
            return torch.stack((p & 15, p >> 4), -1).flatten(-2)[None]
        a = Operand(fmt, nibbles(q), torch.from_numpy(s.reshape(1, M, 66)), torch.tensor([float(gs)]))
        b = Operand(fmt, nibbles(o[0][0].cpu()), P.scales_from_mma(sb[0][0], (1, 500, 66)).cpu(), gw[0].cpu())
    exact, bound = exact_and_bound(a, b)
    assert bool(((out.double().cpu()[None] - exact).abs() <= bound).all())


@pytest.mark.parametrize("shape", [(20, 1040), (1, 48), (2, 5, 16)], ids=lambda s: "x".join(map(str, s)))
def test_norm_of_odd_sixteens_then_product(P, shape):
    """D % 32 == 16: the norm's own output goes into the product, the weight's
    codes into rows padded to 16 bytes through out=."""
    D, N, B = shape[-1], 100, shape[0] if len(shape) == 3 else 1
    x, w, r = inputs(shape, 69)
    lin = W.random_bf16(shape[:-2] + (N, D), seed=70, std=0.02, device=DEV)
    wide = torch.empty(lin.shape[:-1] + (D // 2 + 8,), dtype=torch.uint8, device=DEV)
    o, sb, gw = P.nvfp4_quant_grouped_mma([[lin]], out=[[wide[..., :D // 2]]])
    y, _, _ = reference(x, w, r, 1e-6)
    am = torch.full((B,), float(amax_of(y)), device=DEV)
    packed, scale, ga, _ = P.rms_norm_nvfp4(x.to(DEV), w.to(DEV), am, r.to(DEV))
    assert packed.shape == shape[:-1] + (D // 2,)
    out = P.nvfp4_matmul(packed, scale, ga, o[0][0], sb[0][0], gw[0])

    def operand(p, s, rows, gs):
        p = p.cpu().reshape(B, rows, -1)
        return Operand("nvfp4", torch.stack((p & 15, p >> 4), -1).flatten(-2),
                       P.scales_from_mma(s, (B, rows, D // 16)).cpu(), gs.cpu())

    exact, bound = exact_and_bound(operand(packed, scale, shape[-2], ga), operand(o[0][0], sb[0][0], N, gw[0]))
    assert bool(((out.double().cpu().reshape(exact.shape) - exact).abs() <= bound).all())
    dense = P.rms_norm_nvfp4(x.to(DEV), w.to(DEV), am, r.to(DEV), mma=False)[0]
    assert dense.is_contiguous() and torch.equal(dense, packed)


# ------------------------------------------------------------------ backward

def backward_inputs(shape, seed, dh=True):
    x, w, r = inputs(shape, seed)
    dy = W.random_bf16(shape, seed=seed + 5, std=0.1, device="cpu")
    d = W.random_bf16(shape, seed=seed + 6, std=0.1, device="cpu") if dh else None
    return (x.float() + r.float()).bfloat16(), w, dy, d


def formula(h, w, dy, dh, rstd):
    """dx and dweight in 64 bits, with the sums of magnitudes their errors scale with."""
    D = h.shape[-1]
    xhat, g = h.double() * rstd[..., None], dy.double() * w.double()
    c = (g * xhat).sum(-1, keepdim=True) / D
    cabs = (g * xhat).abs().sum(-1, keepdim=True) / D
    dx = rstd[..., None] * (g - c * xhat)
    mag = rstd[..., None] * (g.abs() + cabs * xhat.abs())
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    t = (dy.double() * xhat).flatten(0, -2)
    return dx, mag, t.sum(0), t.abs().sum(0)


@pytest.mark.parametrize("dh", (True, False), ids=("dh", "no_dh"))
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (2, 2560), (700, 1040), (1000, 2560), (2500, 64), (5, 7168),
                                   (400, 16400), (3, 32768), (3, 50, 320)], ids=lambda s: "x".join(map(str, s)))
def test_backward_against_the_formula(P, shape, dh):
    """FP32 roundings per value: the sum c adds at most 32 terms in a thread, 5
    steps over the lanes and 32 warps, three roundings a term; at most 10
    outside it: |dx - exact| <= 2^-8 |exact| + 84 2^-24 mag.  dweight: three
    roundings a term, M additions in all, whatever the split:
    (M + 8) 2^-24 sum |dy xhat| (and 2^-8 of the value in BF16)."""
    h, w, dy, d = backward_inputs(shape, 71, dh)
    rstd = torch.rsqrt(h.double().square().mean(-1) + 1e-6).float()
    dx, dw = P.rms_norm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), d.to(DEV) if dh else None)
    ex, mag, ew, mw = formula(h, w, dy, d, rstd.double())
    assert bool(((dx.double().cpu() - ex).abs() <= 2.0 ** -8 * ex.abs() + 84 * 2.0 ** -24 * mag).all())
    M = h.numel() // h.shape[-1]
    bound = (M + 8) * 2.0 ** -24 * mw
    assert bool(((dw.double().cpu() - ew).abs() <= bound).all())
    dx2, dwb = P.rms_norm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), d.to(DEV) if dh else None,
                                   dweight_dtype=torch.bfloat16)
    assert torch.equal(dx2, dx) and torch.equal(dwb, dw.bfloat16())      # the same sums, rounded once
    only, none = P.rms_norm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), d.to(DEV) if dh else None,
                                     need_dweight=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("dh", (True, False), ids=("dh", "no_dh"))
@pytest.mark.parametrize("shape", [(650, 4112), (650, 5120), (650, 5136), (650, 7168), (650, 8192), (650, 8208),
                                   (650, 12288), (650, 16384), (320, 16400), (320, 24592), (310, 32768),
                                   (2, 325, 4624)], ids=lambda s: "x".join(map(str, s)))
def test_backward_of_every_launch_shape(P, shape, dh):
    """Both sides of every width at which the launch changes (4096, 5120, 8192,
    16384 columns), with more rows than all CTAs take at once: every ring
    of rows comes around and every CTA adds several rows into its dweight.
    The bounds of the test above hold: 32 terms of c in a thread at most."""
    test_backward_against_the_formula(P, shape, dh)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gradients_against_differences(P, fmt):
    """Autograd through the fake-quantised norm is the gradient of the norm
    itself (straight-through): L = sum dy y + sum dh h in 64 bits, differenced
    along random directions.  The gradients are BF16 (2^-8 each) and the
    central difference of step 1e-4 errs by 1e-8 of curvature: the bound is
    2^-8 sum |grad v| plus 1e-5 of sum |grad| |v|."""
    M, D = 24, 160
    x, w, r = inputs((M, D), 73)
    dy, dh = (W.random_bf16((M, D), seed=s, std=0.5, device="cpu") for s in (80, 81))
    leaves = [t.to(DEV).requires_grad_() for t in (x, r, w)]
    amax = torch.tensor([3.0], device=DEV) if fmt == "nvfp4" else None
    y, h = P.rms_norm_fake_quant_ste(leaves[0], leaves[2], leaves[1], fmt, amax)
    grads = [g.double().cpu() for g in torch.autograd.grad((y, h), leaves, (dy.to(DEV), dh.to(DEV)))]
    # the point of the derivative is the BF16 h that the forward saw
    at = h.detach().double().cpu()

    def loss(hv, wv):
        return ((dy.double() * hv * torch.rsqrt(hv.square().mean(-1, keepdim=True) + 1e-6) * wv).sum() +
                (dh.double() * hv).sum()).item()

    g = torch.Generator().manual_seed(82)
    for i in range(6):
        vh = torch.randn(M, D, generator=g, dtype=torch.float64) if i % 2 == 0 else torch.zeros(M, D, dtype=torch.float64)
        vw = torch.randn(D, generator=g, dtype=torch.float64) if i % 2 else torch.zeros(D, dtype=torch.float64)
        diff = (loss(at + 1e-4 * vh, w.double() + 1e-4 * vw) - loss(at - 1e-4 * vh, w.double() - 1e-4 * vw)) / 2e-4
        for gx in grads[:2]:     # x and the residual have the same gradient
            dot, size = (gx * vh).sum() + (grads[2] * vw).sum(), (gx * vh).abs().sum() + (grads[2] * vw).abs().sum()
            assert abs(float(dot) - diff) <= (2.0 ** -8 + 1e-5) * float(size)


def test_autograd_forms(P):
    """Leaves that need no gradient, unused outputs, no residual, a broadcast
    input and an expanded output gradient."""
    x, w, r = (t.to(DEV) for t in inputs((40, 320), 83))
    dy, dh = (W.random_bf16((40, 320), seed=s, std=0.5, device=DEV) for s in (84, 85))

    def grads(need, outs=(True, True), res=True, x_=x, dy_=dy):
        lv = [t.detach().clone().requires_grad_(n) for t, n in zip((x_, w, r), need)]
        xin = lv[0].expand(40, 320).contiguous() if x_.shape[0] == 1 else lv[0]
        y, h = P.rms_norm_fake_quant_ste(xin, lv[1], lv[2] if res else None)
        pairs = [(o, g) for o, g, u in ((y, dy_, outs[0]), (h, dh, outs[1])) if u and o.requires_grad]
        torch.autograd.backward([p[0] for p in pairs], [p[1] for p in pairs])
        return [t.grad for t in lv]

    gx, gw, gr = grads((True, True, True))
    assert torch.equal(gx, gr)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        got = grads(need)
        for g, ref, n in zip(got, (gx, gw, gr), need):
            assert (g is None) == (not n) and (g is None or torch.equal(g, ref))
    only_h = grads((True, True, True), outs=(False, True))
    assert torch.equal(only_h[0], dh) and only_h[1] is None
    plain = grads((True, True, False), res=False)
    _, _, rstd = P.rms_norm_fake_quant(x, w)
    want = P.rms_norm_backward(dy, x, w, rstd, dweight_dtype=torch.bfloat16)
    # h is x itself: its own gradient dh is added by autograd in BF16
    assert torch.equal(plain[0], want[0] + dh) and torch.equal(plain[1], want[1])
    wide = grads((True, True, True), dy_=torch.ones((), dtype=torch.bfloat16, device=DEV).expand(40, 320))
    full = grads((True, True, True), dy_=torch.ones(40, 320, dtype=torch.bfloat16, device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(wide, full))
    one = grads((True, False, False), x_=x[:1])
    rows = grads((True, False, False), x_=x[:1].expand(40, 320))[0]
    total = rows.double().sum(0, keepdim=True)
    # 40 BF16 rows added by torch in FP32 and rounded to BF16
    assert bool(((one[0].double() - total).abs() <= 2.0 ** -8 * total.abs() +
                 40 * 2.0 ** -24 * rows.double().abs().sum(0)).all())


def test_streams_repeats_and_graph(P):
    """The same bits on every call and stream; forward and backward captured in
    one graph and replayed with rewritten inputs, while an eager graph of the
    same leaves is alive."""
    x, w, r = (t.to(DEV) for t in inputs((600, 2560), 91))
    dy, dh = (W.random_bf16((600, 2560), seed=s, std=0.5, device=DEV) for s in (92, 93))

    def step(x_, r_):
        y, h, rstd = P.rms_norm_fake_quant(x_, w, r_)
        return (y, h) + P.rms_norm_backward(dy, h, w, rstd, dh)

    ref = step(x, r)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(step(x, r))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, ref))
    sx, sr = x.clone(), r.clone()
    leaf = sx.detach().requires_grad_()
    eager = P.rms_norm_fake_quant_ste(leaf, w, sr)        # stays alive during the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sx, sr)
    x2, r2 = x.flip(0).contiguous(), r.roll(3, 0)
    for a, b in ((x, r), (x2, r2)):
        sx.copy_(a)
        sr.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step(a, b)))
    assert eager[0].requires_grad


def test_training_step_captured_through_autograd(P):
    """Forward and backward of the autograd form in one graph, replayed with
    rewritten inputs: the bits of an eager step."""
    x, w, r = (t.to(DEV) for t in inputs((200, 1056), 99))
    dy, dh = (W.random_bf16((200, 1056), seed=s, std=0.5, device=DEV) for s in (100, 101))

    def step(*leaves):
        lv = [t.detach().requires_grad_() for t in leaves]     # no eager graph of these leaves is alive
        y, h = P.rms_norm_fake_quant_ste(lv[0], lv[1], lv[2])
        return (y.detach(), h.detach()) + torch.autograd.grad((y, h), lv, (dy, dh))

    sx, sw, sr = x.clone(), w.clone(), r.clone()
    step(sx, sw, sr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(sx, sw, sr)
    for a, b in ((x, r), (x.flip(0).contiguous(), r.roll(3, 0))):
        sx.copy_(a)
        sr.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step(a, w, b)))


def test_two_streams_captured_in_one_graph(P):
    """A capture that forks: the weight is quantised on a second stream beside
    the norms, the product joins both; kernels with programmatic and full
    dependencies in one graph."""
    D = 1024
    x, w, r = (t.to(DEV) for t in inputs((40, D), 102))
    lin = W.random_bf16((520, D), seed=103, std=0.05, device=DEV)
    side = torch.cuda.Stream()

    def step(fork):
        cur = torch.cuda.current_stream()
        c, s, h = P.rms_norm_mxfp8(x, w, r)
        if fork:
            side.wait_stream(cur)
        with torch.cuda.stream(side if fork else cur):
            (q,), (sq,) = P.mxfp8_quant_grouped_mma([lin])
        c2, s2, h2 = P.rms_norm_mxfp8(h, w, x)
        if fork:
            cur.wait_stream(side)
        y = P.mxfp8_matmul(c2, s2, q, sq)
        y2 = torch.empty_like(y)
        y2.zero_()
        P.mxfp8_matmul(c, s, q, sq, out=y2)
        return y, y2, h2

    ref = step(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(True)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refusals(P):
    x, w, r = (t.to(DEV) for t in inputs((4, 64), 95))
    one = torch.ones(1, device=DEV)
    for f in (lambda: P.rms_norm_mxfp8(x.float(), w), lambda: P.rms_norm_mxfp8(x, w.float()),
              lambda: P.rms_norm_mxfp8(x, w, r.float()), lambda: P.rms_norm_backward(x, x, w, one, dweight_dtype=torch.half)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: P.rms_norm_mxfp8(x, w[:-1]), lambda: P.rms_norm_mxfp8(x, w, h=x),
              lambda: P.rms_norm_mxfp8(x, w, scale=torch.empty(8, dtype=torch.uint8, device=DEV)),
              lambda: P.rms_norm_nvfp4(x, w, one.expand(2)), lambda: P.rms_norm_nvfp4(x, w, one.double()),
              lambda: P.rms_norm_fake_quant(x, w, format="fp8"), lambda: P.rms_norm_fake_quant(x, w, amax=one),
              lambda: P.rms_norm_fake_quant(x, w, format="nvfp4"), lambda: P.rms_norm_mxfp8(x.cpu(), w),
              lambda: P.rms_norm_backward(x, x, w, torch.ones(3, device=DEV))):
        with pytest.raises(ValueError):
            f()

    def status(f):
        with pytest.raises(P.PwqError) as e:
            f()
        return P.status_string(e.value.status)

    assert status(lambda: P.rms_norm_mxfp8(x, w, eps=0.0)) == "PWQ_ERR_ARG"
    assert status(lambda: P.rms_norm_mxfp8(x, w, eps=float("nan"))) == "PWQ_ERR_ARG"
    assert status(lambda: P.rms_norm_mxfp8(x, w, r[:2])) == "PWQ_ERR_SHAPE"
    assert status(lambda: P.rms_norm_mxfp8(x[:, :48].contiguous(), w[:48].clone(),
                                           scale=torch.empty(512, dtype=torch.uint8, device=DEV))) == "PWQ_ERR_SHAPE"
    assert status(lambda: P.rms_norm_mxfp8(x, w, r, h=torch.empty_like(x[:3]))) == "PWQ_ERR_SHAPE"
    buf = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    assert status(lambda: P.rms_norm_mxfp8(buf[:4], w, buf[4:], h=buf[2:6])) == "PWQ_ERR_OVERLAP"
    assert status(lambda: P.rms_norm_backward(x, x, w, torch.ones(4, device=DEV), out=x)) == "PWQ_ERR_OVERLAP"


def test_second_derivative_is_refused(P):
    x, w, r = (t.to(DEV) for t in inputs((4, 64), 96))
    leaf = x.detach().requires_grad_()
    y, h = P.rms_norm_fake_quant_ste(leaf, w, r)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y.float().square().sum(), leaf, create_graph=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", (1, 200))
def test_layers_back_to_back(P, fmt, M):
    """Twelve layers (norm, product, the residual updated in place, small
    buffers reused) enqueued without a pause give the bits that they give with
    a synchronisation after every call: kernels that are set up before the
    one ahead of them has ended still read what it wrote."""
    D, N = 1024, 1056
    g = torch.Generator(device=DEV).manual_seed(98)
    def w(n, k):
        return (torch.randn(n, k, generator=g, device=DEV) * 0.05).bfloat16()
    x0 = torch.randn(M, D, generator=g, device=DEV).bfloat16()
    norm_w = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16()
    up, down = w(N, D), w(D, N)
    amax = torch.full((1,), 5.0, device=DEV)
    if fmt == "mxfp8":
        (qu, qd), (su, sd) = P.mxfp8_quant_grouped_mma([up, down])
    else:
        q, sb, gs = P.nvfp4_quant_grouped_mma([[up], [down]])

    def run(pause):
        x, res, outs = x0.clone(), x0.clone(), []
        def step(t):
            if pause:
                torch.cuda.synchronize()
            return t
        for _ in range(12):
            if fmt == "mxfp8":
                c, s, _h = step(P.rms_norm_mxfp8(x, norm_w, res, h=res))
                mid = step(P.mxfp8_matmul(c, s, qu, su))
                (c,), (s,) = step(P.mxfp8_quant_grouped_mma([mid]))
                x = step(P.mxfp8_matmul(c, s, qd, sd))
            else:
                c, s, ga, _h = step(P.rms_norm_nvfp4(x, norm_w, amax, res, h=res))
                mid = step(P.nvfp4_matmul(c, s, ga, q[0][0], sb[0][0], gs[0]))
                p, b, ga = step(P.nvfp4_quant_grouped_mma([[mid]]))
                x = step(P.nvfp4_matmul(p[0][0], b[0][0], ga[0], q[1][0], sb[1][0], gs[1]))
            outs.append(x.clone())
        outs.append(res)
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(8):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
