"""GPU tests of the block-scaled products (mxfp8_matmul, nvfp4_matmul) against
the same sums in 64 bits, from codes and scales decoded here by the formats'
definitions (tile-layout scales by the layout's index formula).

Tolerance.  The tensor core multiplies codes and scales exactly and adds the
products of one MMA (32 or 64 of them) to an FP32 accumulator.  Counting one
FP32 rounding (at most one unit, 2^-23, of a partial sum, since hardware may
truncate) for the accumulation and one for the alignment inside each MMA, a
sum over K is off by at most 2 (K / 32 + 1) 2^-23 S, with S = sum |a w| (no
partial sum exceeds it); the CPU split of K adds at most 8 more FP32
additions.  The global scales cost three FP32 roundings, the output one
BF16 rounding, at most 2^-8 of the value:
    |y - exact| <= 2^-8 |exact| + (2 (K / 32 + 1) + 12) 2^-23 S,
plus half of the smallest BF16 subnormal for results that underflow.
"""
import numpy as np
import pytest
import torch

import guard

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FORMATS = ("mxfp8", "nvfp4")


@pytest.fixture(scope="module")
def P():
    import precision_weight_quantization_b200 as P
    return P


# ------------------------------------------------------------------ operands and their 64-bit values

def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m / 8 * np.exp2(-6.0))
    v[(b & 0x7f) == 0x7f] = np.nan
    return np.where(b & 0x80, -v, v)


E4M3 = torch.tensor(e4m3_table(), dtype=torch.float64)
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def tile_index(rows, cols):
    """Byte of scale (r, c) inside a slab of the tile layout."""
    r, c = torch.arange(rows)[:, None], torch.arange(cols)[None, :]
    return (r // 128 * -(-cols // 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


class Operand:
    """Codes [B, R, K] (bytes), dense scale bytes [B, R, S] and global scales,
    with the arguments a product takes and the values they stand for."""

    def __init__(self, fmt, codes, scales, gs=None):
        self.fmt, self.codes, self.scales, self.gs = fmt, codes, scales, gs
        B, R, S = scales.shape
        slab = -(-R // 128) * -(-S // 4) * 512
        tiles = torch.zeros(B, slab, dtype=torch.uint8)
        tiles[:, tile_index(R, S).reshape(-1)] = scales.reshape(B, -1)
        self.tiles = tiles.reshape(-1).to(DEV)

    def values(self):
        if self.fmt == "mxfp8":
            v, s = E4M3[self.codes.long()], torch.exp2(self.scales.double() - 127)
            s[self.scales == 255] = float("nan")
            return v * s.repeat_interleave(32, -1)
        return E2M1[self.codes.long()] * E4M3[self.scales.long()].repeat_interleave(16, -1)

    def packed(self, pad=0):
        c = self.codes if self.fmt == "mxfp8" else self.codes[..., 0::2] | self.codes[..., 1::2] << 4
        B, R, n = c.shape
        buf = torch.full((B, R, n + pad), 0x55, dtype=torch.uint8, device=DEV)
        buf[..., :n] = c.to(DEV)
        v = buf[..., :n]
        return v.view(torch.float8_e4m3fn) if self.fmt == "mxfp8" else v

    def args(self, two_d=False, pad=0):
        c = self.packed(pad)
        return (c[0] if two_d else c, self.tiles) + ((self.gs.to(DEV),) if self.fmt == "nvfp4" else ())


def random_operand(fmt, B, R, K, seed, spread=6):
    """Random codes over the whole range (no NaN) and scales over 2^spread."""
    g = torch.Generator().manual_seed(seed)
    if fmt == "mxfp8":
        codes = torch.randint(0, 256, (B, R, K), generator=g, dtype=torch.int32)
        codes[(codes & 0x7f) == 0x7f] = 0x30
        scales = torch.randint(127 - spread, 128 + spread, (B, R, K // 32), generator=g, dtype=torch.int32)
        return Operand(fmt, codes.to(torch.uint8), scales.to(torch.uint8))
    codes = torch.randint(0, 16, (B, R, K), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = torch.randint(0, 0x7f, (B, R, K // 16), generator=g, dtype=torch.int32).to(torch.uint8)
    gs = torch.rand(B, generator=g) * 0.1 + 1e-3
    return Operand(fmt, codes, scales, gs)


def integer_operand(fmt, B, R, K, seed):
    """Values in {-2, -1, 0, 1, 2} with block scales 1 or 2: every partial sum
    is an integer below 2^24, so the FP32 sum is exact in any order."""
    g = torch.Generator().manual_seed(seed)
    pick = torch.randint(0, 5, (B, R, K), generator=g)
    if fmt == "mxfp8":
        codes = torch.tensor([0xc0, 0xb8, 0x00, 0x38, 0x40], dtype=torch.uint8)[pick]
        scales = (127 + torch.randint(0, 2, (B, R, K // 32), generator=g)).to(torch.uint8)
        return Operand(fmt, codes, scales)
    codes = torch.tensor([12, 10, 0, 2, 4], dtype=torch.uint8)[pick]
    scales = torch.tensor([0x38, 0x40], dtype=torch.uint8)[torch.randint(0, 2, (B, R, K // 16), generator=g)]
    return Operand(fmt, codes, scales, torch.ones(B))


def call(P, a, w, out=None, two_d=False, pad=0):
    f = P.mxfp8_matmul if a.fmt == "mxfp8" else P.nvfp4_matmul
    return f(*a.args(two_d, pad), *w.args(two_d, pad), out=out)


def bmm64(x, y):
    return torch.bmm(x.to(DEV), y.to(DEV).transpose(1, 2)).cpu()


def exact_and_bound(a, w):
    x, y = a.values(), w.values()
    K = x.shape[-1]
    exact, S = bmm64(x, y), bmm64(x.abs(), y.abs())
    if a.gs is not None:
        s = (a.gs.double() * w.gs.double())[:, None, None]
        exact, S = exact * s, S * s
    return exact, 2.0 ** -8 * exact.abs() + (2 * (K / 32 + 1) + 12) * 2.0 ** -23 * S + 2.0 ** -134


def check(P, a, w, **kw):
    y = call(P, a, w, **kw)
    exact, bound = exact_and_bound(a, w)
    torch.cuda.synchronize()
    assert P.device_error() == 0
    d = (y.double().cpu().reshape(exact.shape) - exact).abs()
    assert bool((d <= bound).all()), float((d - bound).max())
    return y


def bf16_exact(v):
    """64-bit integers below 2^24 rounded to BF16 (exact in FP32 first)."""
    return v.float().bfloat16()


# ------------------------------------------------------------------ values

# (batch, M, N, K): one token to long prompts, both sides of every tile width
# (16, 32, 64, 128 tokens; 128 and 256 rows), K shorter than a step, ragged K
SHAPES = [(1, 1, 1, 32), (1, 1, 128, 64), (1, 2, 127, 96), (1, 15, 129, 128), (1, 16, 8, 160), (1, 17, 256, 288),
          (1, 32, 1000, 256), (1, 33, 100, 1056), (1, 64, 300, 4096), (1, 65, 257, 512), (1, 128, 128, 128),
          (1, 129, 513, 544), (3, 1, 130, 320), (5, 40, 64, 96), (2, 200, 300, 1312), (1, 300, 2560, 2560),
          (1, 8, 2560, 9728), (130, 3, 40, 64)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_values_over_the_whole_code_range(P, fmt, shape):
    B, M, N, K = shape
    check(P, random_operand(fmt, B, M, K, 1), random_operand(fmt, B, N, K, 2))


# shapes of the wide path: many 256 x 256 tiles, ragged on every side
WIDE = [(1, 256, 256, 256), (1, 257, 511, 800), (1, 1000, 4099, 1056), (1, 2048, 6144, 2560), (3, 520, 1030, 2080),
        (16, 333, 512, 1024), (1, 4096, 2560, 9728), (1, 5000, 256, 288)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "x".join(map(str, s)))
def test_values_of_wide_products(P, fmt, shape):
    B, M, N, K = shape
    check(P, random_operand(fmt, B, M, K, 3), random_operand(fmt, B, N, K, 4))


# one token tile of every width on many weight rows; a few more tokens against few weight rows and a long K
# (K split over a cluster at 64 and 128 tokens a tile); many tiles of few tokens
MIDDLE = [(1, 65, 5400, 320), (1, 96, 5400, 288), (1, 130, 5640, 160), (1, 160, 5400, 320), (1, 200, 5400, 352),
          (1, 224, 5400, 96), (1, 225, 5400, 320), (1, 100, 700, 4160), (1, 200, 300, 8256), (1, 64, 640, 8256),
          (90, 7, 300, 160), (90, 50, 280, 544), (80, 33, 512, 1312)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", MIDDLE, ids=lambda s: "x".join(map(str, s)))
def test_values_between_tokens_and_prompts(P, fmt, shape):
    B, M, N, K = shape
    check(P, random_operand(fmt, B, M, K, 26), random_operand(fmt, B, N, K, 27))


def test_single_rows_with_arbitrary_strides(P):
    """A dimension of size 1 may carry any stride."""
    a, w = random_operand("mxfp8", 1, 1, 96, 28), random_operand("mxfp8", 1, 40, 96, 29)
    ref = check(P, a, w, two_d=True)
    q, s = a.args(True)
    odd = torch.as_strided(q.view(torch.uint8), (1, 96), (7, 1))
    assert torch.equal(P.mxfp8_matmul(odd, s, *w.args(True)), ref)
    three = torch.as_strided(q.view(torch.uint8), (1, 1, 96), (5, 3, 1))
    assert torch.equal(P.mxfp8_matmul(three, s, *w.args())[0], ref)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 1, 300, 4096), (1, 40, 129, 2080), (2, 130, 257, 1056), (1, 700, 1030, 4096),
                                   (1, 2100, 4100, 800)], ids=lambda s: "x".join(map(str, s)))
def test_integer_sums_are_exact(P, fmt, shape):
    B, M, N, K = shape
    a, w = integer_operand(fmt, B, M, K, 5), integer_operand(fmt, B, N, K, 6)
    y = call(P, a, w)
    assert torch.equal(y.cpu(), bf16_exact(bmm64(a.values(), w.values())))


def test_nvfp4_rows_of_odd_sixteens(P):
    """K % 32 == 16 with padded code rows: half an MMA of zeros at the end."""
    for M, K in ((3, 16), (70, 48), (300, 1040)):
        check(P, random_operand("nvfp4", 2, M, K, 7), random_operand("nvfp4", 2, 200, K, 8), pad=8)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", (5, 600))
def test_operand_and_output_strides(P, fmt, M):
    """Padded code rows, 2-D operands, outputs inside wider rows, at odd offsets and widths."""
    a, w = random_operand(fmt, 1, M, 1056, 9), random_operand(fmt, 1, 301, 1056, 10)
    ref = check(P, a, w, two_d=True, pad=48)
    for lead, pad in ((0, 3), (1, 0), (8, 3), (3, 4)):
        out = guard.empty((M, 301), torch.bfloat16, lead=lead, pad=pad)
        y = call(P, a, w, two_d=True, out=out)
        assert y is out and torch.equal(y, ref), (lead, pad)
    # batched, slabs apart, output batch stride larger than a slab
    a, w = random_operand(fmt, 3, M, 256, 11), random_operand(fmt, 3, 136, 256, 12)
    ref = check(P, a, w, pad=32)
    big = torch.full((3, M + 5, 144), 7.0, dtype=torch.bfloat16, device=DEV)
    y = call(P, a, w, out=big[:, :M, :136])
    assert torch.equal(y, ref) and bool((big[:, M:] == 7).all()) and bool((big[:, :, 136:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(70, 5377), (150, 5504), (333, 1001), (400, 1030), (600, 323), (777, 4160)])
def test_output_rows_at_every_alignment(P, fmt, M, N):
    """Rows that begin at every element of a 16-byte unit, even and odd row
    strides, tiles cut on either side; integers, so the sums are exact."""
    a, w = integer_operand(fmt, 1, M, 160, 50), integer_operand(fmt, 1, N, 160, 51)
    ref = bf16_exact(bmm64(a.values(), w.values()))[0].to(DEV)
    for lead, pad in [(i, 0) for i in range(8)] + [(0, 1), (0, 2), (1, 1), (2, 5), (7, 4)]:
        out = guard.empty((M, N), torch.bfloat16, lead=lead, pad=pad)
        assert torch.equal(call(P, a, w, two_d=True, out=out), ref), (lead, pad)


@pytest.mark.parametrize("N", (33000, 33001))
def test_outputs_past_32_bits(P, N):
    """2^31 elements end inside y; both ways to store a row."""
    M = 66000
    a, w = integer_operand("mxfp8", 1, M, 64, 54), integer_operand("mxfp8", 1, N, 64, 55)
    y = call(P, a, w)[0]
    at = 2 ** 31 // N
    rows = torch.tensor([0, 1, at - 1, at, at + 1, at + 300, M - 2, M - 1])
    few = Operand("mxfp8", a.codes[:, rows], a.scales[:, rows])
    assert torch.equal(y[rows.to(DEV)].cpu(), bf16_exact(bmm64(few.values(), w.values()))[0])


@pytest.mark.parametrize("M", (4, 40, 400))
def test_nan_codes_stay_in_their_row(P, M):
    """E4M3 has NaN codes; a token that holds one is NaN, the others are as without it."""
    a, w = random_operand("mxfp8", 1, M, 512, 52), random_operand("mxfp8", 1, 260, 512, 53)
    ref = call(P, a, w)[0]
    a.codes[0, 1, 77] = 0x7f
    y = call(P, Operand("mxfp8", a.codes, a.scales), w)[0]
    assert bool(y[1].isnan().all()) and torch.equal(y[[0] + list(range(2, M))], ref[[0] + list(range(2, M))])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", (4, 400))
def test_nan_scales_stay_in_their_row_and_column(P, fmt, M):
    a, w = random_operand(fmt, 1, M, 512, 13), random_operand(fmt, 1, 260, 512, 14)
    ref = call(P, a, w)[0]
    nan = 255 if fmt == "mxfp8" else 0x7f
    a.scales[0, 2, 5] = nan
    w.scales[0, 131, 0] = nan
    a2, w2 = (Operand(o.fmt, o.codes, o.scales, o.gs) for o in (a, w))
    y = call(P, a2, w2)[0]
    bad = torch.zeros(M, 260, dtype=torch.bool, device=DEV)
    bad[2] = True
    bad[:, 131] = True
    assert bool(y.isnan()[bad].all()) and torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("M", (3, 40, 300))
@pytest.mark.parametrize("sa,sw", [(0, 254), (254, 0), (1, 253), (0, 127), (0, 0), (64, 63), (60, 60), (70, 50), (190, 170)])
def test_block_scales_over_their_range(P, M, sa, sw):
    """UE8M0 scales from 2^-127 to 2^127: integers times 2^(sa + sw - 254), exact
    in FP32, results in BF16's subnormal range and below it among them."""
    a, w = integer_operand("mxfp8", 1, M, 128, 56), integer_operand("mxfp8", 1, 130, 128, 57)
    a.scales[:], w.scales[:] = sa, sw
    want = bmm64(E4M3[a.codes.long()], E4M3[w.codes.long()]) * 2.0 ** (sa + sw - 254)
    y = call(P, *(Operand("mxfp8", o.codes, o.scales) for o in (a, w)))
    assert torch.equal(y.cpu(), want.float().bfloat16())


def test_global_scales_over_their_range(P):
    """Scales whose product leaves the FP32 range although the result does not
    (and results that overflow or underflow)."""
    a, w = integer_operand("nvfp4", 6, 3, 128, 15), integer_operand("nvfp4", 6, 130, 128, 16)
    a.gs = torch.tensor([1e-30, 1e30, 1e-38, 1e38, 0.0, 3e-25])
    w.gs = torch.tensor([1e-8, 1e-30, 1e38, 1e2, 1.0, 1e-20])
    exact, bound = exact_and_bound(a, w)
    y = call(P, a, w).double().cpu()
    big = exact.abs() > 3.3895e38                       # beyond the largest BF16
    assert bool(torch.isinf(y[big]).all()) and bool((y[big].sign() == exact[big].sign()).all())
    assert bool(((y - exact).abs()[~big] <= bound[~big]).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_empty_and_zero_length_products(P, fmt):
    def op(R, K):
        return random_operand(fmt, 2, R, K, 17)
    out = guard.empty((2, 5, 7), torch.bfloat16)
    out.fill_(3)
    assert bool((call(P, op(5, 0), op(7, 0), out=out) == 0).all())      # an empty sum
    assert call(P, op(0, 64), op(7, 64)).shape == (2, 0, 7)
    assert call(P, op(5, 64), op(0, 64)).shape == (2, 5, 0)


# ------------------------------------------------------------------ how a program calls it

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 3, 2560, 4096), (2, 600, 1030, 800)], ids=("tokens", "wide"))
def test_streams_repeats_and_graph(P, fmt, shape):
    """The same bits on every call, on two streams at once, and from a
    captured graph whose operands were rewritten between replays."""
    B, M, N, K = shape
    a, w = random_operand(fmt, B, M, K, 18), random_operand(fmt, B, N, K, 19)
    ref = check(P, a, w)
    aa, ww = [t.clone() for t in a.args()], w.args()      # a keeps its own scale tiles
    f = P.mxfp8_matmul if fmt == "mxfp8" else P.nvfp4_matmul
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(f(*aa, *ww))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(*aa, *ww, out=out)
    b = random_operand(fmt, B, M, K, 20)
    for src, want in ((a, ref), (b, call(P, b, w)), (a, ref)):
        for dst, new in zip(aa, src.args()):
            dst.copy_(new)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert P.device_error() == 0


def test_from_bf16_to_product(P):
    """Quantise into the tile layout, then multiply: equal to the product of
    the library's own dequantised values in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(21)
    x = torch.randn(2, 90, 1056, generator=g, device=DEV).bfloat16()
    w = (torch.randn(2, 300, 1056, generator=g, device=DEV) * 0.02).bfloat16()
    (qx, qw), (sx, sw) = P.mxfp8_quant_grouped_mma([x, w])
    y = P.mxfp8_matmul(qx, sx, qw, sw)
    dense = [P.scales_from_mma(s, t.shape[:-1] + (33,)) for s, t in ((sx, x), (sw, w))]
    vx, vw = (torch.ldexp(q.double().view(*q.shape[:-1], 33, 32), (s.int() - 127)[..., None]).view(q.shape)
              for q, s in ((qx, dense[0]), (qw, dense[1])))
    exact, S = vx @ vw.transpose(1, 2), vx.abs() @ vw.abs().transpose(1, 2)
    assert bool(((y.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + 80 * 2.0 ** -23 * S).all())
    out, sb, gs = P.nvfp4_quant_grouped_mma([[x], [w]])
    y = P.nvfp4_matmul(out[0][0], sb[0][0], gs[0], out[1][0], sb[1][0], gs[1])
    a, b = (Operand("nvfp4", torch.stack((o[0].cpu() & 15, o[0].cpu() >> 4), -1).flatten(-2),
                    P.scales_from_mma(s[0], t.shape[:-1] + (66,)).cpu(), g_.cpu())
            for o, s, t, g_ in ((out[0], sb[0], x, gs[0]), (out[1], sb[1], w, gs[1])))
    exact, bound = exact_and_bound(a, b)
    assert bool(((y.double().cpu() - exact).abs() <= bound).all())


# ------------------------------------------------------------------ refusals

def test_refusals(P):
    a, w = random_operand("mxfp8", 1, 4, 64, 22), random_operand("mxfp8", 1, 8, 64, 23)
    (qa, sa), (qw, sw) = a.args(True), w.args(True)
    for bad in ((qa.view(torch.uint8).float(), sa, qw, sw), (qa, sa, qw.bfloat16(), sw)):
        with pytest.raises(TypeError):
            P.mxfp8_matmul(*bad)
    for bad in ((qa, sa[:-512], qw, sw), (qa, sa, qw, sw[::2]), (qa, sa, qw[None], sw), (qa, sa, qw, sw.float()),
                (qa, sa.cpu(), qw, sw), (qa.cpu(), sa, qw, sw), (qa.t(), sa, qw, sw)):
        with pytest.raises(ValueError):
            P.mxfp8_matmul(*bad)
    with pytest.raises(TypeError):
        P.mxfp8_matmul(qa, sa, qw, sw, out=torch.empty(4, 8, device=DEV))

    def status(*args, **kw):
        with pytest.raises(P.PwqError) as e:
            P.mxfp8_matmul(*args, **kw)
        return P.status_string(e.value.status)

    assert status(qa, sa, qw, sw, out=torch.empty(4, 9, dtype=torch.bfloat16, device=DEV)) == "PWQ_ERR_SHAPE"
    odd = torch.zeros(4, 72, dtype=torch.uint8, device=DEV)
    assert status(odd[:, :64], sa, qw, sw) == "PWQ_ERR_ALIGN"        # rows 72 bytes apart
    assert status(odd.view(-1)[8:8 + 256].view(4, 64), sa, qw, sw) == "PWQ_ERR_ALIGN"
    over = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    assert status(over[:256].view(4, 64), sa, qw, sw, out=over[:64].view(torch.bfloat16).view(4, 8)) == \
        "PWQ_ERR_OVERLAP"
    n, v = random_operand("nvfp4", 1, 4, 64, 24), random_operand("nvfp4", 1, 8, 64, 25)
    (qa, sa, ga), (qw, sw, gw) = n.args(True), v.args(True)
    for bad in ((qa, sa, ga.double(), qw, sw, gw), (qa, sa, ga, qw, sw, gw.expand(2)), (qa, sa, ga.cpu(), qw, sw, gw)):
        with pytest.raises(ValueError):
            P.nvfp4_matmul(*bad)
