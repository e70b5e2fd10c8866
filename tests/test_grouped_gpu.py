"""The grouped products, their weight gradient and the 8-bit product on the GPU
against plain definitions in 64 bits.

Whole-number inputs make every sum exact in 32 bits, so outputs must equal the
definition rounded once to their type, bit for bit.  Other inputs are held to
the rounding bound of a 32-bit sum in any order: each of the K products and
additions is off by at most 2^-23 of what it adds to (twice the half step of
2^-24, for adders that cut instead of rounding), so K steps are off by at most
(K + 4) * 2^-23 * sum |x||w|, and the result's own rounding adds half a step.
"""
import math

import pytest
import torch

import fp32_gemm_amd as fg

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
CANARY = 777.0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, shape, dtype, most=3):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).to(dtype)


def normal(g, shape, dtype):
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


def padded(rows, cols, pad, dtype, skip=0, fill=float("nan")):
    """A rows x cols view whose rows are cols + pad apart and whose first element
    lies `skip` elements into its storage; everything else holds `fill`."""
    ld = cols + pad
    base = torch.full((rows * ld + skip + 64,), fill, device="cuda").to(dtype)
    return base, base[skip:skip + rows * ld].view(rows, ld)[:, :cols]


def layout(sizes, before=0, after=0):
    off = [before]
    for n in sizes:
        off.append(off[-1] + n)
    return off, off[-1] + after


def offsets_of(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def grouped_exact(x, w, off, transposed):
    y = torch.zeros(x.shape[0], w.shape[1] if transposed else w.shape[2], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for e in range(len(off) - 1):
        we = w[e].double()
        we = (we.t() if transposed else we).contiguous()
        rows = x[off[e]:off[e + 1]].double()
        y[off[e]:off[e + 1]] = rows @ we
        size[off[e]:off[e + 1]] = rows.abs() @ we.abs()
    return y, size


SIZES = [
    ([5, 0, 1, 37, 0, 16], 64, 48),        # empty and single-row experts, thin tiles
    ([130, 0, 257, 1], 192, 136),          # middle tiles with ragged edges
    ([0, 0, 0], 32, 32),                   # nothing at all
    ([1], 1, 1),
    ([3, 2], 7, 5),
    ([33, 64, 100], 129, 131),             # odd widths
    ([40, 200], 1, 300),                   # one step of reduction
    ([50, 90], 500, 1),                    # one column
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,K,N", SIZES)
def test_grouped_whole_numbers(dtype, transposed, sizes, K, N):
    g = gen(1)
    off, M = layout(sizes, before=2, after=3)
    E = len(sizes)
    x = whole(g, (M, K), dtype)
    x[:off[0]] = float("nan")
    x[off[-1]:] = float("nan")
    w = whole(g, (E, N, K) if transposed else (E, K, N), dtype)
    y = torch.full((M, N), CANARY, device="cuda").to(dtype)
    got = fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=transposed)
    assert got is y
    want, _ = grouped_exact(x, w, off, transposed)
    owned = slice(off[0], off[-1])
    assert torch.equal(y[owned], want[owned].to(dtype))
    assert (y[:off[0]].float() == y.new_tensor(CANARY).float()).all()
    assert (y[off[-1]:].float() == y.new_tensor(CANARY).float()).all()


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("padx,padw,pady,skip", [(0, 0, 0, 0), (8, 16, 24, 8), (3, 5, 1, 1), (1, 8, 4, 3)])
def test_grouped_strides_and_alignment(dtype, out, transposed, padx, padw, pady, skip):
    g = gen(2)
    sizes, K, N = [70, 3, 0, 150], 96, 88
    off, M = layout(sizes)
    E = len(sizes)
    xb, x = padded(M, K, padx, dtype, skip)
    x.copy_(whole(g, (M, K), dtype))
    r, c = (N, K) if transposed else (K, N)
    wb, w2 = padded(E * r, c, padw, dtype, skip)
    w = w2.unflatten(0, (E, r))
    w.copy_(whole(g, (E, r, c), dtype))
    yb, y = padded(M, N, pady, out, skip, fill=CANARY)
    guard = yb.clone()
    fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=transposed)
    want, _ = grouped_exact(x, w, off, transposed)
    assert torch.equal(y, want.to(out))
    y.copy_(guard[skip:skip + M * (N + pady)].view(M, N + pady)[:, :N])
    assert torch.equal(yb, guard), "a byte outside Y changed"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,K,N", [([700, 300, 1100], 512, 640), ([12, 4, 30], 1000, 264), ([300, 77], 333, 190)])
def test_grouped_rounding(dtype, transposed, sizes, K, N):
    g = gen(3)
    off, M = layout(sizes)
    x = normal(g, (M, K), dtype)
    w = normal(g, (len(sizes), N, K) if transposed else (len(sizes), K, N), dtype)
    y = torch.empty(M, N, device="cuda", dtype=dtype)
    fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=transposed)
    want, size = grouped_exact(x, w, off, transposed)
    bound = (K + 4) * 2.0 ** -23 * size
    bound += HALF_STEP[dtype] * (want.abs() + bound) + torch.finfo(dtype).tiny
    assert ((y.double() - want).abs() <= bound).all()


def test_grouped_alpha_beta():
    g = gen(4)
    sizes, K, N = [20, 0, 141], 64, 72
    off, M = layout(sizes)
    for dtype, out in ((F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)):
        for n in (N, N + 1):  # whole and partial groups of four columns
            x, w = whole(g, (M, K), dtype), whole(g, (3, K, n), dtype)
            y0 = whole(g, (M, n), out, 50)
            y = y0.clone()
            fg.gemm_grouped(x, w, offsets_of(off), y, alpha=0.5, beta=-2.0)
            want, _ = grouped_exact(x, w, off, False)
            assert torch.equal(y, (0.5 * want - 2.0 * y0.double()).to(out))
            # beta == 0 does not read Y.
            y.fill_(float("nan"))
            fg.gemm_grouped(x, w, offsets_of(off), y, alpha=2.0)
            assert torch.equal(y, (2.0 * want).to(out))


def test_grouped_wide_tiles():
    g = gen(5)
    sizes = [900, 0, 1300, 513, 700, 1111, 600, 1024]
    off, M = layout(sizes)
    K, N = 320, 2304
    assert fg.grouped.plan("nn", BF16, 8, M, N, K)["BM"] == 256
    for dtype in (BF16, F16, F32):
        for transposed in (False, True):
            x = whole(g, (M, K), dtype)
            w = whole(g, (8, N, K) if transposed else (8, K, N), dtype)
            y = torch.empty(M, N, device="cuda", dtype=dtype)
            fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=transposed)
            assert torch.equal(y, grouped_exact(x, w, off, transposed)[0].to(dtype))


def test_grouped_many_experts_and_shared_weights():
    g = gen(6)
    sizes = [int(v) for v in torch.randint(0, 4, (150,), generator=torch.Generator().manual_seed(0))]
    off, M = layout(sizes)
    x, w = whole(g, (M, 64), BF16), whole(g, (150, 64, 80), BF16)
    y = torch.empty(M, 80, device="cuda", dtype=BF16)
    fg.gemm_grouped(x, w, offsets_of(off), y)
    assert torch.equal(y, grouped_exact(x, w, off, False)[0].to(BF16))
    shared = w[:1].expand(150, 64, 80)  # one W behind every expert
    fg.gemm_grouped(x, shared, offsets_of(off), y)
    assert torch.equal(y, grouped_exact(x, shared, off, False)[0].to(BF16))


def test_grouped_without_offsets_is_the_dense_product():
    g = gen(7)
    x, w = whole(g, (300, 200), BF16), whole(g, (200, 104), BF16)
    y = torch.empty(300, 104, device="cuda", dtype=F32)
    fg.gemm_grouped(x, w, None, y)
    assert torch.equal(y, (x.double() @ w.double()).to(F32))


def test_grouped_offsets_out_of_order_stay_inside():
    # Wrong offsets give wrong rows, never an access outside the operands: the
    # guard around Y keeps its values.
    g = gen(8)
    M, K, N = 100, 64, 64
    x, w = whole(g, (M, K), BF16), whole(g, (4, K, N), BF16)
    for off in ([50, 20, -7, 300, 10], [-5, 1000, -1000, 1 << 30, -(1 << 30)], [100, 100, 0, 0, 100]):
        yb, y = padded(M, N, 8, BF16, 16, fill=CANARY)
        guard = yb.clone()
        fg.gemm_grouped(x, w, offsets_of(off), y)
        y.copy_(guard[16:16 + M * (N + 8)].view(M, N + 8)[:, :N])
        assert torch.equal(yb, guard)


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    g = gen(9)
    sizes, K, N = [40, 25], 160, 96
    off, M = layout(sizes)
    for dtype in (F32, BF16, F16):
        x, w = whole(g, (M, K), dtype), whole(g, (2, K, N), dtype, 3)
        w[w == 0] = 1
        x[7, 3], x[50, 159], w[1, 159, 11] = float("nan"), float("inf"), float("nan")
        y = torch.empty(M, N, device="cuda", dtype=dtype)
        fg.gemm_grouped(x, w, offsets_of(off), y)
        want = grouped_exact(x, w, off, False)[0].to(dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(y[fine], want[fine])


# ---- weight gradient ---------------------------------------------------------

def wgrad_exact(x, dy, off):
    E = len(off) - 1
    dw = torch.zeros(E, x.shape[1], dy.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dw)
    for e in range(E):
        xt = x[off[e]:off[e + 1]].double().t().contiguous()
        d = dy[off[e]:off[e + 1]].double()
        dw[e], size[e] = xt @ d, xt.abs() @ d.abs()
    return dw, size


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("sizes,K,N", SIZES + [([64, 128, 1, 65], 256, 520), ([200, 0, 31], 77, 150)])
def test_wgrad_whole_numbers(dtype, out, sizes, K, N):
    g = gen(10)
    off, M = layout(sizes, before=3, after=2)
    x, dy = whole(g, (M, K), dtype), whole(g, (M, N), dtype)
    for t in (x, dy):
        t[:off[0]] = float("nan")
        t[off[-1]:] = float("nan")
    dw = torch.full((len(sizes), K, N), float("nan"), device="cuda", dtype=out)
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    assert torch.equal(dw, wgrad_exact(x, dy, off)[0].to(out))


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("padx,pady,padw,skip", [(8, 16, 4, 8), (3, 1, 2, 1), (0, 5, 0, 0)])
def test_wgrad_strides_and_alignment(dtype, out, padx, pady, padw, skip):
    g = gen(11)
    sizes, K, N = [90, 0, 41], 120, 72
    off, M = layout(sizes)
    _, x = padded(M, K, padx, dtype, skip)
    _, dy = padded(M, N, pady, dtype, skip)
    x.copy_(whole(g, (M, K), dtype))
    dy.copy_(whole(g, (M, N), dtype))
    wb, w2 = padded(3 * K, N, padw, out, skip, fill=CANARY)
    guard = wb.clone()
    dw = w2.unflatten(0, (3, K))
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    assert torch.equal(dw, wgrad_exact(x, dy, off)[0].to(out))
    w2.copy_(guard[skip:skip + 3 * K * (N + padw)].view(3 * K, N + padw)[:, :N])
    assert torch.equal(wb, guard), "a byte outside dW changed"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_wgrad_rounding_and_accumulation(dtype):
    g = gen(12)
    sizes, K, N = [1500, 0, 600], 264, 136
    off, M = layout(sizes)
    x, dy = normal(g, (M, K), dtype), normal(g, (M, N), dtype)
    dw0 = normal(g, (3, K, N), F32)
    dw = dw0.clone()
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw, alpha=0.25, beta=1.0)
    want, size = wgrad_exact(x, dy, off)
    bound = (max(sizes) + 4) * 2.0 ** -23 * (0.25 * size + dw0.double().abs())
    assert ((dw.double() - (0.25 * want + dw0.double())).abs() <= bound).all()
    assert torch.equal(dw[1], dw0[1])  # no rows: beta * dW


def test_wgrad_wide_tiles():
    g = gen(13)
    sizes = [1300, 820, 0, 729]
    off, M = layout(sizes)
    K, N = 2048 - 8, 2048 - 16
    assert fg.grouped.plan("tn", BF16, 4, M, N, K)["BM"] == 256
    for dtype in (F32, BF16, F16):
        x, dy = whole(g, (M, K), dtype), whole(g, (M, N), dtype)
        dw = torch.empty(4, K, N, device="cuda", dtype=F32)
        fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
        assert torch.equal(dw, wgrad_exact(x, dy, off)[0].float())


def test_gradients_against_differences():
    # loss = sum(Y * G): its change along a direction, by central differences of
    # the product itself, is the gradients' scalar product with that direction.
    # The loss is bilinear, so the difference is exact but for rounding.
    g = gen(14)
    sizes, K, N = [17, 0, 30], 40, 24
    off, M = layout(sizes)
    o = offsets_of(off)
    x, w, G = (normal(g, s, F32) for s in ((M, K), (3, K, N), (M, N)))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    fg.gemm_grouped(G, w, o, dx, transpose_w=True)
    fg.gemm_grouped_wgrad(x, G, o, dw)

    def loss(x, w):
        y = torch.empty(M, N, device="cuda")
        fg.gemm_grouped(x.contiguous(), w.contiguous(), o, y)
        return (y.double() * G.double()).sum().item()

    u, v = normal(g, x.shape, F32), normal(g, w.shape, F32)
    # Terms of either side are of size 1 and number M * K * N; each carries at
    # most (K + 4) roundings of 2^-23, and the step doubles them.
    bound = 4 * (K + 4) * 2.0 ** -23 * M * K * N
    along_x = (loss(x + u, w) - loss(x - u, w)) / 2
    along_w = (loss(x, w + v) - loss(x, w - v)) / 2
    assert abs(along_x - (dx.double() * u.double()).sum().item()) <= bound
    assert abs(along_w - (dw.double() * v.double()).sum().item()) <= bound


# ---- 8 bits --------------------------------------------------------------------

def codes_exact(x):
    """Codes and 64-bit scales, from the definition, in exact whole-number
    arithmetic on the host: the nearest integer to 127 x / top, ties to even."""
    from fractions import Fraction
    q, s = [], []
    for row in x.double().cpu().tolist():
        if not all(math.isfinite(v) for v in row):
            q.append([0] * len(row))
            s.append(float("nan"))
            continue
        top = max((abs(v) for v in row), default=0.0)
        s.append(top / 127)
        q.append([round(Fraction(v) * 127 / Fraction(top)) if top else 0 for v in row])
    return torch.tensor(q, dtype=torch.int8).reshape(x.shape), torch.tensor(s, dtype=torch.float64)


def check_quantize(x):
    M, K = x.shape
    q = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    fg.quantize_rows(x, q, s)
    want_q, want_s = codes_exact(x)
    assert torch.equal(q.cpu(), want_q)
    got, bad = s.cpu().double(), torch.isnan(want_s)
    assert torch.equal(torch.isnan(got), bad)
    assert (got[~bad] - want_s[~bad]).abs().le(2.0 ** -24 * want_s[~bad] + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 64), (2, 777), (9, 1000), (1, 4096), (2, 1026)])
def test_quantize_rows(dtype, M, K):
    check_quantize(normal(gen(20 + K), (M, K), dtype))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_ties_zeros_and_bad_values(dtype):
    # 127 x / top is a half-integer wherever top / x is 2, 2/3 (no code beyond
    # 127), 254, 254/3 ...: ties must go to the even code.
    rows = [[2.0, 1.0, -1.0, 0.5] * 4,
            [254.0 / 256, 1 / 256, 3 / 256, -5 / 256] * 4,
            [127.0, 0.5, 1.5, -2.5] * 4,
            [0.0] * 16, [-0.0] * 16,
            [1.0] * 15 + [float("nan")], [float("inf")] + [1.0] * 15, [-float("inf")] * 16,
            [torch.finfo(dtype).max] * 8 + [-torch.finfo(dtype).max] * 8,
            [torch.finfo(dtype).smallest_normal] * 16]
    check_quantize(torch.tensor(rows, device="cuda").to(dtype))


def test_quantize_long_rows_and_strides():
    g = gen(30)
    for K in (20000, 17001):  # past what a workgroup keeps in registers
        check_quantize(normal(g, (2, K), BF16))
    for pad, skip in ((8, 8), (3, 1)):
        _, x = padded(6, 500, pad, BF16, skip)
        x.copy_(normal(g, (6, 500), BF16))
        qb = torch.full((6 * (500 + pad) + 64,), 55, dtype=torch.int8, device="cuda")
        q = qb[skip:skip + 6 * (500 + pad)].view(6, 500 + pad)[:, :500]
        s = torch.empty(6, device="cuda")
        fg.quantize_rows(x, q, s)
        assert torch.equal(q.cpu(), codes_exact(x)[0])
        q.fill_(55)
        assert (qb == 55).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", [(4100, 2049), (4096, 1030), (4097, 129), (300, 5001)])
def test_quantize_many_rows(dtype, M, K):
    # 127 x is exact in 64 bits, and the quotient lies on a tie or at least 2^-33
    # from one, so rounding it once in 64 bits moves nothing across.
    x = normal(gen(31), (M, K), dtype)
    x[::7] *= 2.0 ** -13
    q = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    fg.quantize_rows(x, q, s)
    top = x.double().abs().amax(1)
    assert torch.equal(q, torch.round(x.double() * 127 / top[:, None]).to(torch.int8))
    assert ((s.double() - top / 127).abs() <= 2.0 ** -24 * top / 127).all()


def igemm_exact(a, sa, b, sb, bias, off):
    """Groups' products in 64 bits (whole numbers up to 2^31 are exact there)."""
    M, N = a.shape[0], b.shape[-2]
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    b, sb = b.reshape(-1, N, b.shape[-1]), sb.reshape(-1, N)
    for e in range(b.shape[0]):
        rows = slice(off[e], off[e + 1])
        y[rows] = (a[rows].double() @ b[e].double().t().contiguous()) * sa[rows, None].double() * sb[e].double()
        if bias is not None:
            y[rows] += bias.reshape(-1, N)[e].double()
    return y


@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (1, 1000, 777), (7, 33, 100), (16, 256, 4096), (130, 150, 272),
                                   (200, 129, 1), (600, 384, 512), (64, 1, 65), (33, 72, 17)])
def test_igemm(out, M, N, K):
    g = gen(40)
    a = torch.randint(-128, 128, (M, K), device="cuda", generator=g).to(torch.int8)
    b = torch.randint(-128, 128, (N, K), device="cuda", generator=g).to(torch.int8)
    # Powers of two: scaling and, without a bias, the whole result are exact but
    # for the sum's rounding to 24 bits (none up to 1024 full products) and the output's.
    sa = torch.exp2(torch.randint(-8, 0, (M,), device="cuda", generator=g).float())
    sb = torch.exp2(torch.randint(-8, 0, (N,), device="cuda", generator=g).float())
    y = torch.full((M, N), float("nan"), device="cuda", dtype=out)
    fg.igemm(a, sa, b, sb, y)
    want = igemm_exact(a, sa, b, sb, None, [0, M])
    assert torch.equal(y, want.to(F32).to(out))
    bias = normal(g, (N,), F32)
    fg.igemm(a, sa, b, sb, y, bias=bias)
    part, want = want.abs(), want + bias.double()
    # The sum's conversion, the bias' addition, and the output's rounding.
    bound = 2.0 ** -24 * (part + want.abs()) * 1.001 + HALF_STEP[out] * want.abs() * 1.001 + torch.finfo(out).tiny
    # A value past the type's range rounds to its infinity.
    past = torch.isinf(want.to(out))
    assert torch.equal(y[past], want.to(out)[past])
    assert ((y.double() - want).abs() <= bound)[~past].all()


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 1, 30], 96, 128), ([200, 0, 90], 136, 272), ([3, 50], 31, 77)])
def test_igemm_grouped(sizes, N, K):
    g = gen(41)
    off, M = layout(sizes, before=1, after=2)
    E = len(sizes)
    a = torch.randint(-128, 128, (M, K), device="cuda", generator=g).to(torch.int8)
    b = torch.randint(-128, 128, (E, N, K), device="cuda", generator=g).to(torch.int8)
    sa = torch.exp2(torch.randint(-8, 0, (M,), device="cuda", generator=g).float())
    sb = torch.exp2(torch.randint(-8, 0, (E, N), device="cuda", generator=g).float())
    bias = torch.randint(-4, 5, (E, N), device="cuda", generator=g).float()
    y = torch.full((M, N), CANARY, device="cuda")
    fg.igemm(a, sa, b, sb, y, bias=bias, offsets=offsets_of(off))
    # Sums below 2^23, scales down to 2^-16: 64-bit sums with the bias may need
    # more than 24 bits, so the bias' addition may round once.
    want = igemm_exact(a, sa, b, sb, bias, off)
    owned = slice(off[0], off[-1])
    assert ((y[owned].double() - want[owned]).abs() <= 2.0 ** -24 * want[owned].abs()).all()
    assert (y[:off[0]] == CANARY).all() and (y[off[-1]:] == CANARY).all()


def test_igemm_largest_sums():
    # Every product at its largest: 131071 * 2^14, just below 2^31.
    K = 131071
    a = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    b[2] = 127
    one = torch.ones(3, device="cuda")
    y = torch.empty(2, 3, device="cuda")
    fg.igemm(a, one[:2], b, one, y)
    want = torch.tensor([K * 16384.0, K * 16384.0, -K * 16256.0], dtype=torch.float64).float()
    assert torch.equal(y.cpu(), want.expand(2, 3))


def test_igemm_bad_token_is_nan_throughout():
    x = normal(gen(42), (3, 64), BF16)
    x[1, 5] = float("inf")
    q, s = torch.empty(3, 64, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    fg.quantize_rows(x, q, s)
    w = torch.ones(16, 64, dtype=torch.int8, device="cuda")
    y = torch.empty(3, 16, device="cuda")
    fg.igemm(q, s, w, torch.ones(16, device="cuda"), y)
    assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any()


# ---- streams, graphs, repeats ----------------------------------------------------

def test_streams_and_graph_replays():
    g = gen(50)
    sizes, K, N = [40, 0, 90], 128, 96
    off, M = layout(sizes)
    x, w, o = whole(g, (M, K), BF16), whole(g, (3, K, N), BF16), offsets_of(off)
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    wq = whole(g, (3, N, K), torch.int8, 100)
    ws = torch.ones(3, N, device="cuda")
    y, dw, z = torch.empty(M, N, device="cuda", dtype=BF16), torch.empty(3, K, N, device="cuda"), torch.empty(M, N, device="cuda")

    def step():
        fg.gemm_grouped(x, w, o, y)
        fg.gemm_grouped_wgrad(x, y, o, dw)
        fg.quantize_rows(x, q, s)
        fg.igemm(q, s, wq, ws, z, offsets=o)

    def results():
        return [t.clone() for t in (y, dw, z)]

    step()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results(), want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(whole(gen(60 + k), (M, K), BF16))
        o.copy_(offsets_of([[0, 1, 100, 130], [0, 130, 130, 130], [5, 40, 60, 90]][k]))
        for t in (y, dw, z):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = results()
        for t in (y, dw, z):
            t.zero_()
        step()
        assert all(torch.equal(a, b) for a, b in zip(results(), replayed))


def test_repeats_are_bitwise_equal():
    g = gen(51)
    off, M = layout([500, 3, 200])
    x, w, o = normal(g, (M, 1000), BF16), normal(g, (3, 1000, 264), BF16), offsets_of(off)
    y = [torch.empty(M, 264, device="cuda") for _ in range(2)]
    for t in y:
        fg.gemm_grouped(x, w, o, t)
    assert torch.equal(*y)


def test_stack_past_two_gigabytes():
    # Element offsets of the last expert and rows pass 32 bits.
    E, K, N = 5, 16384, 16400
    w = torch.zeros(E, K, N, dtype=BF16, device="cuda")
    w[E - 1, K - 1, N - 8:] = 3
    w[E - 1, 0, 0] = 5
    x = torch.ones(4, K, dtype=BF16, device="cuda")
    y = torch.empty(4, N, dtype=BF16, device="cuda")
    fg.gemm_grouped(x, w, offsets_of([0, 0, 0, 0, 0, 4]), y)
    want = torch.zeros(4, N, dtype=BF16, device="cuda")
    want[:, 0], want[:, N - 8:] = 5, 3
    assert torch.equal(y, want)
    M = 140000
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-1, -1] = 2
    y = torch.empty(M, 16, dtype=BF16, device="cuda")
    one = torch.ones(K, 16, dtype=BF16, device="cuda")
    fg.gemm_grouped(x, one, None, y)
    assert (y[-1] == 2).all() and not y[:-1].any()
    dw = torch.empty(K, 16, dtype=F32, device="cuda")
    y.fill_(1)
    fg.gemm_grouped_wgrad(x, y, None, dw)
    assert (dw[-1] == 2).all() and not dw[:-1].any()


# ---- every tile, at sizes that leave it partly filled -----------------------------
# tests/test_grouped_host.py checks that these sizes reach every compiled tile.

TILES = [  # rows of the groups, K, N
    ([700, 513, 0, 1100, 64, 65, 300, 1], 200, 4100),
    ([700, 400, 0, 300], 500, 2050),
    ([700, 400, 0, 300], 500, 4100),
    ([70, 0, 30, 129, 200], 333, 1003),
    ([17, 1, 0, 5, 9, 20], 520, 1601),
    ([3], 4000, 1000),
]
WGRAD_TILES = [  # type, rows of the groups, K, N
    (BF16, [700, 0, 333, 1000], 1800, 2040), (BF16, [700, 0, 333, 1000], 500, 300),
    (BF16, [100, 0, 1, 333, 64, 65, 200, 90], 900, 700), (F32, [33, 0, 70, 5], 777, 301),
    (BF16, [500, 0, 333, 100], 1000, 1002), (F32, [100, 0, 333, 64, 100, 100], 1001, 1045), (F32, [100, 0, 33, 64], 2000, 2044),
    (F32, [300, 200, 333], 2000, 2044),
]
IGEMM_TILES = [(4090, 4090, 1500), (2100, 3050, 300), (1000, 1700, 900), (130, 1700, 900), (100, 1000, 2000),
               (1, 4000, 4001), (2040, 2040, 700)]  # M, N, K
MANY = [((0, 1, 2, 3), 520, 264), ((0, 1, 2, 3), 72, 64), ((600, 257, 0, 512, 400), 72, 520),
        ((1600, 1257, 0, 1512, 1400), 520, 512)]  # rows of 150 groups in turn, K, N


@pytest.mark.parametrize("sizes,K,N", TILES)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_every_tile(sizes, K, N, trans, dtype):
    g = gen(70)
    off, M = layout(sizes, before=1, after=2)
    E = len(sizes)
    x = whole(g, (M, K), dtype)
    w = whole(g, (E, N, K) if trans else (E, K, N), dtype)
    y = torch.full((M, N), CANARY, device="cuda").to(dtype)
    fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=trans)
    want, _ = grouped_exact(x, w, off, trans)
    assert torch.equal(y[off[0]:off[-1]], want[off[0]:off[-1]].to(dtype))
    canary = y.new_tensor(CANARY).float()
    assert (y[:1].float() == canary).all() and (y[off[-1]:].float() == canary).all()


@pytest.mark.parametrize("dtype,sizes,K,N", WGRAD_TILES)
def test_every_weight_gradient_tile(dtype, sizes, K, N):
    g = gen(71)
    off, M = layout(sizes, before=1, after=2)
    x, dy = whole(g, (M, K), dtype), whole(g, (M, N), dtype)
    dw = torch.full((len(sizes), K, N), float("nan"), device="cuda", dtype=dtype)
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    assert torch.equal(dw, wgrad_exact(x, dy, off)[0].to(dtype))


@pytest.mark.parametrize("M,N,K", IGEMM_TILES)
def test_every_igemm_tile(M, N, K):
    g = gen(72)
    a = torch.randint(-128, 128, (M, K), device="cuda", generator=g).to(torch.int8)
    b = torch.randint(-128, 128, (N, K), device="cuda", generator=g).to(torch.int8)
    sa = torch.exp2(torch.randint(-8, 0, (M,), device="cuda", generator=g).float())
    sb = torch.exp2(torch.randint(-8, 0, (N,), device="cuda", generator=g).float())
    y = torch.full((M, N), float("nan"), device="cuda")
    fg.igemm(a, sa, b, sb, y)
    assert torch.equal(y, igemm_exact(a, sa, b, sb, None, [0, M]).float())


@pytest.mark.parametrize("each,K,N", MANY)
def test_more_groups_than_lanes(each, K, N):
    # Groups past the 64 that a wave looks at together.
    g = gen(73)
    sizes = [each[(5 * e + e // 7) % len(each)] for e in range(150)]
    off, M = layout(sizes, before=2, after=1)
    x, w = whole(g, (M, K), BF16), whole(g, (150, K, N), BF16)
    y = torch.full((M, N), CANARY, device="cuda", dtype=F32)
    fg.gemm_grouped(x, w, offsets_of(off), y)
    owned = slice(off[0], off[-1])
    assert torch.equal(y[owned], grouped_exact(x, w, off, False)[0][owned].float())
    assert (y[:2] == CANARY).all() and (y[off[-1]:] == CANARY).all()
    dy = whole(g, (M, N), BF16)
    dw = torch.full((150, K, N), float("nan"), device="cuda")
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    assert torch.equal(dw, wgrad_exact(x, dy, off)[0].float())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K,N", [(1, 3), (3, 1), (2, 2), (7, 7), (200, 3), (5, 130), (1, 1)])
def test_rows_shorter_than_a_load(dtype, K, N):
    # Rows of fewer than 16 bytes, over many slices, in every form; the operands
    # end with their storage.
    g = gen(74)
    sizes = [300, 0, 1, 77]
    off, M = layout(sizes)
    for trans in (False, True):
        x, w = whole(g, (M, K), dtype), whole(g, (4, N, K) if trans else (4, K, N), dtype)
        y = torch.empty(M, N, device="cuda", dtype=dtype)
        fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=trans)
        assert torch.equal(y, grouped_exact(x, w, off, trans)[0].to(dtype))
        if not trans:
            tall = whole(g, (1, 1000, N), dtype)
            xs = whole(g, (40, 1000), dtype, 1)
            ys = torch.empty(40, N, device="cuda", dtype=F32)
            fg.gemm_grouped(xs, tall[0], None, ys)
            assert torch.equal(ys, (xs.double() @ tall[0].double()).float())
    dy = whole(g, (M, N), dtype)
    dw = torch.empty(4, K, N, device="cuda", dtype=F32)
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    assert torch.equal(dw, wgrad_exact(x, dy, off)[0].float())


def test_alpha_beta_on_every_kind_of_tile():
    g = gen(75)
    for sizes, K, N in (([700, 600, 900, 512], 64, 2050), ([300, 260], 64, 514), ([70, 65], 64, 67), ([3, 1], 64, 31)):
        off, M = layout(sizes)
        x, w, y0 = whole(g, (M, K), BF16), whole(g, (len(sizes), K, N), BF16), whole(g, (M, N), BF16, 50)
        y = y0.clone()
        fg.gemm_grouped(x, w, offsets_of(off), y, alpha=0.5, beta=-2.0)
        assert torch.equal(y, (0.5 * grouped_exact(x, w, off, False)[0] - 2.0 * y0.double()).to(BF16))
        dy, dw0 = whole(g, (M, N), BF16), whole(g, w.shape, F32, 50)
        dw = dw0.clone()
        fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw, beta=1.0)
        assert torch.equal(dw, (wgrad_exact(x, dy, off)[0] + dw0.double()).float())
