"""Microscaled 4-bit floats on the GPU: quantisation against a definition that
compares with the borders between codes, code for code, and the product against
sums in 64 bits.

A code is one rounding of an exact quotient, so all codes and scales must be equal.
Products of codes are exact; where the whole sum fits 24 bits, results must equal the
sum rounded once to their type.  Other sums are held to (K + 4) * 2^-23 * sum |a||b|,
the bound of K additions in any order, each off by at most twice the half step of
2^-24, and half a step of the result's type.
"""
import pytest
import torch

import fp32_gemm_amd as fg

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
BORDERS = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5], dtype=torch.float64)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def blocks_of(K):
    return (K + 31) // 32


def codes_of(x):
    """Codes (M x K) and scale bytes of x, from the definition."""
    x = x.double().cpu()
    M, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 32)).view(M, -1, 32)
    bad = ~torch.isfinite(b).all(2)
    top = torch.where(torch.isfinite(b), b, torch.zeros(())).abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent.double() - 3, -127.0).clamp(min=-127)
    a = b.abs() / torch.ldexp(torch.ones(()).double(), e)[:, :, None]
    code = torch.bucketize(a, BORDERS, right=False)      # at a border: the lower code,
    at = torch.isin(a, BORDERS) & (code % 2 == 1)         # or the even one above it
    code = code + at + 8 * torch.signbit(b)
    code[bad] = 0
    scale = (e + 127).to(torch.uint8)
    scale[bad] = 255
    return code.view(M, -1)[:, :K], scale


def pack(code):
    M, K = code.shape
    c = torch.nn.functional.pad(code, (0, K % 2))
    return (c[:, ::2] | c[:, 1::2] << 4).to(torch.uint8)


def unpack(q, scale):
    """The values of packed codes, K = 2 q columns, in 64 bits on the GPU."""
    q, scale = q.cuda().long(), scale.cuda()
    v = torch.cat([VALUES, -VALUES]).cuda()[torch.stack((q & 15, q >> 4), -1)].flatten(-2)
    s = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scale.double() - 127)
    s = torch.where(scale == 255, float("nan"), s)
    return v * s.repeat_interleave(32, -1)[..., :v.shape[-1]]


def quantized(x, q=None, scale=None):
    M, K = x.shape
    q = torch.empty(M, (K + 1) // 2, dtype=torch.uint8, device="cuda") if q is None else q
    scale = torch.empty(M, blocks_of(K), dtype=torch.uint8, device="cuda") if scale is None else scale
    got = fg.quantize_mx4(x, q, scale)
    assert got[0] is q and got[1] is scale
    return q, scale


def check_codes(x, q, scale):
    code, want = codes_of(x)
    assert torch.equal(scale.cpu(), want)
    assert torch.equal(q.cpu(), pack(code))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (7, 100), (300, 257), (1, 8192),
                                 (9, 2048), (4, 2050), (2, 40001), (1000, 96)])
def test_quantize(dtype, M, K):
    g = gen(M * 100003 + K)
    x = torch.randn(M, K, device="cuda", generator=g) * torch.exp2(
        torch.randint(-20, 12, (M, K), device="cuda", generator=g).float())
    check_codes(x.to(dtype), *quantized(x.to(dtype)))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_borders(dtype):
    # Each border between codes, the values next to it, and their negatives, under
    # several scales; 4 in every block fixes its scale.
    v = torch.cat([BORDERS, VALUES]).to(dtype)
    up, down = (torch.nextafter(v.float(), torch.tensor(t)) if dtype is F32 else None for t in (9.0, -1.0))
    if dtype is not F32:
        bits = v.view(torch.int16)
        up, down = (bits + 1).view(dtype), torch.where(v > 0, bits - 1, bits).view(dtype)
    all_v = torch.cat([v, up.to(dtype), down.to(dtype)])
    all_v = torch.cat([all_v, -all_v])
    all_v = torch.nn.functional.pad(all_v, (0, -len(all_v) % 31)).view(-1, 31)
    rows = torch.cat([torch.full((len(all_v), 1), 4.0, dtype=dtype), all_v], 1)
    for power in (0, -9, 11):
        x = (rows.float() * 2.0 ** power).to(dtype).cuda()
        check_codes(x, *quantized(x))


def test_quantize_extremes():
    tiny, top = 2.0 ** -149, torch.finfo(F32).max
    rows = [[0.0] * 32, [-0.0] + [0.0] * 31, [tiny] * 32, [2.0 ** -127] + [tiny] * 31, [2.0 ** -126, 2.0 ** -128] * 16,
            [2.0 ** -125, 2.0 ** -127, -2.0 ** -128, 3 * 2.0 ** -129] * 8, [top, -top, 2.0 ** 126, 2.0 ** 120] * 8,
            [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("-inf")], [1.0, float("nan")] * 16, [7.9, -7.9, 6.1] + [1.0] * 29]
    x = torch.tensor(rows, device="cuda")
    q, scale = quantized(x)
    check_codes(x, q, scale)
    assert scale[:2].sum() == 0 and (scale[7:10] == 255).all() and q[7:10].sum() == 0
    x = torch.tensor([[float("inf")] * 3 + [1.0] * 37], device="cuda", dtype=BF16)  # the other block is its own
    q, scale = quantized(x)
    check_codes(x, q, scale)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("padx,padq,skip", [(0, 0, 0), (3, 1, 1), (8, 16, 8), (1, 5, 3)])
def test_quantize_windows(dtype, padx, padq, skip):
    g, M, K = gen(5), 37, 333
    base = torch.full((M * (K + padx) + skip,), float("nan"), device="cuda", dtype=dtype)
    x = base[skip:].view(M, K + padx)[:, :K]
    x.copy_(torch.randn(M, K, device="cuda", generator=g))
    C = (K + 1) // 2
    room = torch.full((M * (C + padq) + skip + 8,), 0xA5, device="cuda", dtype=torch.uint8)
    q = room[skip:skip + M * (C + padq)].view(M, C + padq)[:, :C]
    wide = torch.full((M * blocks_of(K) + skip + 8,), 0xA5, device="cuda", dtype=torch.uint8)
    scale = wide[skip:skip + M * blocks_of(K)].view(M, -1)
    quantized(x, q, scale)
    check_codes(x, q, scale)
    q.fill_(0xA5), scale.fill_(0xA5)
    assert (room == 0xA5).all() and (wide == 0xA5).all(), "a byte outside the outputs changed"


def test_quantize_empty():
    for M, K in ((0, 64), (4, 0)):
        quantized(torch.empty(M, K, device="cuda"))


def random_operand(g, shape_rows, K2, low=126, high=128):
    q = torch.randint(0, 256, (*shape_rows, K2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(low, high + 1, (*shape_rows, (K2 + 15) // 16), dtype=torch.uint8, device="cuda", generator=g)
    return q, s


def product(a, sa, b, sb, off, bias=None):
    """The sums, and the sums of magnitudes, in 64 bits."""
    a, b = unpack(a, sa), unpack(b, sb)
    off = [0, a.shape[0]] if off is None else off
    b = b if b.dim() == 3 else b[None]
    y = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for e in range(len(off) - 1):
        rows = a[off[e]:off[e + 1]]
        y[off[e]:off[e + 1]] = rows @ b[e].t().contiguous()
        size[off[e]:off[e + 1]] = rows.abs() @ b[e].abs().t().contiguous()
        if bias is not None:
            y[off[e]:off[e + 1]] += bias.reshape(len(b), -1)[e].double()
    return y, size


# Rows of the groups, N, bytes of a row.  tests/test_layer_ops_host.py checks that
# they reach every tile.
PRODUCTS = [
    ([1], 1, 1), ([1], 17, 16), ([3], 40, 5), ([1, 0, 2], 33, 64), ([20], 100, 127), ([64], 64, 128), ([5, 0, 11], 48, 129),
    ([10, 6, 0, 1], 77, 349), ([1], 4096, 2048), ([1, 14, 51, 0], 3755, 303), ([130, 0, 257, 1], 136, 192),
    ([250, 0, 258, 262, 209, 116, 174, 1], 2139, 307), ([2048], 2048, 1000), ([2000], 2100, 4096 + 17),
    ([900, 0, 1300, 513, 700, 1111, 600, 1024], 2304, 320), ([1100], 4100, 161), ([70, 3, 0, 150], 88, 144),
    ([1024, 1000, 17], 1024, 512), ([4, 0, 4, 1], 1713, 353), ([30], 4100, 300), ([67, 45, 1, 101, 49, 84, 0, 81], 4059, 661),
    ([1900], 2000, 2501),
]


@pytest.mark.parametrize("sizes,N,K2", PRODUCTS)
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_product_exact(sizes, N, K2, out):
    g = gen(N + K2)
    M, E = sum(sizes) + 3, len(sizes)
    off = [2]
    for n in sizes:
        off.append(off[-1] + n)
    # Multiples of 1/2 under scales of 1/2 and 1: sums are multiples of 2^-4, exact in
    # 32 bits below 2^20.
    a, sa = random_operand(g, (M,), K2, 126, 127)
    b, sb = random_operand(g, (E, N), K2, 126, 127)
    y = torch.full((M, N), 777.0, device="cuda").to(out)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    assert fg.gemm_mx4(a, sa, b, sb, y, offsets=offsets) is y
    want, size = product(a, sa, b, sb, off)
    assert size.max() < 2 ** 20
    rows = slice(off[0], off[-1])
    assert torch.equal(y[rows], want[rows].float().to(out))
    rest = torch.cat([y[:off[0]], y[off[-1]:]]).float()
    assert (rest == torch.tensor(777.0).to(out).float()).all()


@pytest.mark.parametrize("M,N,K2,bias", [(1, 300, 500, True), (40, 77, 1000, False), (300, 500, 2048, True), (257, 1000, 33, False)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_product_rounding(M, N, K2, bias, out):
    g = gen(K2)
    a, sa = random_operand(g, (M,), K2, 110, 130)
    b, sb = random_operand(g, (N,), K2, 100, 128)
    c = torch.randn(N, device="cuda", generator=g) if bias else None
    y = torch.empty(M, N, device="cuda", dtype=out)
    fg.gemm_mx4(a, sa, b, sb, y, bias=c)
    want, size = product(a, sa, b, sb, None, c)
    bound = (2 * K2 + 4) * 2.0 ** -23 * size
    bound = bound + 2.0 ** -24 * (want.abs() + bound) * bias
    bound = bound + HALF_STEP[out] * (want.abs() + bound)
    assert ((y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("pada,padb,padc,skip", [(0, 0, 0, 0), (1, 3, 1, 1), (16, 128, 8, 16), (5, 0, 3, 7)])
def test_product_windows(pada, padb, padc, skip):
    g = gen(9)
    M, N, K2, E = 150, 90, 200, 3

    def window(rows, cols, pad, fill, dtype):
        base = torch.full((rows * (cols + pad) + skip + 16,), fill, device="cuda").to(dtype)
        return base, base[skip:skip + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    _, a = window(M, K2, pada, 0xFF, torch.uint8)
    _, b = window(E * N, K2, padb, 0xFF, torch.uint8)
    b = b.unflatten(0, (E, N))
    qa, sa = random_operand(g, (M,), K2)
    qb, sb = random_operand(g, (E, N), K2)
    a.copy_(qa), b.copy_(qb)
    S = blocks_of(2 * K2)
    tight = torch.full((M * S + skip + 16,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN around the scales
    sa2 = tight[skip:skip + M * S].view(M, S)
    sa2.copy_(sa)
    base, y = window(M, N, padc, 777.0, F32)
    before = base.clone()
    offsets = torch.tensor([0, 70, 70, 150], dtype=torch.int32, device="cuda")
    fg.gemm_mx4(a, sa2, b, sb, y, offsets=offsets)
    want, _ = product(qa, sa, qb, sb, [0, 70, 70, 150])
    assert torch.equal(y, want.float())
    y.fill_(777.0)
    assert torch.equal(base, before), "a byte outside C changed"


@pytest.mark.parametrize("M,N,K2", [(1, 64, 300), (300, 300, 300)])
def test_scales_that_are_no_numbers(M, N, K2):
    # Scale 255 makes its row's results NaN, whatever the codes; the others keep theirs.
    g = gen(3)
    a, sa = random_operand(g, (M,), K2)
    b, sb = random_operand(g, (N,), K2)
    sb[5, -1] = 255
    b[5] = 0
    sb[9, 0], sb[10, 3] = 0, 0  # 2^-127: as good as nothing here
    y = torch.empty(M, N, device="cuda")
    fg.gemm_mx4(a, sa, b, sb, y)
    want, size = product(a, sa, b, sb, None)
    assert torch.isnan(y[:, 5]).all() and torch.isnan(want[:, 5]).all()
    keep = [i for i in range(N) if i != 5]
    assert torch.isfinite(y[:, keep]).all()
    assert ((y.double() - want).abs() <= (2 * K2 + 4) * 2.0 ** -23 * size)[:, keep].all()


def test_product_without_a_reduction():
    bias = torch.randn(8, device="cuda")
    y = torch.full((4, 8), 777.0, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    fg.gemm_mx4(e(4, 0), e(4, 0), e(8, 0), e(8, 0), y, bias=bias)
    assert torch.equal(y, bias.expand(4, 8))
    fg.gemm_mx4(e(4, 0), e(4, 0), e(8, 0), e(8, 0), y)
    assert (y == 0).all()
    fg.gemm_mx4(e(0, 6), e(0, 1), e(8, 6), e(8, 1), torch.empty(0, 8, device="cuda"))


def test_shared_weights_and_wrong_offsets():
    g = gen(12)
    M, N, K2 = 100, 64, 96
    a, sa = random_operand(g, (M,), K2)
    b, sb = random_operand(g, (1, N), K2)
    sb4 = sb.expand(4, N, -1).contiguous()
    y = torch.empty(M, N, device="cuda")
    fg.gemm_mx4(a, sa, b.expand(4, N, K2), sb4, y, offsets=torch.tensor([0, 10, 30, 31, 100], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, product(a, sa, b, sb, None)[0].float())
    base = torch.full((M + 2, N), 777.0, device="cuda")
    for off in ([50, 20, -7, 300, 10], [-5, 1000, -1000, 1 << 30, -(1 << 30)], [100, 100, 0, 0, 100]):
        fg.gemm_mx4(a, sa, b.expand(4, N, K2), sb4, base[1:-1], offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert (base[0] == 777).all() and (base[-1] == 777).all()


def test_quantized_products_stand_for_the_rows():
    # A round trip: rows and weights brought to 4 bits, multiplied, against the
    # products of the values that the codes stand for.
    g = gen(21)
    x, w = torch.randn(70, 515, device="cuda", generator=g).bfloat16(), torch.randn(45, 515, device="cuda", generator=g)
    (q, s), (p, t) = quantized(x), quantized(w)
    y = torch.empty(70, 45, device="cuda")
    fg.gemm_mx4(q, s, p, t, y)
    want, size = product(q, s, p, t, None)
    assert ((y.double() - want).abs() <= (520 + 4) * 2.0 ** -23 * size).all()
    # Each value is off by at most an eighth of its block's largest, or half the
    # distance of 4 and 6, or, where it saturates, from 6 to 8, times the scale.
    def worst(v):
        b = torch.nn.functional.pad(v.double(), (0, -v.shape[1] % 32)).view(v.shape[0], -1, 32).abs().amax(2)
        return (b / 4).repeat_interleave(32, 1)[:, :v.shape[1]]
    assert ((unpack(q, s)[:, :515] - x.double()).abs() <= worst(x)).all()
    assert ((unpack(p, t)[:, :515] - w.double()).abs() <= worst(w)).all()


@pytest.mark.parametrize("M,N", [(3, 5), (40, 70), (700, 600)])
def test_the_longest_reduction(M, N):
    # Rows of 2^22 - 2 values that are zero but for one byte in each of a few blocks, the
    # first and the last among them: the sums are exact.
    g = gen(M)
    K2 = (1 << 21) - 1
    at = torch.cat([torch.tensor([0, K2 - 1], device="cuda"), 16 * torch.randperm(K2 // 16 - 2, device="cuda", generator=g)[:6] + 19])
    block, inside = at // 16, at % 16
    wide, short = [], []
    for rows in (M, N):
        codes = torch.randint(0, 256, (rows, len(at)), dtype=torch.uint8, device="cuda", generator=g)
        s = torch.randint(126, 129, (rows, len(at)), dtype=torch.uint8, device="cuda", generator=g)
        q, scale = torch.zeros(rows, K2, dtype=torch.uint8, device="cuda"), torch.full((rows, (K2 + 15) // 16), 127, dtype=torch.uint8, device="cuda")
        q[:, at], scale[:, block] = codes, s
        p = torch.zeros(rows, len(at), 16, dtype=torch.uint8, device="cuda")
        p[:, torch.arange(len(at), device="cuda"), inside] = codes
        wide += [q, scale]
        short += [p.view(rows, -1), s]
    y = torch.full((M, N), 777.0, device="cuda")
    fg.gemm_mx4(*wide, y)
    assert torch.equal(y.double(), product(*short, None)[0])
