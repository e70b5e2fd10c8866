"""Corners of the grouped and 8-bit products on the GPU: errors of the program
around them, launches past what one grid dimension holds, wrong offsets, bad
values and every compiled tile."""
import pytest
import torch

import fp32_gemm_amd as fg
from fp32_gemm_amd.binding import _lib

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, shape, dtype, most=3):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).to(dtype)


def offsets_of(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def test_an_earlier_error_is_left_to_the_program():
    # A failed call of the program's own leaves its error with the runtime. The
    # products neither report nor clear it.
    g = gen(1)
    x, w, o = whole(g, (40, 32), BF16), whole(g, (2, 32, 24), BF16), offsets_of([0, 10, 40])
    y, dw = torch.empty(40, 24, dtype=BF16, device="cuda"), torch.empty(2, 32, 24, dtype=F32, device="cuda")
    q, s, z = torch.empty(40, 32, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda"), torch.empty(40, 40, device="cuda")
    torch.cuda.synchronize()
    assert _lib.hipSetDevice(9999) != 0
    left = _lib.hipPeekAtLastError()
    try:
        fg.gemm_grouped(x, w, o, y)
        fg.gemm_grouped_wgrad(x, y, o, dw)
        fg.quantize_rows(x, q, s)
        fg.igemm(q, s, q, s, z)
        assert _lib.hipPeekAtLastError() == left
    finally:
        _lib.hipGetLastError()
    assert left != 0
    want = torch.cat([x[:10].double() @ w[0].double(), x[10:].double() @ w[1].double()])
    assert torch.equal(y, want.to(BF16))


# ---- every compiled tile of every form and type ------------------------------------
# tests/test_grouped_edges_host.py checks that these sizes reach each of them.

PRODUCTS = [  # rows of the groups, K, N
    ([10, 6, 0, 1], 349, 77),
    ([1, 14, 51, 0], 303, 3755),
    ([250, 0, 258, 262, 209, 116, 174, 1], 307, 2139),
    ([4, 0, 4, 1], 353, 1713),
    ([941, 321, 0, 1253, 663, 976, 1, 346], 301, 2881),
    ([1, 147, 119, 187, 140, 78, 204, 0], 311, 4053),
    ([67, 45, 1, 101, 49, 84, 0, 81], 661, 4059),
]
WEIGHT_GRADIENTS = [  # rows of the groups, K, N
    ([121, 1, 337, 0], 247, 85),
    ([1, 0, 200, 91], 203, 3045),
    ([0, 310, 100, 1, 75], 751, 3543),
    ([0, 130, 20, 1, 75], 751, 3543),
    ([1, 0, 77, 31], 203, 3045),
    ([149, 240, 172, 351, 1, 518, 0, 285], 1555, 133),
    ([211, 563, 261, 1, 359, 155, 282, 0], 217, 3653),
]


def layout(sizes):
    """Offsets of groups that leave one row in front and two behind."""
    off = [1]
    for n in sizes:
        off.append(off[-1] + n)
    return off, off[-1] + 2


def spans(off):
    return [slice(off[e], off[e + 1]) for e in range(len(off) - 1)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,K,N", PRODUCTS)
def test_products_in_every_tile(sizes, K, N, transposed, dtype):
    # Whole numbers: sums are exact in 32 bits, the result is rounded once.
    g = gen(2)
    off, M = layout(sizes)
    x = whole(g, (M, K), dtype)
    w = whole(g, (len(sizes), N, K) if transposed else (len(sizes), K, N), dtype)
    y = torch.full((M, N), 77.0, device="cuda", dtype=dtype)
    want = y.clone()
    for e, rows in enumerate(spans(off)):
        we = w[e].double()
        want[rows] = (x[rows].double() @ (we.t().contiguous() if transposed else we)).to(dtype)
    fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=transposed)
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("sizes,K,N", WEIGHT_GRADIENTS)
def test_weight_gradients_in_every_tile(sizes, K, N, dtype):
    g = gen(3)
    off, M = layout(sizes)
    x, dy = whole(g, (M, K), dtype), whole(g, (M, N), dtype)
    dw = torch.full((len(sizes), K, N), float("nan"), device="cuda", dtype=dtype)
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    want = torch.stack([x[rows].double().t().contiguous() @ dy[rows].double() for rows in spans(off)])
    assert torch.equal(dw, want.to(dtype))


@pytest.mark.parametrize("sizes,K,N", PRODUCTS)
def test_8_bit_products_in_every_tile(sizes, K, N):
    g = gen(4)
    off, M = layout(sizes)
    E = len(sizes)
    a, b = whole(g, (M, K), torch.int8, 127), whole(g, (E, N, K), torch.int8, 127)
    # Powers of two, and sums below 2^24: the result is exact in 32 bits.
    sa = torch.exp2(torch.randint(-8, 0, (M,), device="cuda", generator=g).float())
    sb = torch.exp2(torch.randint(-8, 0, (E, N), device="cuda", generator=g).float())
    y = torch.full((M, N), 77.0, device="cuda")
    want = y.clone()
    for e, rows in enumerate(spans(off)):
        want[rows] = ((a[rows].double() @ b[e].double().t().contiguous()) * sa[rows, None].double() * sb[e].double()).float()
    fg.igemm(a, sa, b, sb, y, offsets=offsets_of(off))
    assert torch.equal(y, want)


# ---- as many rows as there may be ----------------------------------------------------

def test_a_thousand_million_rows():
    # Tiles of 128 rows and 512 threads would take 2^32 threads.
    M, K, N = 1 << 30, 8, 8
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    w = torch.arange(64, device="cuda").view(K, N).to(BF16)
    y = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 1, 255, 256, (1 << 29) - 1, 1 << 29, M - 257, M - 2, M - 1], device="cuda")
    x[rows] = whole(gen(5), (len(rows), K), BF16)
    fg.gemm_grouped(x, w, None, y)
    assert torch.equal(y[rows], (x[rows].double() @ w.double()).to(BF16))
    y[rows] = 0
    assert not y.view(torch.int64).any()


def test_quantising_more_rows_than_a_grid_dimension_holds():
    # Past 2^26 rows, four to a workgroup of 256 threads, x alone would need 2^32.
    M, K = (1 << 26) + 5, 8
    x = torch.ones(M, K, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 3, 4, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, (1 << 26) - 1, 1 << 26, M - 1], device="cuda")
    x[rows] = torch.arange(1, 10, device="cuda").to(BF16)[:, None] * 2
    x[rows, 0] = 0.5
    q = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    s = torch.zeros(M, device="cuda")
    fg.quantize_rows(x, q, s)
    top = torch.arange(1, 10, device="cuda").double() * 2
    want = torch.full((9, K), 127, dtype=torch.int8, device="cuda")
    want[:, 0] = torch.round(127 * 0.5 / top).to(torch.int8)
    assert torch.equal(q[rows], want) and torch.equal(s[rows], (top / 127).float())
    q[rows], s[rows] = 127, 1.0 / 127
    assert (q == 127).all() and (s == 1.0 / 127).all()


# ---- wrong offsets, bad values ---------------------------------------------------------

def guarded(rows, cols, dtype, fill):
    """A rows x cols view amid `fill`, its rows 8 elements more than cols apart."""
    base = torch.full((rows + 4, cols + 8), fill, device="cuda").to(dtype)
    return base, base[2:2 + rows, :cols]


WRONG = [[50, 20, -7, 300, 10], [-5, 1000, -1000, 1 << 30, -(1 << 30)], [100, 100, 0, 0, 100], [0, 90, 30, 60, 2000]]


def spans_of_wrong(off, M):
    out = []
    for e in range(len(off) - 1):
        lo = min(max(off[e], 0), M)
        out.append(slice(lo, min(max(off[e + 1], lo), M)))
    return out


MANY_WRONG = [[0 if e % 2 else 4000 for e in range(151)],  # more tiles than the rows can have: nothing is computed
              [-5 if e == 0 else 26 * (e + (e == 70) - (e == 71)) for e in range(151)]]


@pytest.mark.parametrize("off", WRONG + MANY_WRONG)
@pytest.mark.parametrize("M,K,N", [(100, 64, 64), (4000, 72, 1100), (4000, 72, 3600)])
@pytest.mark.parametrize("dtype,trans", [(BF16, True), (BF16, False), (F32, False), (torch.int8, True)])
def test_wrong_offsets_write_products_of_their_own_rows(off, M, K, N, dtype, trans):
    # Whatever the offsets hold, an output is left alone or the product of its own
    # row of X and some group's weights; what surrounds the operands (NaN, or codes
    # that no product has) neither enters nor changes.
    g = gen(20)
    E = len(off) - 1
    if N == 3600:
        assert fg.grouped.plan("nt" if trans else "nn", dtype, E, M, N, K, out=F32)["BM"] == 256
    _, x = guarded(M, K, dtype, 99 if dtype is torch.int8 else float("nan"))
    x.copy_(whole(g, (M, K), dtype))
    _, w2 = guarded(E * (N if trans else K), K if trans else N, dtype, 99 if dtype is torch.int8 else float("nan"))
    w = w2.unflatten(0, (E, N if trans else K))
    w.copy_(whole(g, tuple(w.shape), dtype))
    yb, y = guarded(M, N, F32, 7777.0)
    before = yb.clone()
    if dtype is torch.int8:
        one = torch.ones(E, N, device="cuda")
        fg.igemm(x, torch.ones(M, device="cuda"), w, one, y, offsets=offsets_of(off))
    else:
        fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=trans)
    known = y == 7777.0
    for e in range(E):
        we = w[e].float()
        known |= y == x.float() @ (we.t().contiguous() if trans else we)
    assert known.all()
    if off in (WRONG[0], WRONG[2], MANY_WRONG[1]):  # no more tiles than groups in order can have
        assert (y != 7777.0).any()
    y.copy_(before[2:2 + M, :N])
    assert torch.equal(yb, before)


@pytest.mark.parametrize("off", WRONG)
@pytest.mark.parametrize("dtype,K,N", [(BF16, 72, 100), (F32, 72, 100), (F16, 1000, 1030), (F32, 1000, 1030)])
def test_weight_gradients_of_wrong_offsets(off, dtype, K, N):
    g = gen(21)
    M, E = 1500, len(off) - 1
    _, x = guarded(M, K, dtype, float("nan"))
    _, dy = guarded(M, N, dtype, float("nan"))
    x.copy_(whole(g, (M, K), dtype))
    dy.copy_(whole(g, (M, N), dtype))
    wb, w2 = guarded(E * K, N, F32, 7777.0)
    before = wb.clone()
    dw = w2.unflatten(0, (E, K))
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    for e, rows in enumerate(spans_of_wrong(off, M)):
        assert torch.equal(dw[e], (x[rows].double().t().contiguous() @ dy[rows].double()).float())
    w2.copy_(before[2:2 + E * K, :N])
    assert torch.equal(wb, before)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("sizes,K,N", [([40, 25], 160, 96), ([40, 25], 161, 97), ([600, 700], 161, 2100)])
def test_bad_values_stay_in_their_rows_and_columns_with_transposed_weights(dtype, sizes, K, N):
    g = gen(22)
    off, M = layout(sizes)
    x, w = whole(g, (M, K), dtype), whole(g, (2, N, K), dtype)
    w[w == 0] = 1
    x[7, 3], x[50, K - 1], w[1, 11, K - 1], w[0, N - 1, 0] = float("nan"), float("inf"), float("nan"), -float("inf")
    x[off[1] - 1, K - 1] = float("inf")
    y = torch.full((M, N), 7.0, device="cuda", dtype=F32)
    want = y.clone()
    for e, rows in enumerate(spans(off)):
        want[rows] = (x[rows].double() @ w[e].double().t().contiguous()).float()
    fg.gemm_grouped(x, w, offsets_of(off), y, transpose_w=True)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(y[fine], want[fine])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K,N", [(72, 96), (73, 97), (1000, 1030)])
def test_bad_values_stay_in_their_group_row_and_column_of_weight_gradients(dtype, K, N):
    # A bad token spoils its own group's weights: one row of dW by X, one column by
    # dY. Rows that no group owns, in front and behind, spoil nothing.
    g = gen(23)
    off, M = layout([130, 0, 257])
    x, dy = whole(g, (M, K), dtype), whole(g, (M, N), dtype)
    for t in (x, dy):
        t[t == 0] = 1
        t[0], t[-2:] = float("nan"), float("inf")
    x[5, 3], x[140, K - 1], dy[130, 2], dy[M - 3, N - 1] = float("nan"), float("inf"), float("inf"), float("nan")
    dw = torch.full((3, K, N), 7.0, device="cuda")
    fg.gemm_grouped_wgrad(x, dy, offsets_of(off), dw)
    want = torch.stack([x[rows].double().t().contiguous() @ dy[rows].double() for rows in spans(off)]).float()
    assert torch.equal(torch.isnan(dw), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(dw[fine], want[fine])
