"""The norm, its 8-bit output and its gradient on the GPU against 64 bits.

H rounds once in 32 bits, so its squares are off by 2 * 2^-24 and s by half of that.
Y = H * s * weight: H, what s has from it, s itself and two products round, so Y is off
by at most 5 * 2^-24 of itself, and half a step of its type.  The scale is made in 64
bits from the exact largest value and s, and rounded once: 2 * 2^-24.  Codes must be
those of the quotients in 64 bits.
"""
import pytest
import torch

import fp32_gemm_amd as fg

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in (F32, BF16, F16)}
CANARY = 777.0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def window(rows, cols, pad, dtype, skip=0, fill=float("nan")):
    ld = cols + pad
    base = torch.full((rows * ld + skip + 64,), fill, device="cuda").to(dtype)
    return base, base[skip:skip + rows * ld].view(rows, ld)[:, :cols]


def reference(x, r, w, eps):
    h = x.double() if r is None else x.double() + r.double()
    s = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    v = h if w is None else h * w.double()
    return h, s, v


def codes_of(v, s):
    top = v.abs().amax(1, keepdim=True) if v.shape[1] else torch.zeros(v.shape[0], 1, dtype=torch.float64, device="cuda")
    usable = torch.isfinite(v).all(1, keepdim=True)
    q = torch.where(usable & (top > 0), torch.round(v * 127 / torch.where(top > 0, top, 1)), 0.0)
    scale = torch.where(usable, top / 127 * s, float("nan"))[:, 0]
    return q.nan_to_num().to(torch.int8), scale


def check(x, r, w, eps, y=None, h=None, q=None, scale=None):
    H, s, v = reference(x, r, w, eps)
    if h is not None:
        assert torch.equal(h, (x.float() + r.float() if r is not None else x).to(h.dtype))
    if y is not None:
        want = v * s
        bound = want.abs() * (5 * 2.0 ** -24 + HALF_STEP[y.dtype]) * 1.01 + TINY[y.dtype]
        assert ((y.double() - want).abs() <= bound).all()
    if q is not None:
        code, sc = codes_of(v, s)
        assert torch.equal(q, code)
        assert ((scale.double() - sc).abs() <= sc.abs() * (2 * 2.0 ** -24 + 2.0 ** -40)).all()


SIZES = [(1, 1), (1, 7), (3, 64), (5, 100), (2, 511), (4, 512), (9, 1031), (6, 2048), (3, 4097), (2, 8192), (1, 16384), (2, 16390),
         (1, 70001), (4100, 1000), (4096, 2053)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(dtype, M, K):
    g = gen(M * 1000003 + K)
    x = torch.randn(M, K, device="cuda", generator=g).to(dtype)
    r = (3 * torch.randn(M, K, device="cuda", generator=g)).to(dtype)
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)
    for weight in (w.to(dtype), w, None):
        y, h = torch.empty_like(x), torch.empty_like(x)
        q, scale = torch.empty(M, K, device="cuda", dtype=torch.int8), torch.empty(M, device="cuda")
        assert fg.rms_norm(x, weight, y, residual=r, H=h, Q=q, scale=scale) is y
        check(x, r, weight, 1e-6, y, h, q, scale)
    wide = torch.empty(M, K, device="cuda")
    assert fg.rms_norm(x, w, wide, eps=1e-3) is wide
    check(x, None, w, 1e-3, wide)
    got = fg.rms_norm(x, w.to(dtype), Q=q, scale=scale, eps=0.0)
    assert got[0] is q and got[1] is scale
    check(x, None, w.to(dtype), 0.0, None, None, q, scale)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K", [130, 4096, 16500])
def test_in_place(dtype, K):
    g = gen(K)
    x = torch.randn(3, K, device="cuda", generator=g).to(dtype)
    r = torch.randn(3, K, device="cuda", generator=g).to(dtype)
    w = torch.randn(K, device="cuda", generator=g).to(dtype)
    y = torch.empty_like(x)
    q, scale = torch.empty(3, K, device="cuda", dtype=torch.int8), torch.empty(3, device="cuda")
    for target in ("residual", "X"):
        a, b = x.clone(), r.clone()
        h = b if target == "residual" else a
        fg.rms_norm(a, w, y, residual=b, H=h, Q=q, scale=scale)
        check(x, r, w, 1e-6, y, h, q, scale)
        assert torch.equal(a if h is b else b, x if h is b else r)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pads,skip", [((0, 0, 0, 0, 0), 0), ((3, 5, 1, 7, 2), 1), ((8, 16, 8, 8, 16), 8), ((1, 0, 4, 2, 3), 5)])
@pytest.mark.parametrize("K", [333, 2500])
def test_windows(dtype, pads, skip, K):
    g, M = gen(4), 11
    _, x = window(M, K, pads[0], dtype, skip)
    _, r = window(M, K, pads[1], dtype, skip)
    x.copy_(torch.randn(M, K, device="cuda", generator=g)), r.copy_(torch.randn(M, K, device="cuda", generator=g))
    w = torch.full((K + 2 * skip + 8,), float("nan"), device="cuda", dtype=dtype)[skip:skip + K]
    w.copy_(torch.randn(K, device="cuda", generator=g))
    hb, h = window(M, K, pads[2], dtype, skip, CANARY)
    yb, y = window(M, K, pads[3], F32, skip, CANARY)
    qb, q = window(M, K, pads[4], torch.int8, skip, 99)
    sb = torch.full((M + 2,), CANARY, device="cuda")
    before = [t.clone() for t in (hb, yb, qb)]
    fg.rms_norm(x, w, y, residual=r, H=h, Q=q, scale=sb[1:-1])
    check(x, r, w, 1e-6, y, h, q, sb[1:-1])
    h.fill_(CANARY), y.fill_(CANARY), q.fill_(99)
    for base, was in zip((hb, yb, qb), before):
        assert torch.equal(base, was), "a byte outside an output changed"
    assert sb[0] == CANARY and sb[-1] == CANARY


def test_codes_on_ties():
    # 127 v / max|v| lies on n + 1/2 exactly, and a step of 2^-23 and of 2^-30 beside it.
    n = torch.arange(0, 127, dtype=torch.float64, device="cuda") + 0.5
    for K in (160, 1200):
        v = torch.zeros(4, K, dtype=torch.float64, device="cuda")
        v[:, :127] = n
        v[:, 127] = 127
        v[1, :127] *= 1 + 2.0 ** -23
        v[2, :127] *= 1 - 2.0 ** -23
        x = v.float()
        x[3] = v[3].float() * -1
        assert torch.equal(x[0].double(), v[0])
        q, scale = torch.empty(4, K, device="cuda", dtype=torch.int8), torch.empty(4, device="cuda")
        fg.rms_norm(x, None, Q=q, scale=scale)
        check(x, None, None, 1e-6, None, None, q, scale)
        # With a residual and weights the products pass 32 bits.
        r = x * 2.0 ** -18
        w = torch.full((K,), 1 + 2.0 ** -20, device="cuda")
        fg.rms_norm(x, w, residual=r, Q=q, scale=scale)
        check(x, r, w, 1e-6, None, None, q, scale)


@pytest.mark.parametrize("K", [96, 3000])
def test_extremes(K):
    # Squares that leave 32 bits, rows of zeros, the smallest numbers.
    g = gen(K)
    base = torch.randn(6, K, device="cuda", generator=g)
    x = base * torch.tensor([1e30, 1e-30, 1e-42, 1.0, 3e37, 1e-20], device="cuda")[:, None]
    x[3] = 0
    w = 1 + 0.1 * torch.randn(K, device="cuda", generator=g)
    for eps in (1e-6, 0.0):
        rows = [0, 1, 2, 4, 5] if eps == 0 else list(range(6))
        y = torch.empty_like(x)
        q, scale = torch.empty(6, K, device="cuda", dtype=torch.int8), torch.empty(6, device="cuda")
        fg.rms_norm(x, w, y, Q=q, scale=scale, eps=eps)
        H, s, v = reference(x, None, w, eps)
        want = (v * s)[rows]
        assert ((y[rows].double() - want).abs() <= want.abs() * 6 * 2.0 ** -24 * 1.01 + 2.0 ** -149).all()
        code, sc = codes_of(v, s)
        assert torch.equal(q, torch.where(torch.isfinite(scale)[:, None], code, q))
        assert ((scale[rows].double() - sc[rows]).abs() <= sc[rows].abs() * (2 * 2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150).all()
        if eps:
            assert (q[3] == 0).all() and scale[3] == 0 and (y[3] == 0).all()


@pytest.mark.parametrize("K", [70, 3000])
def test_values_that_are_no_numbers(K):
    x = torch.ones(5, K, device="cuda")
    x[1, 3], x[2, K - 1], x[3, 0] = float("inf"), float("nan"), float("-inf")
    w = torch.ones(K, device="cuda")
    y = torch.empty_like(x)
    q, scale = torch.empty(5, K, device="cuda", dtype=torch.int8), torch.empty(5, device="cuda")
    fg.rms_norm(x, w, y, Q=q, scale=scale)
    assert torch.isnan(scale[1:4]).all() and (q[1:4] == 0).all()
    assert torch.isfinite(scale[[0, 4]]).all() and (q[[0, 4]] == 127).all()
    assert torch.isnan(y[1, 3]) and (y[1, 4:] == 0).all() and torch.isnan(y[2]).all()
    w[5] = float("nan")  # a weight spoils its column, and every row's codes
    fg.rms_norm(x, w, y, Q=q, scale=scale)
    assert torch.isnan(scale).all() and (q == 0).all()
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[0, :5]).all()


def test_empty():
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    scale = torch.full((3,), CANARY, device="cuda")
    fg.rms_norm(e(3, 0), None, Q=e(3, 0).to(torch.int8), scale=scale)
    assert (scale == 0).all()
    fg.rms_norm(e(0, 5), e(5), e(0, 5))
    dw = torch.full((5,), CANARY, device="cuda")
    fg.rms_norm_grad(e(0, 5), e(0, 5), e(5), e(0, 5), dw)
    assert (dw == 0).all()
    fg.rms_norm_grad(e(3, 0), e(3, 0), e(0), e(3, 0), e(0))


# ---- the gradient -------------------------------------------------------------------

def gradient(dy, h, w, dh, eps):
    h, dy = h.double(), dy.double()
    s = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    g = dy if w is None else dy * w.double()
    n = h * s
    mean = (g * n).mean(1, keepdim=True)
    dx = s * (g - n * mean)
    # s, g, the products and sums round once each; n twice, the mean's terms and s.
    size = 2.0 ** -24 * (5 * (s * g).abs() + 8 * s * n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + 2.0 ** -24 * dx.abs()
    dw = (dy * n).sum(0)
    return dx, size, dw, (h.shape[0] + 8) * 2.0 ** -24 * (dy * n).abs().sum(0)


def check_gradient(dy, h, w, dh, eps, dx, dw):
    want, size, want_w, size_w = gradient(dy, h, w, dh, eps)
    assert ((dx.double() - want).abs() <= 1.01 * size + HALF_STEP[dx.dtype] * (want.abs() + size) + TINY[dx.dtype]).all()
    if dw is not None:
        assert ((dw.double() - want_w).abs() <= 1.01 * size_w + HALF_STEP[dw.dtype] * (want_w.abs() + size_w) + TINY[dw.dtype]).all()


GRADS = [(1, 1), (2, 7), (5, 64), (600, 100), (3, 513), (700, 1031), (4, 2048), (17, 4097), (3, 8192), (2, 16390), (2, 33000),
         (1500, 257), (20000, 40)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K", GRADS)
def test_gradient(dtype, M, K):
    g = gen(M + 7 * K)
    h, dy, dh = (torch.randn(M, K, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)
    for weight, into, more in ((w.to(dtype), dtype, dh), (w, F32, None), (None, F32, dh)):
        dx, dw = torch.empty_like(h), torch.full((K,), CANARY, device="cuda").to(into)
        got = fg.rms_norm_grad(dy, h, weight, dx, dw, residual_grad=more)
        assert got[0] is dx and got[1] is dw
        check_gradient(dy, h, weight, more, 1e-6, dx, dw)
    again = torch.empty_like(dw)
    fg.rms_norm_grad(dy, h, None, dx, again, residual_grad=dh,
                     workspace=torch.empty(fg.layers.rms_norm_grad_workspace(M, K), dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, dw)
    fg.rms_norm_grad(dy, h, w, dx)  # without the weight's
    check_gradient(dy, h, w, None, 1e-6, dx, None)


@pytest.mark.parametrize("K", [200, 3001, 20000])
def test_gradient_in_place_and_windows(K):
    g, M = gen(K), 9
    for dtype in (F32, BF16):
        h, dy, dh = (window(M, K, p, dtype, 3)[1] for p in (1, 8, 5))
        for t in (h, dy, dh):
            t.copy_(torch.randn(M, K, device="cuda", generator=g))
        w = torch.randn(K, device="cuda", generator=g).to(dtype)
        base, dx = window(M, K, 7, dtype, 5, CANARY)
        before = base.clone()
        dw = torch.empty(K, device="cuda")
        fg.rms_norm_grad(dy, h, w, dx, dw, residual_grad=dh)
        check_gradient(dy, h, w, dh, 1e-6, dx, dw)
        kept = dx.clone()
        dx.fill_(CANARY)
        assert torch.equal(base, before), "a byte outside dX changed"
        for t in (dy, dh):
            a = t.clone()
            fg.rms_norm_grad(a if t is dy else dy, h, w, a, None, residual_grad=a if t is dh else dh)
            assert torch.equal(a, kept)


def test_gradient_against_differences():
    # f(x, w) = sum(c * norm(x) w): central differences of the forward call in 32 bits, whose
    # values are off by some 5 * 2^-24 of their sum of magnitudes, over a step of 2^-7.
    g = gen(8)
    M, K, step = 4, 24, 2.0 ** -7
    x, c = (torch.randn(M, K, device="cuda", generator=g) for _ in range(2))
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)

    def f(x, w):
        y = torch.empty_like(x)
        return (fg.rms_norm(x, w, y, eps=1e-5).double() * c.double()).sum()

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    fg.rms_norm_grad(c, x, w, dx, dw, eps=1e-5)
    noise = 6 * 2.0 ** -24 * (2 * c.abs().sum().item()) * 3 / step  # |norm w| is below 3 nearly throughout
    for grad, v, call in ((dx, x, lambda t: f(t, w)), (dw, w, lambda t: f(x, t))):
        for i in range(v.numel()):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += step
            down.view(-1)[i] -= step
            real = (up.view(-1)[i] - down.view(-1)[i]).item()
            diff = (call(up) - call(down)).item() / real
            # The third derivative over six times the step squared: below 30 here.
            assert abs(grad.view(-1)[i].item() - diff) <= noise + 30 * step ** 2


def test_no_columns_and_no_eps():
    scale = torch.full((3,), CANARY, device="cuda")
    fg.rms_norm(torch.empty(3, 0, device="cuda"), None, Q=torch.empty(3, 0, dtype=torch.int8, device="cuda"), scale=scale, eps=0.0)
    assert (scale == 0).all()


@pytest.mark.parametrize("K", [40, 3000, 20000])
def test_gradient_of_huge_and_tiny_rows(K):
    g = gen(K + 2)
    size = torch.tensor([1e38, 1e37, 1e-38, 1e-37, 1e30, 1.0], device="cuda")[:, None]
    h = size * (1 + torch.rand(6, K, device="cuda", generator=g))
    # Gradients that keep dX among the ordinary numbers, where half a step is relative.
    dy = torch.randn(6, K, device="cuda", generator=g) * size.clamp(1e-18, 1e18)
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)
    dx, dw = torch.empty_like(h), torch.empty(K, device="cuda")
    fg.rms_norm_grad(dy, h, w, dx, dw, eps=0.0)
    check_gradient(dy, h, w, None, 0.0, dx, dw)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M", [256, 512, 513])
@pytest.mark.parametrize("K", [2100, 3001, 6005, 12000, 18003])
def test_long_rows_few_and_many(dtype, M, K):
    test_norm(dtype, M, K)
