"""Where the norm, its gradient and the layer of experts leave the ordinary range:
sums and products that pass 32 bits, hidden values that pass 16, scale bytes at the
ends, rows of the longest kinds.  Bounds count roundings, as in the files whose
references are used here.
"""
import pytest
import torch

import fp32_gemm_amd as fg
from test_expert_layer_gpu import HALF_STEP, TINY, make_weights

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# Hidden values of 16-bit tokens are sums of two bfloat16: the first leaves at most half
# a step, 2^-8 of the value's power of two, and the second half a step of that, 2^-17.
HELD = {F32: 2.0 ** -24, BF16: 2.0 ** -17, F16: 2.0 ** -17}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def layer_reference(x, ids, share, w_in, w_out, gated, held, scaled):
    """y in 64 bits and how far a result may be off before its own rounding, as in
    test_expert_layer_gpu, with hidden values that are off by `held` of themselves."""
    x, share = x.double(), share.double()
    y, off = torch.zeros(x.shape[0], w_out.shape[1], dtype=torch.float64, device="cuda"), 0
    off = torch.zeros_like(y)
    step, F, deep = 2.0 ** -24, w_out.shape[2], w_in.shape[2]
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w_in.shape[0]:
                continue
            u = w_in[e] @ x[t]
            du = (2 * (deep + 4) + 2 * scaled) * step * (w_in[e].abs() @ x[t].abs())
            a, da = (u[:F], du[:F]) if gated else (u, du)
            h = a * torch.sigmoid(a)
            dh = 1.1 * da + 8 * step * h.abs()
            if gated:
                dh = dh * (u[F:].abs() + du[F:]) + h.abs() * du[F:]
                h = h * u[F:]
                dh = dh + step * h.abs()
            dh = dh + held * (h.abs() + dh) + 2.0 ** -133
            y[t] += share[t, j] * (w_out[e] @ h)
            # Products of two parts of a value by up to two of a weight: up to 4 F sums.
            off[t] += share[t, j].abs() * (w_out[e].abs() @ dh + (2 * (4 * F + 4) + 2 * scaled + 24) * step * (w_out[e].abs() @ (h.abs() + dh)))
    return y, off


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("E,T,top,D,F", [(3, 1, 2, 64, 64), (8, 16, 2, 96, 200), (5, 3, 2, 40, 77), (4, 20, 2, 70, 129), (12, 9, 3, 64, 7),
                                         (2, 2, 1, 33, 2500), (2, 30, 1, 33, 2500), (3, 18, 1, 96, 1030), (24, 12, 2, 520, 96),
                                         (16, 20, 2, 2100, 1100), (16, 20, 1, 2056, 2047), (32, 20, 2, 2100, 600)])
def test_hidden_values_keep_their_bits(dtype, kind, E, T, top, D, F):
    # Results in 32 bits show how the values between the two products were held.
    g = gen(E + F)
    for gated in (True, False):
        x = torch.randn(T, D, device="cuda", generator=g).to(dtype)
        w_in, s_in, v_in = make_weights(g, kind, E, 2 * F if gated else F, D, dtype)
        w_out, s_out, v_out = make_weights(g, kind, E, D, F, dtype)
        ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:top] for _ in range(T)]).to(torch.int32)
        share = torch.rand(T, top, device="cuda", generator=g)
        y = torch.empty(T, D, device="cuda")
        fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out, gated=gated)
        want, off = layer_reference(x, ids, share, v_in, v_out, gated, HELD[dtype], kind == "int8")
        assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32]).all()


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
@pytest.mark.parametrize("E,T", [(2, 3), (12, 30)])
def test_hidden_values_past_16_bits(kind, E, T):
    # u * silu(u) passes 65504, the largest of float16, and the result does not.
    g = gen(T)
    D, F = 64, 40
    x = torch.randn(T, D, device="cuda", generator=g).half() * 40
    w_in, s_in, v_in = make_weights(g, kind, E, 2 * F, D, F16)
    if kind == "same":
        w_in, v_in = w_in * 16, v_in * 16
    elif kind == "int8":
        s_in, v_in = s_in * 16, v_in * 16
    else:
        s_in, v_in = s_in + 4, v_in * 16
    w_out, s_out, v_out = make_weights(g, kind, E, D, F, F16)
    if kind == "same":
        w_out = w_out * 2.0 ** -8
        v_out = w_out.double()
    elif kind == "int8":
        s_out, v_out = s_out * 2.0 ** -8, v_out * 2.0 ** -8
    else:
        s_out, v_out = s_out - 8, v_out * 2.0 ** -8
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    share = torch.rand(T, 1, device="cuda", generator=g)
    u = torch.stack([v_in[int(e)] @ row for e, row in zip(ids[:, 0], x.double())])
    assert (torch.nn.functional.silu(u[:, :F]) * u[:, F:]).abs().amax(1).min() > 70000
    y = torch.empty(T, D, dtype=F16, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out)
    want, off = layer_reference(x, ids, share, v_in, v_out, True, HELD[F16], kind == "int8")
    assert want.abs().max() < 60000
    assert ((y.double() - want).abs() <= off + HALF_STEP[F16] * (want.abs() + off) + TINY[F16]).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("E,T", [(2, 3), (12, 30)])
def test_infinite_hidden_values(dtype, E, T):
    # Weights of one sign, zeros of the lower bits among them: infinite sums, not NaN.
    x = torch.ones(T, 64, device="cuda", dtype=dtype)
    x[0, 5] = float("inf")
    w_in = torch.ones(E, 16, 64, device="cuda", dtype=dtype)
    w_out = (1 + torch.arange(16, device="cuda") / 1024).to(dtype).expand(E, 64, 16).contiguous()
    y = torch.empty_like(x)
    ids = torch.arange(T, device="cuda", dtype=torch.int32)[:, None] % E
    fg.expert_layer(x, ids, torch.ones(T, 1, device="cuda"), w_in, w_out, y, gated=False)
    assert (y[0] == float("inf")).all() and torch.isfinite(y[1:]).all()


def norm_reference(x, r, w, eps):
    """y, scales and codes in 64 bits, from the sum that is not rounded."""
    h = x.double() + r.double()
    s = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    v = h if w is None else h * w.double()
    top = v.abs().amax(1, keepdim=True)
    q = torch.round(v * 127 / torch.where(top > 0, top, 1.0))
    return v * s, (top / 127 * s)[:, 0], q.to(torch.int8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K", [(5, 1), (5, 96), (5, 3001), (600, 2100), (5, 40000), (4100, 1500), (300, 9000)])
def test_norm_of_sums_past_32_bits(dtype, M, K):
    # X + R passes the largest float where neither does: Y, scale and codes are made from
    # the sum itself, and H alone is infinite.
    g = gen(K)
    x = torch.randn(M, K, device="cuda", generator=g)
    r = torch.randn(M, K, device="cuda", generator=g)
    for row, factor in ((0, 1.0), (1, -1.0), (3, 0.9)):
        x[row], r[row] = x[row].clamp(-1.5, 1.5) * 1e38, r[row].clamp(-1.5, 1.5) * 1e38
        x[row, K // 2], r[row, K // 2] = factor * 3.3e38, factor * 2e38
    x[4], r[4] = 3e38, 3e38
    x, r = x.to(dtype), r.to(dtype)
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)
    for weight in (w, w.to(dtype), None):
        want, ws, wq = norm_reference(x, r, weight, 1e-6)
        bound = want.abs() * 5 * 2.0 ** -24 * 1.01 + TINY[F32]
        y, h = torch.empty(M, K, device="cuda"), torch.empty_like(x)
        q, scale = torch.empty(M, K, device="cuda", dtype=torch.int8), torch.empty(M, device="cuda")
        fg.rms_norm(x, weight, y, residual=r, H=h, Q=q, scale=scale)
        assert ((y.double() - want).abs() <= bound).all()
        assert ((scale.double() - ws).abs() <= ws * (2 * 2.0 ** -24 + 2.0 ** -40)).all()
        assert torch.equal(q, wq)
        assert torch.equal(h, (x.float() + r.float()).to(dtype)) and torch.isinf(h[0, K // 2])
        fg.rms_norm(x, weight, y.fill_(0), residual=r)
        assert ((y.double() - want).abs() <= bound).all()
        a = r.clone()  # H in the residual's place, nothing else in 32 bits
        fg.rms_norm(x, weight, residual=a, H=a, Q=q.fill_(0), scale=scale.fill_(0))
        assert torch.equal(q, wq) and torch.equal(a, h)
        assert ((scale.double() - ws).abs() <= ws * (2 * 2.0 ** -24 + 2.0 ** -40)).all()


@pytest.mark.parametrize("K", [70, 3000, 20000])
def test_sums_of_infinities_are_no_numbers(K):
    x, r = torch.ones(4, K, device="cuda"), torch.ones(4, K, device="cuda")
    x[0, 3], r[1, K - 1], x[2, 5], r[2, 5] = float("inf"), float("-inf"), float("inf"), float("-inf")
    y, h = torch.empty_like(x), torch.empty_like(x)
    q, scale = torch.empty(4, K, device="cuda", dtype=torch.int8), torch.empty(4, device="cuda")
    fg.rms_norm(x, None, y, residual=r, H=h, Q=q, scale=scale)
    assert torch.isnan(scale[:3]).all() and (q[:3] == 0).all() and (q[3] == 127).all()
    assert torch.isnan(y[0, 3]) and (y[0, 4:] == 0).all() and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()
    assert torch.equal(h[[0, 1, 3]], (x + r)[[0, 1, 3]]) and torch.isnan(h[2, 5])


@pytest.mark.parametrize("K", [(1 << 27) + 64, (1 << 28) - 63, (1 << 28) + 77])
def test_gradient_of_the_longest_rows(K):
    # The weight's sums are a launch of their own, sixteen threads a column: from 2^28
    # columns on those are 2^32, more than a dimension takes.
    g = gen(K % 1000)
    h, dy = (torch.randn(1, K, device="cuda", generator=g).bfloat16() for _ in range(2))
    dx, dw = torch.empty_like(h), torch.full((K,), 777.0, device="cuda").bfloat16()
    fg.rms_norm_grad(dy, h, None, dx, dw)
    h, dy = h.double(), dy.double()
    s = (h.square().mean() + 1e-6).rsqrt()
    n = h.mul_(s)
    want = dy * n
    off = 9 * 2.0 ** -24 * want.abs()
    assert ((dw.double() - want).abs() <= 1.01 * off + HALF_STEP[BF16] * (want.abs() + off) + TINY[BF16]).all()
    mean, size = want.mean(), want.abs().mean()
    want = s * (dy - n * mean)
    off = 2.0 ** -24 * (5 * (s * dy).abs() + 8 * s * n.abs() * size)
    assert ((dx.double() - want).abs() <= 1.01 * off + HALF_STEP[BF16] * (want.abs() + off) + TINY[BF16]).all()


@pytest.mark.parametrize("K", [1 << 28, 1 << 30])
def test_weight_gradient_of_no_rows(K):
    e = lambda *s: torch.empty(*s, device="cuda", dtype=BF16)  # noqa: E731
    dw = torch.full((K,), 777.0, device="cuda", dtype=BF16)
    fg.rms_norm_grad(e(0, K), e(0, K), None, e(0, K), dw)
    assert not dw.any()


def gradient_reference(dy, h, w, dh):
    """dX, how far it may be off before its own rounding, dweight and its bound, as in test_norm_gpu."""
    h, dy = h.double(), dy.double()
    s = (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    g = dy if w is None else dy * w.double()
    n = h * s
    dx = s * (g - n * (g * n).mean(1, keepdim=True))
    size = 2.0 ** -24 * (5 * (s * g).abs() + 8 * s * n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + 2.0 ** -24 * dx.abs()
    dw = (dy * n).sum(0)
    return dx, size, dw, (h.shape[0] + 8) * 2.0 ** -24 * (dy * n).abs().sum(0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K", [(5, 1), (5, 70), (5, 1000), (5, 3001), (700, 5000), (5, 12000), (5, 20000)])
def test_gradient_of_products_past_32_bits(dtype, M, K):
    # dY * weight passes the largest float, and the norm's factor brings it back.
    g = gen(K + 1)
    h, dy, dh = (torch.randn(M, K, device="cuda", generator=g) for _ in range(3))
    for row, factor in ((0, 1e37), (2, 2e36), (3, 1e36)):  # the last: the products stay below, their sums do not
        h[row] *= 1e30
        dy[row] *= factor
    h[:, K // 2], dy[:, K // 2] = h[:, K // 2] * 2 + h[:, K // 2].sign(), dy[:, K // 2] * 3
    h, dy, dh = h.to(dtype), dy.to(dtype), dh.to(dtype)
    w = 200 * (1 + 0.3 * torch.randn(K, device="cuda", generator=g))
    for weight, more in ((w, dh), (w.to(dtype), None)):
        dx, dw = torch.empty_like(h), torch.empty(K, device="cuda")
        want, size, want_w, size_w = gradient_reference(dy, h, weight, more)
        assert want.abs().max() < 1e30 and (size_w * 2.0 ** 24 / (M + 8)).max() < torch.finfo(F32).max  # sums of magnitudes
        bound = 1.01 * size + HALF_STEP[dtype] * (want.abs() + size) + TINY[dtype]
        fg.rms_norm_grad(dy, h, weight, dx, dw, residual_grad=more)
        assert ((dx.double() - want).abs() <= bound).all()
        assert ((dw.double() - want_w).abs() <= 1.01 * size_w + HALF_STEP[F32] * (want_w.abs() + size_w) + TINY[F32]).all()
        for place in ("dY", "dH"):
            a = (dy if place == "dY" else dh).clone()
            fg.rms_norm_grad(a if place == "dY" else dy, h, weight, a, residual_grad=None if more is None else a if place == "dH" else more)
            if place == "dY" or more is not None:
                assert torch.equal(a, dx)


@pytest.mark.parametrize("K", [500, 3001, 20000])
def test_gradient_of_means_past_32_bits(K):
    # Every product is finite, and their mean times a large value of the row is not.
    g = gen(K + 5)
    h = torch.randn(3, K, device="cuda", generator=g) * 1e25
    h[1, 7] = 2e26
    dy = h.sign() * 3.2e38
    dx = torch.empty_like(h)
    fg.rms_norm_grad(dy, h, None, dx)
    want, size, _, _ = gradient_reference(dy, h, None, None)
    assert ((dx.double() - want).abs() <= 1.01 * size + HALF_STEP[F32] * (want.abs() + size)).all()


@pytest.mark.parametrize("K", [70, 3000, 20000])
def test_gradient_of_values_that_are_no_numbers(K):
    g = gen(K + 6)
    h, dy, dh = (torch.randn(5, K, device="cuda", generator=g) for _ in range(3))
    clean = torch.empty_like(h)
    fg.rms_norm_grad(dy, h, None, clean, residual_grad=dh)
    dh[0, 3], dy[1, 5], h[3, K - 1] = float("inf"), float("nan"), float("nan")
    dx, dw = torch.empty_like(h), torch.empty(K, device="cuda")
    fg.rms_norm_grad(dy, h, None, dx, dw, residual_grad=dh)
    assert dx[0, 3] == float("inf") and torch.equal(dx[0, 4:], clean[0, 4:])
    assert torch.isnan(dx[1]).all() and torch.isnan(dx[3]).all() and torch.equal(dx[[2, 4]], clean[[2, 4]])
    assert torch.isnan(dw).all()


@pytest.mark.parametrize("dtype,K", [(BF16, 16400), (BF16, 16501), (F16, 17003), (F32, 8300), (F32, 8203)])
@pytest.mark.parametrize("M", [513, 1100])
def test_weight_gradient_of_many_long_rows(dtype, K, M):
    # Rows too long for registers, and more of them than teams: a team adds to its sums in memory.
    from test_norm_gpu import check_gradient
    g = gen(M + K)
    h, dy, dh = (torch.randn(M, K, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = 1 + 0.3 * torch.randn(K, device="cuda", generator=g)
    room = torch.full((fg.layers.rms_norm_grad_workspace(M, K),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    for weight, into, more in ((w.to(dtype), dtype, dh), (w, F32, None)):
        dx, dw = torch.empty_like(h), torch.empty(K, device="cuda", dtype=into)
        fg.rms_norm_grad(dy, h, weight, dx, dw, residual_grad=more, workspace=room)
        check_gradient(dy, h, weight, more, 1e-6, dx, dw)
        a, again = dy.clone(), torch.empty_like(dw)
        fg.rms_norm_grad(a, h, weight, a, again, residual_grad=more, workspace=room)
        assert torch.equal(a, dx) and torch.equal(again, dw)


def block_values(q, s):
    """What codes stand for under their scale bytes, in 64 bits: 255 is no number."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.cat([table, -table])[torch.stack((q & 15, q >> 4), -1).long()].flatten(-2)
    step = torch.where(s == 255, float("nan"), torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), s.double() - 127))
    return v * step.repeat_interleave(32, -1)[..., :v.shape[-1]]


FORMS = [(2, 3), (12, 30)]  # experts, tokens: the direct second product, and the other


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("byte", [0, 1, 2, 30, 250, 252])
@pytest.mark.parametrize("E,T", FORMS)
@pytest.mark.parametrize("D,F", [(256, 128), (200, 77)])
def test_scale_bytes_of_the_first_weights(dtype, byte, E, T, D, F):
    # Every block has its scale near an end of the range, tokens bring the sums back: each
    # product is a normal float, or a subnormal bfloat16 times one.
    g = gen(byte + D)
    power = 127 - byte
    x = (torch.randn(T, D, device="cuda", generator=g) * 2.0 ** max(min(power, 120), -100)).to(dtype)
    w_in = torch.randint(0, 256, (E, F, (D + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    s_in = torch.full((E, F, (D + 31) // 32), byte, dtype=torch.uint8, device="cuda")
    v_in = block_values(w_in, s_in)[..., :D]
    w_out, s_out, v_out = make_weights(g, "mx4", E, D, F, dtype)
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    share = torch.rand(T, 1, device="cuda", generator=g)
    y = torch.empty(T, D, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out, gated=False)
    want, off = layer_reference(x, ids, share, v_in, v_out, False, HELD[dtype], False)
    assert want.abs().amax() > 2.0 ** -10 and torch.isfinite(y).all()
    assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("byte", [0, 1, 2, 30, 250, 252])
@pytest.mark.parametrize("E,T", FORMS)
@pytest.mark.parametrize("D,F", [(64, 256), (40, 205)])
def test_scale_bytes_of_the_second_weights(dtype, byte, E, T, D, F):
    # Shares bring the results back.
    g = gen(byte + F)
    x = torch.randn(T, D, device="cuda", generator=g).to(dtype)
    w_in, s_in, v_in = make_weights(g, "mx4", E, F, D, dtype)
    w_out = torch.randint(0, 256, (E, D, (F + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    s_out = torch.full((E, D, (F + 31) // 32), byte, dtype=torch.uint8, device="cuda")
    if byte >= 250:  # sums of one expert stay finite: a block of each row, the others zero
        w_out[:, :, 16:] = 0
        w_out &= 0x33
    v_out = block_values(w_out, s_out)[..., :F]
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    share = torch.rand(T, 1, device="cuda", generator=g) * 2.0 ** max(min(127 - byte, 110), -120)
    if byte >= 250:
        w_in, s_in = w_in, s_in - 8
        v_in = v_in * 2.0 ** -8
    y = torch.empty(T, D, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out, gated=False)
    want, off = layer_reference(x, ids, share, v_in, v_out, False, HELD[dtype], False)
    # Sums of numbers near the smallest lose their last bits: a subnormal's half step each.
    lost = (4 * F + 4) * 2.0 ** -149 * share.double()
    assert want.abs().amax() > 0 and torch.isfinite(y).all()
    assert ((y.double() - want).abs() <= off + lost + 2.0 ** -24 * (want.abs() + off) + TINY[F32]).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("E,T", FORMS)
@pytest.mark.parametrize("D,F", [(256, 128), (200, 77)])
def test_blocks_that_are_no_numbers(dtype, E, T, D, F):
    # Scale byte 255, codes zero: its row of W_in makes the token's results NaN, its row of
    # W_out one column.  Blocks of zeros, as quantize_mx4 writes them, change nothing.
    g = gen(D + E)
    x = torch.randn(T, D, device="cuda", generator=g).to(dtype)
    w_in, s_in, v_in = make_weights(g, "mx4", E, F, D, dtype)
    w_out, s_out, v_out = make_weights(g, "mx4", E, D, F, dtype)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E)[:, None].contiguous()
    share = torch.rand(T, 1, device="cuda", generator=g) + 0.5
    def spoil(w, s, v, e, row, block, byte):
        w[e, row, 16 * block:16 * block + 16], s[e, row, block] = 0, byte
        v[e, row, 32 * block:32 * block + 32] = 0
    last_d, last_f = (D - 1) // 32, (F - 1) // 32
    for e in range(E):
        spoil(w_in, s_in, v_in, e, 1, 0, 0), spoil(w_in, s_in, v_in, e, F - 1, last_d, 0)
        spoil(w_out, s_out, v_out, e, 2, 0, 0), spoil(w_out, s_out, v_out, e, D - 1, last_f, 0)
    for block in (0, last_f):
        w, s = w_out.clone(), s_out.clone()
        spoil(w, s, v_out.clone(), 0, 5, block, 255)
        y = torch.empty(T, D, device="cuda")
        fg.expert_layer(x, ids, share, w_in, w, y, s_in, s, gated=False)
        want, off = layer_reference(x, ids, share, v_in, v_out, False, HELD[dtype], False)
        hit = torch.zeros(T, D, dtype=torch.bool, device="cuda")
        hit[ids[:, 0] == 0, 5] = True
        assert torch.isnan(y[hit]).all()
        assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32])[~hit].all()
    for block in (0, last_d):
        w, s = w_in.clone(), s_in.clone()
        spoil(w, s, v_in.clone(), 0, 3, block, 255)
        y = torch.empty(T, D, device="cuda")
        fg.expert_layer(x, ids, share, w, w_out, y, s, s_out, gated=False)
        assert torch.isnan(y[ids[:, 0] == 0]).all()
        rest = ids[:, 0] != 0
        assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32])[rest].all()


@pytest.mark.parametrize("kind", ["int8", "mx4"])
@pytest.mark.parametrize("power", [-100, -112, -120, -126])
@pytest.mark.parametrize("E,T", FORMS)
def test_tiny_floats_times_narrow_weights(kind, power, E, T):
    # 32-bit tokens are sums of three bfloat16, which end at 2^-133: what is below is lost,
    # once a value.  Scales and shares bring the results back.
    g = gen(-power)
    D, F = 96, 40
    x = torch.randn(T, D, device="cuda", generator=g) * 2.0 ** power
    w_in, s_in, v_in = make_weights(g, kind, E, F, D, F32)
    up = min(-power, 110)
    s_in = s_in * 2.0 ** up if kind == "int8" else s_in + up
    v_in = v_in * 2.0 ** up
    w_out, s_out, v_out = make_weights(g, kind, E, D, F, F32)
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    share = torch.rand(T, 1, device="cuda", generator=g)
    y = torch.empty(T, D, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out, gated=False)
    want, off = layer_reference(x, ids, share, v_in, v_out, False, HELD[F32], kind == "int8")
    # A sum over D is off by 2^-133 |w| for each value, and by a subnormal's half step for
    # each addition; silu's slope is below 1.1.  So is h, where it falls below 2^-110.
    for t in range(T):
        e = int(ids[t, 0])
        lost = v_in[e].abs().sum(1) * 2.0 ** -133 + (4 * D + 4) * 2.0 ** -149 * 2.0 ** up
        off[t] += share[t, 0].double() * (v_out[e].abs() @ (1.1 * lost + 2.0 ** -133)) + (4 * F + 4) * 2.0 ** -149
    assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("byte,codes", [(253, 0x33), (254, 0x11), (254, 0x77)])
@pytest.mark.parametrize("E,T", FORMS)
def test_largest_scale_bytes(dtype, byte, codes, E, T):
    # Weights are multiplied as bfloat16: past 2^128 they are infinite.
    g = gen(byte + codes)
    D, F = 64, 32
    x = (torch.randn(T, D, device="cuda", generator=g) * 2.0 ** -100).to(dtype)
    w_in = torch.full((E, F, D // 2), codes, dtype=torch.uint8, device="cuda")
    s_in = torch.full((E, F, D // 32), byte, dtype=torch.uint8, device="cuda")
    w_out, s_out, v_out = make_weights(g, "mx4", E, D, F, dtype)
    v_out = v_out * 2.0 ** -30
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=g, dtype=torch.int32)
    share = torch.rand(T, 1, device="cuda", generator=g)
    y = torch.empty(T, D, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out - 30, gated=False)
    if codes == 0x77:
        assert not torch.isfinite(y).any()
        return
    v_in = block_values(w_in, s_in)
    want, off = layer_reference(x, ids, share, v_in, v_out, False, HELD[dtype], False)
    assert ((y.double() - want).abs() <= off + 2.0 ** -24 * (want.abs() + off) + TINY[F32]).all()
