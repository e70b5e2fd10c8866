"""The whole layer of experts for a few tokens on the GPU against 64 bits.

Bounds count roundings: a sum of n exact products in 32 bits is off by at most
(n + 4) * 2^-23 of the sum of magnitudes (as for the grouped products), scales,
silu's quotient and products round a few times 2^-24, h rounds by half a step of its
type, and y by half a step of its own.
"""
import pytest
import torch

import fp32_gemm_amd as fg
from fp32_gemm_amd.binding import _lib
from test_mx4_gpu import unpack

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F32, BF16, F16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in (F32, BF16, F16)}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_weights(g, kind, E, rows, depth, dtype):
    """Weights in the form that is multiplied, their scales, and their values in 64 bits."""
    if kind == "same":
        w = (torch.randn(E, rows, depth, device="cuda", generator=g) * depth ** -0.5).to(dtype)
        return w, None, w.double()
    if kind == "int8":
        q = torch.randint(-127, 128, (E, rows, depth), device="cuda", generator=g).to(torch.int8)
        s = (0.5 + torch.rand(E, rows, device="cuda", generator=g)) * depth ** -0.5 / 70
        return q, s, q.double() * s.double()[..., None]
    q = torch.randint(0, 256, (E, rows, (depth + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(119, 125, (E, rows, (depth + 31) // 32), dtype=torch.uint8, device="cuda", generator=g)
    return q, s, unpack(q, s)[..., :depth]


def reference(x, ids, share, w_in, w_out, gated, held, scaled, terms=None):
    """y in 64 bits, and how far a result may be off before its own rounding; `held`:
    the type of h, `scaled`: whether sums are scaled afterwards, `terms`: how many
    products of either sum are not zero (adding zero rounds nothing), if not all."""
    x, share = x.double(), share.double()
    y, off = torch.zeros_like(x), torch.zeros_like(x)
    step = 2.0 ** -24
    F = w_out.shape[2]
    deep, wide = terms or (w_in.shape[2], F)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w_in.shape[0]:
                continue
            u = w_in[e] @ x[t]
            du = (2 * (deep + 4) + 2 * scaled) * step * (w_in[e].abs() @ x[t].abs())
            a, da = (u[:F], du[:F]) if gated else (u, du)
            h = a * torch.sigmoid(a)
            dh = 1.1 * da + 8 * step * h.abs()  # silu's slope stays below 1.1; exponential, sum and quotient
            if gated:
                dh = dh * (u[F:].abs() + du[F:]) + h.abs() * du[F:]
                h = h * u[F:]
                dh = dh + step * h.abs()
            dh = dh + HALF_STEP[held] * (h.abs() + dh) + TINY[held]
            y[t] += share[t, j] * (w_out[e] @ h)
            # The sum over F, its scale and share, and the sum over waves and experts.
            off[t] += share[t, j].abs() * (w_out[e].abs() @ dh + (2 * (wide + 4) + 2 * scaled + 24) * step * (w_out[e].abs() @ (h.abs() + dh)))
    return y, off


def run(case, seed=0, ids=None, out=None, strides=None, terms=None):
    dtype, kind, gated, E, T, top, D, F = case
    g = gen(seed)
    x = torch.randn(T, D, device="cuda", generator=g).to(dtype)
    w_in, s_in, v_in = make_weights(g, kind, E, 2 * F if gated else F, D, dtype)
    w_out, s_out, v_out = make_weights(g, kind, E, D, F, dtype)
    if ids is None:
        ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:top] for _ in range(T)]).to(torch.int32)
    share = torch.rand(T, top, device="cuda", generator=g)
    y = torch.full((T, D), 777.0, device="cuda").to(out or dtype)
    if strides:
        x, w_in, w_out, y = strides(x, w_in, w_out, y)
    assert fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out, gated=gated) is y
    want, off = reference(x, ids, share, v_in, v_out, gated, dtype, kind == "int8", terms)
    bound = off + HALF_STEP[y.dtype] * (want.abs() + off) + TINY[y.dtype]
    assert ((y.double() - want).abs() <= bound).all()
    return y


SHAPES = [  # experts, tokens, choices, D, F
    (1, 1, 1, 1, 1), (2, 1, 1, 7, 5), (4, 1, 2, 64, 64), (8, 1, 2, 512, 256), (6, 5, 2, 129, 77), (3, 16, 3, 100, 33),
    (8, 17, 2, 256, 128), (5, 33, 2, 96, 160), (2, 64, 2, 130, 70), (16, 64, 8, 65, 31), (300, 20, 4, 48, 40),
    (4, 2, 2, 2100, 1100), (3, 40, 1, 1030, 516), (1, 64, 1, 520, 264),
    (2, 3, 2, 4500, 300), (2, 20, 2, 300, 4500),        # reductions whose values do not stay in registers
    (16, 16, 4, 2048, 256), (32, 16, 4, 500, 1030), (32, 12, 4, 2100, 130),  # several sets of rows a workgroup
    (40, 10, 8, 64, 96), (90, 60, 2, 40, 64), (1024, 30, 3, 33, 20),         # many experts
]


@pytest.mark.parametrize("dtype,kind", [(F32, "same"), (BF16, "same"), (F16, "same"), (F32, "int8"), (BF16, "int8"), (F16, "int8"),
                                        (F32, "mx4"), (BF16, "mx4"), (F16, "mx4")])
@pytest.mark.parametrize("E,T,top,D,F", SHAPES)
def test_layer(dtype, kind, E, T, top, D, F):
    for gated in (True, False):
        run((dtype, kind, gated, E, T, top, D, F), seed=E + T + D)


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
def test_output_in_32_bits(kind):
    run((BF16, kind, True, 4, 9, 2, 200, 100), out=F32)


@pytest.mark.parametrize("kind", ["same", "mx4"])
def test_ids(kind):
    i32 = lambda rows: torch.tensor(rows, dtype=torch.int32, device="cuda")  # noqa: E731
    case = (BF16, kind, True, 5, 6, 3, 96, 64)
    # No expert, ids that are no expert's, the same one twice and three times.
    y = run(case, ids=i32([[-1, -1, -1], [0, 5, -7], [2, 2, 1], [3, 3, 3], [4, -1, 4], [1 << 30, 0, -(1 << 31)]]))
    assert (y[0] == 0).all()
    y = run(case, ids=i32([[-1] * 3] * 6))
    assert (y == 0).all()
    run(case, ids=i32([[1, 1, 1]] * 6))
    run((BF16, kind, False, 5, 64, 8, 96, 64), ids=i32([[1, 2, 1, 2, 0, 0, 2, 1]] * 64))
    run((F16, kind, False, 5, 50, 2, 96, 64), ids=i32([[4, 4]] * 50))


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
@pytest.mark.parametrize("pad,skip", [(1, 1), (3, 2), (16, 16)])
def test_windows(kind, pad, skip):
    held = {}

    def strided(t, fill):
        n = 1
        for v in t.shape[:-1]:
            n *= v
        ld = t.shape[-1] + pad
        base = torch.full((n * ld + skip + 16,), fill, device="cuda").to(t.dtype)
        view = base[skip:skip + n * ld].view(*t.shape[:-1], ld)[..., :t.shape[-1]]
        view.copy_(t)
        return base, view

    def strides(x, w_in, w_out, y):
        fill = float("nan") if kind == "same" else 0x7F
        x, w_in, w_out = (strided(t, f)[1] for t, f in ((x, float("nan")), (w_in, fill), (w_out, fill)))
        held["base"], y = strided(y, 555.0)
        held["before"] = held["base"].clone()
        return x, w_in, w_out, y

    for dtype in (BF16, F32):
        y = run((dtype, kind, True, 4, 7, 2, 150, 90), strides=strides)
        y.fill_(777.0)
        assert torch.equal(held["base"], held["before"]), "a byte outside Y changed"


def test_other_experts_are_not_looked_at():
    # Weights of experts that no token names may hold anything.
    g = gen(2)
    w_in, _, v_in = make_weights(g, "same", 4, 64, 80, BF16)
    w_out, _, v_out = make_weights(g, "same", 4, 80, 32, BF16)
    w_in[[0, 2]], w_out[[0, 2]] = float("nan"), float("inf")
    x = torch.randn(3, 80, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([[1, 3], [3, -1], [1, 1]], dtype=torch.int32, device="cuda")
    share = torch.rand(3, 2, device="cuda", generator=g)
    share[1, 1] = float("nan")  # of no expert
    y = torch.empty_like(x)
    fg.expert_layer(x, ids, share, w_in, w_out, y)
    want, off = reference(x, ids, share, v_in, v_out, True, BF16, False)
    assert ((y.double() - want).abs() <= off + HALF_STEP[BF16] * (want.abs() + off) + TINY[BF16]).all()


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_bad_values_stay_with_their_token(dtype, kind):
    g = gen(6)
    x = torch.randn(4, 70, device="cuda", generator=g).to(dtype)
    clean = x.clone()
    x[1, 3], x[2, 69] = float("nan"), float("inf")
    w_in, s_in, _ = make_weights(g, kind, 2, 40, 70, dtype)
    w_out, s_out, _ = make_weights(g, kind, 2, 70, 20, dtype)
    ids = torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda")
    share = torch.rand(4, 2, device="cuda", generator=g)
    y, z = torch.empty_like(x), torch.empty_like(x)
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out)
    fg.expert_layer(clean, ids, share, w_in, w_out, z, s_in, s_out)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    assert torch.equal(y[[0, 3]], z[[0, 3]])


def test_infinite_values_times_narrow_weights():
    # One infinity, weights of one sign: the sums are infinite, not NaN.
    for dtype in (F32, BF16, F16):
        x = torch.ones(1, 64, device="cuda", dtype=dtype)
        x[0, 5] = float("inf")
        w_in, s_in = torch.ones(1, 16, 64, dtype=torch.int8, device="cuda"), torch.ones(1, 16, device="cuda")
        w_out, s_out = torch.ones(1, 64, 16, dtype=torch.int8, device="cuda"), torch.ones(1, 64, device="cuda")
        y = torch.empty_like(x)
        fg.expert_layer(x, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"), w_in, w_out, y,
                        s_in, s_out, gated=False)
        assert (y == float("inf")).all()


def test_nothing_to_multiply():
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    ids, share = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), e(3, 2)
    y = torch.full((3, 8), 777.0, device="cuda")
    fg.expert_layer(e(3, 8), ids, share, e(2, 0, 8), e(2, 8, 0), y)
    assert (y == 0).all()
    fg.expert_layer(e(0, 8), ids[:0], share[:0], e(2, 4, 8), e(2, 8, 2), e(0, 8))


@pytest.mark.parametrize("dtype,kind", [(F32, "same"), (BF16, "same"), (F16, "same"), (F32, "int8"), (BF16, "int8"), (F16, "int8"),
                                        (F32, "mx4"), (BF16, "mx4"), (F16, "mx4")])
@pytest.mark.parametrize("E,T,top,D,F", [(3, 1, 2, 517, 291), (5, 7, 2, 1030, 700), (4, 30, 3, 333, 1100), (2, 4, 1, 4610, 64),
                                         (2, 21, 2, 64, 4610), (32, 16, 4, 300, 1030)])
def test_every_place_counts_once(dtype, kind, E, T, top, D, F):
    # A handful of values and columns that are not zero, anywhere, the first and last
    # among them: sums of few terms leave little room for a piece lost or taken twice.
    g = gen(D + F)
    few = 6
    w_in, s_in, v_in = make_weights(g, kind, E, 2 * F, D, dtype)
    w_out, s_out, v_out = make_weights(g, kind, E, D, F, dtype)
    x = torch.zeros(T, D, device="cuda", dtype=dtype)
    for t in range(T):
        at = torch.cat([torch.tensor([0, D - 1], device="cuda"), torch.randint(0, D, (few - 2,), device="cuda", generator=g)])
        x[t, at] = torch.randn(few, device="cuda", generator=g).to(dtype)
    keep = torch.zeros(F, dtype=torch.bool, device="cuda")
    keep[torch.cat([torch.tensor([0, F - 1], device="cuda"), torch.randint(0, F, (few - 2,), device="cuda", generator=g)])] = True
    v_out = torch.where(keep, v_out, 0.0)
    if kind == "mx4":
        pairs = torch.nn.functional.pad(keep, (0, F % 2)).view(-1, 2)
        w_out &= (pairs[:, 0] * 15 + pairs[:, 1] * 240).to(torch.uint8)
    else:
        w_out[..., ~keep] = 0
    ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:top] for _ in range(T)]).to(torch.int32)
    share = torch.rand(T, top, device="cuda", generator=g)
    y = torch.empty(T, D, device="cuda")  # 32 bits: nothing is lost at the end
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out)
    want, off = reference(x, ids, share, v_in, v_out, True, dtype, kind == "int8", terms=(few, few))
    assert ((y.double() - want).abs() <= off * (1 + 2.0 ** -20) + 2.0 ** -24 * want.abs() + TINY[F32]).all()


@pytest.mark.parametrize("kind", ["same", "int8", "mx4"])
@pytest.mark.parametrize("T,top", [(1, 40), (1, 128), (4, 20), (16, 8), (3, 170)])
def test_the_same_expert_many_times(kind, T, top):
    # More pairs than tokens: an expert's second sets of 16 pairs hold no token.  The sum
    # over the choices rounds `top` times more.
    g = gen(top)
    for used in (1, 2):
        ids = torch.randint(0, used, (T, top), device="cuda", generator=g, dtype=torch.int32)
        run((BF16, kind, True, 4, T, top, 96, 64), ids=ids, out=F32, terms=(96, 64 + top))


def test_more_columns_than_a_workgroup_lists():
    # 256 experts of 2048 blocks of columns each: a late workgroup is the last at
    # hundreds of them.
    E, D = 256, 1 << 18
    g = gen(12)
    x = torch.randn(1, D, device="cuda", generator=g).bfloat16()
    w_in = (torch.randn(E, 1, D, device="cuda", generator=g) * 2.0 ** -9).bfloat16()
    w_out = torch.randn(E, D, 1, device="cuda", generator=g).bfloat16()
    ids = torch.randperm(E, device="cuda", generator=g).to(torch.int32)[None]
    share = torch.rand(1, E, device="cuda", generator=g)
    want, off = reference(x, ids, share, w_in.double(), w_out.double(), False, BF16, False, (D, 1 + E))
    y = torch.full((1, D), 777.0, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, gated=False)
    assert ((y.double() - want).abs() <= off + HALF_STEP[F32] * (want.abs() + off) + TINY[F32]).all()


@pytest.mark.parametrize("T,top", [(3, 2), (20, 2), (64, 8)])
@pytest.mark.parametrize("weights", [1, 3, 5])
def test_no_hidden_width_and_no_operands(T, top, weights):
    y = torch.full((T, 40), 777.0, device="cuda")
    room = torch.empty(_lib.expert_layer_workspace(1, T, 40, 0, top), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert _lib.expert_layer(1, weights, 0, 1, T, 40, 0, 4, top, None, 40, None, None, None, 40, 0, None, None, 1, 0, None,
                             y.data_ptr(), 40, room.data_ptr(), room.numel(), None) == 0
    torch.cuda.synchronize()
    assert (y == 0).all()


@pytest.mark.parametrize("dtype,kind", [(F32, "same"), (BF16, "mx4"), (BF16, "int8")])
@pytest.mark.parametrize("D,F", [(1 << 19, 3), (5, 1 << 19)])
def test_the_widest_layers(dtype, kind, D, F):
    # 64 tokens of 8 choices: a token's values and products lie furthest apart.  Values
    # and weights that are zero but at a few places keep the sums short.
    g, T, top, E = gen(D % 1000), 64, 8, 2
    w_in, s_in, v_in = make_weights(g, kind, E, 2 * F, D, dtype)
    w_out, s_out, v_out = make_weights(g, kind, E, D, F, dtype)
    x = torch.zeros(T, D, device="cuda", dtype=dtype)
    n = min(D, 4)
    places = torch.cat([torch.tensor([0, D - 1], device="cuda"), torch.randint(0, D, (n - 2,), device="cuda", generator=g)])
    x[:, places] = torch.randn(T, n, device="cuda", generator=g).to(dtype)
    keep = torch.zeros(F, dtype=torch.bool, device="cuda")
    keep[torch.tensor([0, F // 2, F - 1], device="cuda")] = True
    v_out = torch.where(keep, v_out, 0.0)
    if kind == "mx4":
        pairs = torch.nn.functional.pad(keep, (0, F % 2)).view(-1, 2)
        w_out &= (pairs[:, 0] * 15 + pairs[:, 1] * 240).to(torch.uint8)
    else:
        w_out[..., ~keep] = 0
    ids = torch.full((T, top), -1, dtype=torch.int32, device="cuda")
    ids[::7, -1], ids[-1, 0], ids[-1, 3] = 1, 0, 1
    share = torch.rand(T, top, device="cuda", generator=g)
    y = torch.full((T, D), 777.0, device="cuda")
    fg.expert_layer(x, ids, share, w_in, w_out, y, s_in, s_out)
    want, off = reference(x, ids, share, v_in, v_out, True, dtype, kind == "int8", (n, 3 + top))
    assert ((y.double() - want).abs() <= off * (1 + 2.0 ** -20) + 2.0 ** -24 * want.abs() + TINY[F32]).all()
