"""The norm, the 8-bit and 4-bit products and the layer of experts together, as a
serving step uses them: captured and replayed, on other streams, side by side, and
what they refuse."""
import os
import sys

import pytest
import torch

import fp32_gemm_amd as fg
from fp32_gemm_amd.binding import _lib
from test_expert_layer_gpu import make_weights, reference
from test_mx4_gpu import unpack

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def empty(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Step:
    """norm with a residual -> 8-bit projection -> norm -> 4-bit projection -> layer of experts."""

    def __init__(self, T, D, F, E, top, seed):
        g = gen(seed)
        self.T, self.D, self.g = T, D, g
        self.x, self.r = empty(T, D, dtype=BF16), empty(T, D, dtype=BF16)
        self.ids, self.share = empty(T, top, dtype=torch.int32), empty(T, top)
        self.weight = 1 + 0.1 * torch.randn(D, device="cuda", generator=g)
        self.w8, self.s8, _ = make_weights(g, "int8", 1, D, D, BF16)
        self.w4, self.s4, _ = make_weights(g, "mx4", 1, D, D, BF16)
        self.w_in, self.s_in, self.v_in = make_weights(g, "mx4", E, 2 * F, D, BF16)
        self.w_out, self.s_out, self.v_out = make_weights(g, "mx4", E, D, F, BF16)
        self.q, self.qs = empty(T, D, dtype=torch.int8), empty(T)
        self.p, self.ps = empty(T, D // 2, dtype=torch.uint8), empty(T, D // 32, dtype=torch.uint8)
        self.a, self.b, self.n = (empty(T, D, dtype=BF16) for _ in range(3))
        self.y = empty(T, D)
        self.room = empty(fg.layers.expert_layer_workspace(self.x, self.ids, F), dtype=torch.uint8)
        self.experts = E
        self.fill()

    def fill(self):
        self.x.normal_(generator=self.g)
        self.start = torch.randn(self.T, self.D, device="cuda", generator=self.g).to(BF16)
        self.ids.random_(-1, self.experts, generator=self.g)
        self.share.uniform_(generator=self.g)

    def run(self, stream=None, workspace=True):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.r.copy_(self.start)
        self.calls(stream, workspace)

    def calls(self, stream=None, workspace=True):
        fg.rms_norm(self.x, self.weight, residual=self.r, H=self.r, Q=self.q, scale=self.qs, stream=stream)
        fg.igemm(self.q, self.qs, self.w8[0], self.s8[0], self.a, stream=stream)
        fg.rms_norm(self.a, self.weight, self.n, residual=self.r, H=self.r, stream=stream)
        fg.quantize_mx4(self.n, self.p, self.ps, stream=stream)
        fg.gemm_mx4(self.p, self.ps, self.w4[0], self.s4[0], self.b, stream=stream)
        fg.expert_layer(self.b, self.ids, self.share, self.w_in, self.w_out, self.y, self.s_in, self.s_out,
                        workspace=self.room if workspace else None, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.q, self.qs, self.r, self.n, self.p, self.ps, self.b, self.y)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


SIZES = [(5, 128, 96, 6, 2), (40, 256, 64, 40, 3)]


@pytest.mark.parametrize("size", SIZES)
def test_step_by_step(size):
    # Each link against its definition on what the link before it gave.
    s = Step(*size, seed=1)
    s.run()
    h = s.x.double() + s.start.double()
    v = h * s.weight.double()
    top = v.abs().amax(1, keepdim=True)
    assert torch.equal(s.q, torch.round(v * 127 / top).to(torch.int8))
    first = s.r.clone()
    a = (s.q.double() @ s.w8[0].double().t()) * s.qs.double()[:, None] * s.s8[0].double()
    assert ((s.a.double() - a).abs() <= a.abs() * (4 * 2.0 ** -24 + 2.0 ** -8) * 1.01 + 1e-30).all()
    h = (s.x.float() + s.start.float()).to(BF16).double() + s.a.double()
    assert torch.equal(s.r, h.float().to(BF16)) and first.shape == s.r.shape
    n = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * s.weight.double()
    assert ((s.n.double() - n).abs() <= n.abs() * (5 * 2.0 ** -24 + 2.0 ** -8) * 1.01 + 1e-30).all()
    p, w = unpack(s.p, s.ps), unpack(s.w4[0], s.s4[0])
    size_b = p.abs() @ w.abs().t()
    b = p @ w.t()
    off = (s.D + 4) * 2.0 ** -23 * size_b
    assert ((s.b.double() - b).abs() <= off + 2.0 ** -8 * (b.abs() + off)).all()
    y, off = reference(s.b, s.ids, s.share, s.v_in, s.v_out, True, BF16, False)
    assert ((s.y.double() - y).abs() <= off + 2.0 ** -23 * y.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("size", SIZES)
def test_captured_and_replayed(size):
    s = Step(*size, seed=2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run(workspace=False)
        s.run()
    for turn in range(4):
        s.start.normal_(generator=s.g)  # the captured copy reads the same buffer
        s.x.normal_(generator=s.g), s.ids.random_(-1, s.experts, generator=s.g)
        s.room.fill_(0xFF)  # whatever an earlier call left there
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.y.fill_(float("nan"))
        s.run()
        torch.cuda.synchronize()
        assert same(got, s.outputs()), turn


def test_two_captured_graphs_share_a_workspace():
    # One after the other on a stream: nothing is kept in it from call to call.
    a, b = Step(*SIZES[0], seed=3), Step(*SIZES[0], seed=4)
    b.room = a.room
    want = []
    for s in (a, b):
        s.run()
        want.append(s.outputs())
    graphs = []
    for s in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run()
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for i in order:
            (a, b)[i].y.fill_(float("nan"))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert same(want[i], (a, b)[i].outputs())


def test_streams_side_by_side():
    steps = [Step(*SIZES[i % 2], seed=5 + i) for i in range(4)]
    want = []
    for s in steps:
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for workspace in (True, False):
        for s in steps:
            s.y.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for s, stream in zip(steps, streams):
                s.run(stream=stream, workspace=workspace)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert same(w, s.outputs())
    handle = streams[0].cuda_stream  # a stream by its handle, its workspace from torch
    steps[0].y.fill_(float("nan"))
    torch.cuda.synchronize()
    s = steps[0]
    fg.expert_layer(s.b, s.ids, s.share, s.w_in, s.w_out, s.y, s.s_in, s.s_out, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(s.y, want[0][-1])
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_runs_agree():
    # Sums are made in a fixed order, whichever workgroup comes last.
    s = Step(64, 256, 128, 12, 4, seed=9)
    s.run()
    want = s.outputs()
    for _ in range(20):
        s.run()
        assert same(want, s.outputs())


def test_an_earlier_error_is_left_to_the_program():
    s = Step(*SIZES[0], seed=10)
    s.run()
    want = s.outputs()
    dw, dx = empty(s.D), empty(s.T, s.D, dtype=BF16)
    room = empty(fg.layers.rms_norm_grad_workspace(s.T, s.D), dtype=torch.uint8)
    s.r.copy_(s.start)
    torch.cuda.synchronize()
    assert _lib.hipSetDevice(9999) != 0
    left = _lib.hipPeekAtLastError()
    try:
        s.calls()
        fg.rms_norm_grad(s.n, s.a, s.weight, dx, dw, workspace=room)
        assert _lib.hipPeekAtLastError() == left
    finally:
        _lib.hipGetLastError()
    assert left != 0 and same(want, s.outputs()) and torch.isfinite(dw).all()


def test_long_rows_and_many():
    # Offsets past 32 bits: rows far apart, and rows enough for a second grid dimension's worth.
    K, ld = 40, 1 << 24
    base = torch.zeros(200 * ld, dtype=F16, device="cuda")
    x = base.view(200, ld)[:, :K]
    x.copy_(torch.randn(200, K, device="cuda", generator=gen(1)))
    y, q, scale = empty(200, K), empty(200, K // 2, dtype=torch.uint8), empty(200, 2, dtype=torch.uint8)
    fg.rms_norm(x, None, y)
    z = empty(200, K)
    fg.rms_norm(x.contiguous(), None, z)
    assert torch.equal(y, z)
    fg.quantize_mx4(x, q, scale)
    p, t = torch.empty_like(q), torch.empty_like(scale)
    fg.quantize_mx4(x.contiguous(), p, t)
    assert torch.equal(q, p) and torch.equal(scale, t)
    dx, dy = empty(200, K, dtype=F16), empty(200, K, dtype=F16)
    fg.rms_norm_grad(y.half(), x, None, dx)
    fg.rms_norm_grad(y.half(), x.contiguous(), None, dy)
    assert torch.equal(dx, dy)
    del base, x
    M = (1 << 25) + 5  # four rows a workgroup: more than 2^23 of them
    x = torch.randn(64, 8, device="cuda", generator=gen(2)).half()
    many = x.repeat(M // 64 + 1, 1)[:M]
    q, scale = empty(M, 8, dtype=torch.int8), empty(M)
    fg.rms_norm(many, None, Q=q, scale=scale)
    p, t = empty(64, 8, dtype=torch.int8), empty(64)
    fg.rms_norm(x, None, Q=p, scale=t)
    for i in (0, 1 << 23, 1 << 24, (1 << 25) - 64):
        assert torch.equal(q[i:i + 64], p) and torch.equal(scale[i:i + 64], t)
    assert torch.equal(q[-5:], p[(M - 5) % 64:][:5] if (M - 5) % 64 <= 59 else q[-5:])
    p4, t4 = empty(M, 4, dtype=torch.uint8), empty(M, 1, dtype=torch.uint8)
    fg.quantize_mx4(many, p4, t4)
    q4, s4 = empty(64, 4, dtype=torch.uint8), empty(64, 1, dtype=torch.uint8)
    fg.quantize_mx4(x, q4, s4)
    for i in (0, 1 << 24, (1 << 25) - 64):
        assert torch.equal(p4[i:i + 64], q4) and torch.equal(t4[i:i + 64], s4)


def test_refusals():
    s = Step(*SIZES[0], seed=11)
    s.run()
    x, y, w = s.x, s.y, s.weight
    out = empty(s.T, s.D, dtype=BF16)
    bad = [
        (ValueError, lambda: fg.rms_norm(x, w)),
        (ValueError, lambda: fg.rms_norm(x, w, out[:, :-1])),
        (ValueError, lambda: fg.rms_norm(x, w[:-1], out)),
        (ValueError, lambda: fg.rms_norm(x, w, out, Q=s.q)),
        (TypeError, lambda: fg.rms_norm(x, w.half(), out)),
        (TypeError, lambda: fg.rms_norm(x, w, out, residual=y)),
        (TypeError, lambda: fg.rms_norm(x, w, out.half())),
        (ValueError, lambda: fg.rms_norm(x.t(), None, out.t())),
        (ValueError, lambda: fg.rms_norm(x, w.cpu(), out)),
        (fg.LayerError, lambda: fg.rms_norm(x, w, x)),
        (fg.LayerError, lambda: fg.rms_norm(x, w, out, eps=-1.0)),
        (fg.LayerError, lambda: fg.rms_norm(x, w, out, H=out)),
        (TypeError, lambda: fg.rms_norm_grad(x, x, w, out, dweight=empty(s.D, dtype=F16))),
        (fg.LayerError, lambda: fg.rms_norm_grad(x, s.r, w, s.r)),
        (fg.LayerError, lambda: fg.rms_norm_grad(x, s.r, w, out, empty(s.D), workspace=empty(8, dtype=torch.uint8))),
        (TypeError, lambda: fg.rms_norm_grad(x, s.r, w, out, empty(s.D), workspace=empty(1 << 20))),
        (ValueError, lambda: fg.quantize_mx4(x, s.p[:, :-1], s.ps)),
        (ValueError, lambda: fg.quantize_mx4(x, s.p, s.ps[:, :-1])),
        (TypeError, lambda: fg.quantize_mx4(x, s.q, s.ps)),
        (ValueError, lambda: fg.gemm_mx4(s.p, s.ps, s.w4[0], s.s4[0, :-1], s.b)),
        (ValueError, lambda: fg.gemm_mx4(s.p, s.ps, s.w4, s.s4, s.b)),
        (TypeError, lambda: fg.gemm_mx4(s.p, s.ps.int(), s.w4[0], s.s4[0], s.b)),
    ]

    def layer(**change):
        a = dict(X=s.b, ids=s.ids, share=s.share, W_in=s.w_in, W_out=s.w_out, Y=y, scale_in=s.s_in, scale_out=s.s_out)
        a.update(change)
        return lambda: fg.expert_layer(**a)

    many = empty(65, s.D, dtype=BF16)
    bad += [
        (TypeError, layer(ids=s.ids.long())), (TypeError, layer(share=s.share.double())), (ValueError, layer(share=s.share[:, :1])),
        (ValueError, layer(ids=s.ids[:, :0], share=s.share[:, :0])), (ValueError, layer(W_in=s.w_in[:, :-1])),
        (ValueError, layer(gated=False)), (TypeError, layer(scale_in=None)), (TypeError, layer(W_in=s.w_in.to(torch.int8))),
        (ValueError, layer(scale_in=s.s_in[:, :-2])), (TypeError, layer(Y=out.half())), (ValueError, layer(Y=y[:-1])),
        (fg.LayerError, layer(workspace=empty(64, dtype=torch.uint8))),
        (ValueError, layer(workspace=empty(1 << 20, 2, dtype=torch.uint8)[:, 0])),
        (fg.LayerError, layer(X=many, ids=s.ids[:1].repeat(65, 1), share=s.share[:1].repeat(65, 1), Y=empty(65, s.D))),
        (TypeError, layer(W_in=s.w_in.float(), W_out=s.w_out.float())),
    ]
    before = s.outputs()
    for error, call in bad:
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()
    assert same(before, s.outputs())


def test_the_norm_as_a_torch_function():
    g = gen(12)
    x = torch.randn(9, 40, device="cuda", generator=g).requires_grad_()
    w = (1 + 0.1 * torch.randn(40, device="cuda", generator=g)).requires_grad_()
    dy = torch.randn(9, 40, device="cuda", generator=g)
    expert_layer.Norm.apply(x, w).backward(dy)
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    (xd * (xd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wd).backward(dy.double())
    # A dozen roundings of terms of size up to about 8, and 9 rows of sums.
    assert (x.grad - xd.grad).abs().max() <= 16 * 8 * 2.0 ** -24
    assert (w.grad - wd.grad).abs().max() <= (9 + 8) * 9 * 8 * 2.0 ** -24


def test_serving_in_4_bits():
    _, _, errors = expert_layer.main(width=256, hidden=512, tokens=256, steps=2, bits=4)
    assert all(e == e for e in errors)


def test_the_default_stream_by_its_handle():
    s = Step(*SIZES[0], seed=12)
    s.run()
    want = s.outputs()
    s.y.fill_(float("nan"))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()) as _:
        now = torch.cuda.current_stream()
        fg.expert_layer(s.b, s.ids, s.share, s.w_in, s.w_out, s.y, s.s_in, s.s_out, stream=0)
        assert torch.cuda.current_stream() == now
    torch.cuda.synchronize()
    assert torch.equal(s.y, want[-1])
