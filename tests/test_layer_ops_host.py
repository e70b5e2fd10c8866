"""C ABI, argument checks and refusals of the norm, the 4-bit product and the layer
of experts for few tokens, without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp32_gemm_amd as fg
from fp32_gemm_amd import grouped, layers
from fp32_gemm_amd.binding import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "layer_ops.h")
FAKE = 1 << 40  # a well-aligned, never-dereferenced address


def test_header_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))
    assert declared == layers.exported_symbols()
    lib = ctypes.CDLL(fg.library_path())
    for name in declared:
        assert hasattr(lib, name), name


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "layer_ops.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-c", str(src),
                    "-o", str(tmp_path / "h.o")], check=True)


def quantize_call(type=1, M=8, K=40, X=FAKE, ldx=40, Q=FAKE * 2, ldq=20, scale=FAKE * 4):
    return _lib.quantize_mx4(type, M, K, X, ldx, Q, ldq, scale, None)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(M=-1), -2), (dict(K=-1), -3), (dict(X=None), -4), (dict(ldx=39), -5), (dict(Q=None), -6),
    (dict(ldq=19), -7), (dict(K=39, ldq=19), -7), (dict(scale=None), -8), (dict(M=(1 << 30) + 1), 5), (dict(Q=FAKE + 8), 3),
    (dict(scale=FAKE + 8 * 80 - 1), 3), (dict(scale=FAKE * 2 + 16), 3), (dict(scale=FAKE * 2 - 15), 3),
])
def test_quantize_mx4_codes(change, code):
    assert quantize_call(**change) == code


def mx4_call(out=1, groups=4, off=FAKE * 8, M=64, N=32, K=64, A=FAKE, lda=32, sa=FAKE * 16, B=FAKE * 2, ldb=32,
             stride=1024, sb=FAKE * 32, bias=None, C=FAKE * 4, ldc=32):
    return _lib.gemm_mx4(out, groups, off, M, N, K, A, lda, sa, B, ldb, stride, sb, bias, C, ldc, None)


@pytest.mark.parametrize("change,code", [
    (dict(out=3), -1), (dict(groups=0), -2), (dict(off=None), -2), (dict(M=-1), -4), (dict(N=-1), -5), (dict(K=-1), -6),
    (dict(A=None), -7), (dict(lda=31), -8), (dict(K=65), -8), (dict(sa=None), -9), (dict(B=None), -10), (dict(ldb=31), -11),
    (dict(stride=-1), -12), (dict(sb=None), -13), (dict(C=None), -15), (dict(ldc=31), -16), (dict(lda=1 << 21), 5),
    (dict(groups=(1 << 16) + 1), 5), (dict(K=(1 << 30) + 2, lda=1 << 30, ldb=1 << 30), 5), (dict(C=FAKE * 16 + 127), 3),
    (dict(C=FAKE * 32 + 4 * 64 - 1), 3), (dict(bias=FAKE * 4), 3), (dict(C=FAKE + 8), 3), (dict(C=FAKE * 2 + 3 * 1024 + 1023), 3),
])
def test_gemm_mx4_codes(change, code):
    assert mx4_call(**change) == code


def test_quick_returns():
    assert mx4_call(M=0, A=None, C=None, sa=None) == 0 and mx4_call(N=0, B=None, C=None, sb=None) == 0
    assert quantize_call(M=0, X=None, Q=None, scale=None) == 0 and quantize_call(K=0, Q=None, scale=None) == 0
    assert norm_call(M=0, X=None, Y=None, scale=None) == 0 and norm_call(K=0, X=None, Y=None) == 0
    assert grad_call(K=0, dY=None, H=None, dX=None, dw=None) == 0 and grad_call(M=0, dY=None, H=None, dX=None, dw=None) == 0
    assert layer_call(T=0, X=None, Y=None, room=0) == 0 and layer_call(D=0, W_in=None, Y=None, F=4) == 0


def test_the_gpu_tests_reach_every_tile():
    import test_mx4_gpu as on_gpu
    for out in (torch.float32, torch.bfloat16):
        seen = {grouped.plan("nt", torch.uint8, len(s), sum(s) + 3, N, K2, out=out)["tile"] for s, N, K2 in on_gpu.PRODUCTS}
        assert seen == set(grouped.tiles("nt", torch.uint8)) == set(grouped.TILES)
    with pytest.raises(ValueError):
        grouped.tiles("nn", torch.uint8)


@pytest.mark.parametrize("groups,M,N,K", [(1, 1 << 28, 16, 16), (1, 1 << 30, 16, 16), (65536, 65536, 16384, 64),
                                          (4096, 1 << 20, 4096, 2048)])
def test_launches_hold_every_plan(groups, M, N, K):
    p = grouped.plan("nt", torch.uint8, groups, M, N, K)  # HIP takes fewer than 2^32 threads a launch
    assert 0 < p["grid"] * (512 if p["BM"] >= 128 else 256) < 1 << 32


def norm_call(type=1, wt=1, out=1, M=8, K=16, eps=1e-6, X=FAKE, ldx=16, R=None, ldr=16, w=FAKE * 2, H=None, ldh=16, Y=FAKE * 4,
              ldy=16, Q=None, ldq=16, scale=None):
    return _lib.rms_norm(type, wt, out, M, K, eps, X, ldx, R, ldr, w, H, ldh, Y, ldy, Q, ldq, scale, None)


CODES = dict(Q=FAKE * 8, scale=FAKE * 16)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(wt=2), -2), (dict(type=0, wt=1), -2), (dict(out=2), -3), (dict(type=0, wt=0, out=1), -3), (dict(M=-1), -4),
    (dict(K=-1), -5), (dict(eps=-1e-6), -6), (dict(eps=float("nan")), -6), (dict(X=None), -7), (dict(ldx=15), -8),
    (dict(R=FAKE * 32, ldr=15), -10), (dict(H=FAKE * 32, ldh=15), -13), (dict(Y=None), -15), (dict(ldy=15), -15),
    (dict(Q=FAKE * 8, scale=FAKE * 16, ldq=15), -17), (dict(Q=FAKE * 8), -18), (dict(scale=FAKE * 16), -16),
    (dict(M=(1 << 30) + 1), 5), (dict(ldx=(1 << 30) + 1), 5),
    (dict(Y=FAKE), 3), (dict(Y=FAKE * 2 + 16), 3), (dict(H=FAKE + 32), 3), (dict(H=FAKE, ldh=17), 3), (dict(R=FAKE * 32, H=FAKE * 32 + 2), 3),
    (dict(H=FAKE * 4), 3), (dict(R=FAKE * 4), 3), (dict(H=FAKE * 2), 3), (dict(CODES, Q=FAKE * 4), 3), (dict(CODES, scale=FAKE * 8), 3),
    (dict(CODES, scale=FAKE + 8), 3), (dict(CODES, scale=FAKE * 4 + 8), 3), (dict(CODES, Q=FAKE * 2), 3),
])
def test_rms_norm_codes(change, code):
    assert norm_call(**change) == code


def grad_call(type=1, wt=1, dwt=0, M=8, K=16, eps=1e-6, dY=FAKE, lddy=16, H=FAKE * 2, ldh=16, w=FAKE * 4, dH=None, lddh=16,
              dX=FAKE * 8, lddx=16, dw=FAKE * 16, room=FAKE * 32, size=None):
    size = _lib.rms_norm_grad_workspace(M, K) if size is None else size
    return _lib.rms_norm_grad(type, wt, dwt, M, K, eps, dY, lddy, H, ldh, w, dH, lddh, dX, lddx, dw, room, size, None)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(wt=2), -2), (dict(dwt=2), -3), (dict(M=-1), -4), (dict(K=-1), -5), (dict(eps=float("nan")), -6),
    (dict(dY=None), -7), (dict(lddy=15), -8), (dict(H=None), -9), (dict(ldh=15), -10), (dict(dH=FAKE * 64, lddh=15), -13),
    (dict(dX=None), -14), (dict(lddx=15), -15), (dict(room=None), -17), (dict(room=FAKE * 32 + 2), -17), (dict(size=0), -18),
    (dict(size=8 * 16 * 4 - 1), -18), (dict(K=(1 << 30) + 1, lddy=1 << 31, ldh=1 << 31, lddx=1 << 31, size=1 << 62), 5),
    (dict(dX=FAKE * 2), 3), (dict(dX=FAKE + 2), 3), (dict(dX=FAKE, lddx=17), 3), (dict(dX=FAKE * 4), 3), (dict(dw=FAKE), 3),
    (dict(dw=FAKE * 8), 3), (dict(room=FAKE * 16), 3), (dict(room=FAKE * 8 + 4), 3), (dict(dH=FAKE * 64, dX=FAKE * 64 + 4), 3),
])
def test_rms_norm_grad_codes(change, code):
    assert grad_call(**change) == code


def test_gradient_workspace():
    assert _lib.rms_norm_grad_workspace(0, 5) == 0
    for M in (1, 100, 512, 513, 16384, 1 << 20):
        teams = _lib.rms_norm_grad_workspace(M, 7) // 28
        assert 1 <= teams <= M and teams <= 1024
    assert _lib.rms_norm_grad_workspace(-1, 5) == _lib.rms_norm_grad_workspace(5, (1 << 30) + 1) == -1
    with pytest.raises(ValueError):
        layers.rms_norm_grad_workspace(-1, 1)


def layer_call(type=1, weights=1, out=1, gated=1, T=4, D=32, F=16, E=8, top=2, X=FAKE, ldx=32, ids=FAKE * 2, share=FAKE * 4,
               W_in=FAKE * 8, ldi=32, si=1024, sci=None, W_out=FAKE * 16, ldo=16, so=512, sco=None, Y=FAKE * 32, ldy=32,
               work=FAKE * 64, room=None):
    if room is None:
        room = _lib.expert_layer_workspace(type, T, D, F, top)
    return _lib.expert_layer(type, weights, out, gated, T, D, F, E, top, X, ldx, ids, share, W_in, ldi, si, sci, W_out, ldo, so,
                             sco, Y, ldy, work, room, None)


SCALED = dict(weights=3, sci=FAKE * 128, sco=FAKE * 256)
BLOCKS = dict(weights=5, sci=FAKE * 128, sco=FAKE * 256, ldi=16, si=512, ldo=8, so=256)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(weights=2), -2), (dict(weights=4), -2), (dict(out=2), -3), (dict(gated=2), -4), (dict(T=-1), -5),
    (dict(D=-1), -6), (dict(F=-1), -7), (dict(E=0), -8), (dict(top=0), -9), (dict(X=None), -10), (dict(ldx=31), -11),
    (dict(ids=None), -12), (dict(share=None), -13), (dict(W_in=None), -14), (dict(ldi=31), -15), (dict(si=-1), -16),
    (dict(sci=FAKE * 128), -17), (dict(SCALED, sci=None), -17), (dict(BLOCKS, ldi=15), -15), (dict(W_out=None), -18),
    (dict(ldo=15), -19), (dict(BLOCKS, ldo=7), -19), (dict(so=-1), -20), (dict(sco=FAKE * 256), -21), (dict(BLOCKS, sco=None), -21),
    (dict(Y=None), -22), (dict(ldy=31), -23), (dict(work=None), -24), (dict(work=FAKE * 64 + 8), -24), (dict(room=2175), -25),
    (dict(T=65, room=1 << 20), 5), (dict(T=64, top=9, room=1 << 20), 5), (dict(E=1025), 5), (dict(ldi=1 << 21), 5),
    (dict(F=(1 << 19) + 1, ldo=1 << 20, room=1 << 40), 5), (dict(si=(1 << 40) + 1), 5),
    (dict(Y=FAKE + 2), 3), (dict(Y=FAKE * 2 + 31), 3), (dict(Y=FAKE * 4), 3), (dict(Y=FAKE * 8 + 2 * (7 * 1024 + 1023)), 3),
    (dict(Y=FAKE * 16 + 2 * (7 * 512 + 511)), 3), (dict(work=FAKE * 32), 3), (dict(work=FAKE * 8), 3), (dict(work=FAKE), 3),
    (dict(SCALED, Y=FAKE * 128 + 4 * 8 * 32 - 4), 3), (dict(BLOCKS, Y=FAKE * 256 + 8 * 32 - 2), 3),
])
def test_expert_layer_codes(change, code):
    assert layer_call(**change) == code


def test_layer_workspace():
    f = _lib.expert_layer_workspace
    # h and products of every pair in whole lines of 128 bytes, and counters.
    assert f(1, 4, 32, 16, 2) == 4 * 2 * (128 + 128) + 128
    assert f(0, 3, 33, 65, 1) == 3 * (384 + 256) + 128
    assert f(1, 0, 32, 16, 2) == f(1, 4, 0, 16, 2) == 0
    assert f(1, 65, 8, 16, 1) == f(1, 64, 8, 16, 9) == f(3, 1, 1, 1, 1) == f(1, 1, 1, 1, 0) == f(1, 1, 1 << 20, 1, 1) == -1


def test_status_strings():
    f = _lib.layer_status_string
    assert f(-25) == b"argument 25 is illegal" and f(-17) == b"argument 17 is illegal" and f(-18) == b"argument 18 is illegal"
    assert f(3) == b"an output overlaps an input" and f(0) == b"ok" and f(-26) == b"unknown status"


def test_python_refusals():
    x, w, y = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4, 64)
    q4, s4 = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        fg.quantize_mx4(x.double(), q4, s4)
    with pytest.raises(TypeError):
        fg.quantize_mx4(x.int(), q4, s4)
    with pytest.raises(ValueError, match="GPU"):
        fg.quantize_mx4(x, q4, s4)
    with pytest.raises(TypeError):
        fg.gemm_mx4(x, s4, q4, s4, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="GPU"):
        fg.gemm_mx4(q4, s4, q4, s4, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="GPU"):
        fg.rms_norm(x, w, y)
    with pytest.raises(TypeError):
        fg.rms_norm(x.long(), w, y)
    with pytest.raises(TypeError):
        fg.rms_norm_grad(None, x, w, y)
    with pytest.raises(ValueError, match="GPU"):
        fg.rms_norm_grad(y, x, w, y)
    with pytest.raises(ValueError, match="GPU"):
        fg.expert_layer(x, torch.zeros(4, 1, dtype=torch.int32), x[:, :1], torch.zeros(2, 8, 64), torch.zeros(2, 64, 4), y)
