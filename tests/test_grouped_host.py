"""The grouped and 8-bit products' C ABI and argument checks, without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp32_gemm_amd as fg
from fp32_gemm_amd import grouped
from fp32_gemm_amd.binding import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "grouped_gemm.h")
FAKE = 1 << 40  # a well-aligned, never-dereferenced address


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def test_header_and_library_agree():
    assert declared() == grouped.exported_symbols()
    lib = ctypes.CDLL(fg.library_path())
    for name in declared():
        assert hasattr(lib, name), name


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "grouped_gemm.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-c", str(src),
                    "-o", str(tmp_path / "h.o")], check=True)


def grouped_call(type=1, out=1, trans=0, groups=4, off=FAKE * 8, M=64, N=32, K=16, X=FAKE, ldx=16, W=FAKE * 2, ldw=32,
                 stride=512, Y=FAKE * 4, ldy=32):
    return _lib.gemm_grouped(type, out, trans, groups, off, M, N, K, 1.0, X, ldx, W, ldw, stride, 0.0, Y, ldy, None)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(type=-1), -1), (dict(out=2), -2), (dict(type=0, out=1), -2), (dict(trans=2), -3),
    (dict(groups=0), -4), (dict(off=None), -4), (dict(M=-1), -6), (dict(N=-1), -7), (dict(K=-1), -8),
    (dict(X=None), -10), (dict(ldx=15), -11), (dict(W=None), -12), (dict(ldw=31), -13), (dict(trans=1, ldw=15), -13),
    (dict(stride=-1), -14), (dict(Y=None), -16), (dict(ldy=31), -17),
    (dict(M=(1 << 30) + 1), 5), (dict(ldx=1 << 21), 5), (dict(groups=(1 << 16) + 1), 5), (dict(stride=(1 << 40) + 1), 5),
    (dict(Y=FAKE + 16), 3), (dict(Y=FAKE * 2 + 3 * 512 * 2), 3), (dict(Y=FAKE * 8), 3),
])
def test_gemm_grouped_codes(change, code):
    assert grouped_call(**change) == code


def test_gemm_grouped_quick_returns():
    assert grouped_call(M=0, X=None, Y=None) == 0
    assert grouped_call(N=0, W=None, Y=None, ldw=1) == 0


def wgrad_call(type=1, out=0, groups=4, off=FAKE * 8, M=64, N=32, K=16, X=FAKE, ldx=16, dY=FAKE * 2, lddy=32,
               dW=FAKE * 4, lddw=32, stride=512):
    return _lib.gemm_grouped_wgrad(type, out, groups, off, M, N, K, 1.0, X, ldx, dY, lddy, 0.0, dW, lddw, stride, None)


@pytest.mark.parametrize("change,code", [
    (dict(type=4), -1), (dict(out=2), -2), (dict(groups=-1), -3), (dict(off=None), -3), (dict(M=-1), -5),
    (dict(N=-1), -6), (dict(K=-1), -7), (dict(X=None), -9), (dict(ldx=15), -10), (dict(dY=None), -11),
    (dict(lddy=31), -12), (dict(dW=None), -14), (dict(lddw=31), -15), (dict(stride=511), -16), (dict(stride=0), -16),
    (dict(N=(1 << 30) + 1, lddy=(1 << 30) + 1, lddw=(1 << 30) + 1), 5), (dict(dW=FAKE), 3), (dict(dW=FAKE * 2 + 64), 3),
])
def test_wgrad_codes(change, code):
    assert wgrad_call(**change) == code


def test_wgrad_quick_returns():
    assert wgrad_call(K=0, X=None, dW=None, ldx=1) == 0
    assert wgrad_call(N=0, dY=None, dW=None) == 0


def igemm_call(out=1, groups=4, off=FAKE * 8, M=64, N=32, K=16, A=FAKE, lda=16, sa=FAKE * 16, B=FAKE * 2, ldb=16,
               stride=512, sb=FAKE * 32, bias=None, C=FAKE * 4, ldc=32):
    return _lib.igemm(out, groups, off, M, N, K, A, lda, sa, B, ldb, stride, sb, bias, C, ldc, None)


@pytest.mark.parametrize("change,code", [
    (dict(out=3), -1), (dict(groups=0), -2), (dict(off=None), -2), (dict(M=-1), -4), (dict(N=-1), -5), (dict(K=-1), -6),
    (dict(A=None), -7), (dict(lda=15), -8), (dict(sa=None), -9), (dict(B=None), -10), (dict(ldb=15), -11),
    (dict(stride=-1), -12), (dict(sb=None), -13), (dict(C=None), -15), (dict(ldc=31), -16),
    (dict(K=131072, lda=131072, ldb=131072), 5), (dict(C=FAKE * 16), 3), (dict(C=FAKE * 32 + 4), 3),
    (dict(bias=FAKE * 4), 3), (dict(C=FAKE + 8), 3),
])
def test_igemm_codes(change, code):
    assert igemm_call(**change) == code


def quantize_call(type=1, M=8, K=16, X=FAKE, ldx=16, Q=FAKE * 2, ldq=16, scale=FAKE * 4):
    return _lib.quantize_rows(type, M, K, X, ldx, Q, ldq, scale, None)


@pytest.mark.parametrize("change,code", [
    (dict(type=3), -1), (dict(M=-1), -2), (dict(K=-1), -3), (dict(X=None), -4), (dict(ldx=15), -5), (dict(Q=None), -6),
    (dict(ldq=15), -7), (dict(scale=None), -8), (dict(M=(1 << 30) + 1), 5), (dict(Q=FAKE + 8), 3),
    (dict(scale=FAKE), 3), (dict(scale=FAKE * 2 + 16), 3),
])
def test_quantize_codes(change, code):
    assert quantize_call(**change) == code


def test_status_strings():
    f = _lib.gemm_grouped_status_string
    assert f(-17) == b"argument 17 is illegal" and f(-1) == b"argument 1 is illegal"
    assert f(3) == b"an output overlaps an input" and f(0) == b"ok"
    assert f(99) == b"unknown status" and f(-18) == b"unknown status"


@pytest.mark.parametrize("form,dtype", [("nt", torch.int8), ("nt", torch.bfloat16), ("nn", torch.float32),
                                        ("tn", torch.float16)])
def test_plan_covers_any_split_of_the_rows(form, dtype):
    # The grid is sized without the offsets: it must hold the tiles of the worst split.
    for groups, M, N, K in [(1, 1, 64, 64), (64, 7, 100, 64), (8, 1000, 777, 640), (16, 16384, 2048, 4096), (3, 0, 64, 64)]:
        p = grouped.plan(form, dtype, groups, M, N, K)
        up = lambda n, t: -(-n // t)  # noqa: E731
        if form == "tn":
            assert p["grid"] == groups * up(up(K, p["BM"]) * up(N, p["BN"]), 8) * 8
            continue
        used = min(groups, M)
        ones = [1] * max(used - 1, 0) + ([M - used + 1] if used else [])  # one row each, the rest in one group
        even = [M // used + (i < M % used) for i in range(used)] if used else []
        for split in (ones, even):
            assert sum(up(n, p["BM"]) for n in split) * up(N, p["BN"]) <= p["grid"]
    with pytest.raises(ValueError):
        grouped.plan(form, dtype, 0, 1, 1, 1)


def test_the_gpu_tests_reach_every_tile():
    import test_grouped_gpu as on_gpu
    bf16, every = torch.bfloat16, {(256, 256), (128, 128), (64, 64), (16, 32), (16, 16)}

    def tile(form, dtype, groups, M, N, K):
        p = grouped.plan(form, dtype, groups, M, N, K)
        return p["BM"], p["BN"]

    for form in ("nt", "nn"):
        seen = {tile(form, bf16, len(s), sum(s) + 3, N, K) for s, K, N in on_gpu.TILES}
        assert seen == (every if form == "nt" else every - {(16, 16)})
    assert {tile("nt", torch.int8, 1, M, N, K) for M, N, K in on_gpu.IGEMM_TILES} == every
    for dtype in (bf16, torch.float32):
        seen = {tile("tn", d, len(s), sum(s) + 3, N, K) for d, s, K, N in on_gpu.WGRAD_TILES if d is dtype}
        assert seen == {(256, 256), (128, 128), (64, 64)}
    seen = {tile("nn", bf16, 150, 150 * sum(each) // len(each), N, K) for each, K, N in on_gpu.MANY}
    assert seen >= {(256, 256), (16, 32)}


def test_python_refusals():
    x, w, y = torch.zeros(4, 8), torch.zeros(2, 8, 6), torch.zeros(4, 6)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        fg.gemm_grouped(x.double(), w, off, y)
    with pytest.raises(TypeError):
        fg.gemm_grouped([1.0], w, off, y)
    with pytest.raises(ValueError, match="GPU"):
        fg.gemm_grouped(x, w, off, y)
    with pytest.raises(ValueError, match="2-D"):
        fg.gemm_grouped(x[0], w, off, y)
    with pytest.raises(TypeError):
        fg.quantize_rows(x.int(), x.to(torch.int8), x[:, 0])
    with pytest.raises(TypeError):
        fg.igemm(x, x[:, 0], x, x[:, 0], y)
    with pytest.raises(ValueError, match="GPU"):
        fg.gemm_grouped_wgrad(x, y, off, torch.zeros(2, 8, 6))
