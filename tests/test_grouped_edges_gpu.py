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
