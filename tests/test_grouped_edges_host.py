"""What the plan of the grouped and 8-bit products chooses, without a GPU."""
import pytest
import torch

from fp32_gemm_amd import grouped

F32, BF16, F16, I8 = torch.float32, torch.bfloat16, torch.float16, torch.int8
FORMS = [("nt", t) for t in (F32, BF16, F16, I8)] + [(f, t) for f in ("nn", "tn") for t in (F32, BF16, F16)]


@pytest.mark.parametrize("form,dtype", FORMS)
def test_the_gpu_tests_reach_every_compiled_tile(form, dtype):
    import test_grouped_edges_gpu as on_gpu
    out = F32 if dtype is I8 else dtype
    cases = on_gpu.WEIGHT_GRADIENTS if form == "tn" else on_gpu.PRODUCTS
    seen = {grouped.plan(form, dtype, len(s), sum(s) + 3, N, K, out=out)["tile"] for s, K, N in cases}
    assert seen == set(grouped.tiles(form, dtype))


def test_tiles_refuse_what_does_not_exist():
    with pytest.raises(ValueError):
        grouped.tiles("nn", I8)
    assert grouped._lib.gemm_grouped_tile(0, 4, 0, 1, 1, 1, 1) == -1
    assert grouped._lib.gemm_grouped_tile(0, 0, 0, 0, 1, 1, 1) == -1


def test_long_weight_gradients_of_two_tiles_a_unit():
    # 512 tiles of 128 x 128: in 32 bits one resident tile a unit is faster where
    # groups differ in length, in 16 bits two are, or are as fast.
    for dtype, tile in ((F32, "128x128 deep"), (BF16, "128x128"), (F16, "128x128")):
        assert grouped.plan("tn", dtype, 8, 8000, 1024, 1024, out=F32)["tile"] == tile


THREADS = {"256x256": 512, "128x128": 512, "128x128 deep": 512, "64x64": 256, "16x32": 256, "16x16": 256}


@pytest.mark.parametrize("form,dtype", FORMS)
@pytest.mark.parametrize("groups,M,N,K", [
    (1, 1 << 28, 16, 16), (1, 1 << 30, 16, 16), (65536, 65536, 16384, 64), (65536, 1 << 24, 2048, 64),
    (4096, 1 << 20, 4096, 2048), (1, 16, 1 << 20, 1 << 17)])
def test_launches_hold_every_plan(form, dtype, groups, M, N, K):
    # HIP takes fewer than 2^32 threads a launch.
    p = grouped.plan(form, dtype, groups, M, N, K)
    assert 0 < p["grid"] * THREADS[p["tile"]] < 1 << 32


def test_what_no_launch_holds_is_unsupported():
    far = [1 << b for b in (40, 44, 48, 52)]
    bf16 = 1
    for groups, M, N, K in ((1, 1 << 30, 1 << 12, 16), (65536, 1 << 30, 1 << 12, 16)):
        with pytest.raises(ValueError):
            grouped.plan("nt", BF16, groups, M, N, K)
        assert grouped._lib.gemm_grouped_tile(0, bf16, bf16, groups, M, N, K) == -1
        assert grouped._lib.gemm_grouped(bf16, bf16, 1, groups, far[3], M, N, K, 1.0, far[0], K, far[1], K, N * K, 0.0,
                                         far[2], N, None) == 5
        assert grouped._lib.igemm(bf16, groups, far[3], M, N, K, far[0], K, far[1] + (1 << 42), far[1], K, N * K,
                                  far[1] + (1 << 43), None, far[2], N, None) == 5
    with pytest.raises(ValueError):  # 2^64 tiles
        grouped.plan("tn", BF16, 65536, 1, 1 << 30, 1 << 30)
    K = N = 1 << 20
    assert grouped._lib.gemm_grouped_wgrad(bf16, bf16, 65536, 1 << 39, 16, N, K, 1.0, far[0], K, far[1], N, 0.0,
                                           far[2], N, N * K, None) == 5
