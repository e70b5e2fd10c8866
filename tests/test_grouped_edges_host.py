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
