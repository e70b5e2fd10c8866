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


# ---- the order of the tiles, by the kernels' own code on the host ---------------------

ROWS = {"256x256": 256, "128x128": 128, "128x128 deep": 128, "64x64": 64, "16x32": 16, "16x16": 16}
COLS = {"256x256": 256, "128x128": 128, "128x128 deep": 128, "64x64": 64, "16x32": 32, "16x16": 16}


def splits(bm):
    """Groups' lengths: each with one row more than whole tiles (the most tiles
    there can be), each with only a part of a tile, single rows, gaps, more groups
    than the 64 that a wave looks at together, and ordinary ones."""
    import random
    r = random.Random(bm)
    yield [1]
    yield [bm + 1] * 3
    yield [1] * 7
    yield [0, 0, 5, 0]
    yield [2 * bm + 1, 1, bm + 1, 0, 1]
    yield [1, 0] * 40
    yield [bm * (i % 3) + 1 for i in range(70)]
    yield [r.randrange(1, bm) for _ in range(150)]
    for groups in (2, 9, 64, 65, 129):
        yield [r.choice((0, 1, r.randrange(3 * bm), bm * r.randrange(3))) for _ in range(groups)]


@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "16x32", "16x16"])
@pytest.mark.parametrize("tiles_n", [1, 2, 3, 5, 12])
def test_every_output_tile_has_one_workgroup(tile, tiles_n):
    bm, N = ROWS[tile], COLS[tile] * (tiles_n - 1) + 1
    for sizes in splits(bm):
        off = [0]
        for n in sizes:
            off.append(off[-1] + n)
        order = grouped.tile_order("nt", BF16, tile, off, off[-1], N, 64)
        got = sorted(t for t in order if t[0] >= 0)
        want = sorted((e, row, off[e + 1], n) for e in range(len(sizes)) for row in range(off[e], off[e + 1], bm)
                      for n in range(tiles_n))
        assert got == want


@pytest.mark.parametrize("tile", ["256x256", "128x128 deep", "64x64"])
@pytest.mark.parametrize("K,N", [(1, 1), (700, 300), (513, 1025)])
def test_every_weight_gradient_tile_has_one_workgroup(tile, K, N):
    for sizes in ([3000, 1, 0, 900, 3000], [0], [10] * 70, list(range(600, 664))):
        off = [0]
        for n in sizes:
            off.append(off[-1] + n)
        order = grouped.tile_order("tn", BF16, tile, off, off[-1], N, K)
        up = lambda n, t: -(-n // t)  # noqa: E731
        want = sorted((e, m, 0, n) for e in range(len(sizes)) for m in range(up(K, ROWS[tile]))
                      for n in range(up(N, COLS[tile])))
        assert sorted(t for t in order if t[0] >= 0) == want
        if len(sizes) <= 64 and sum(sizes) / len(sizes) >= 512:  # long: the longest first
            lengths = [sizes[t[0]] for t in order if t[0] >= 0]
            assert lengths == sorted(lengths, reverse=True)


def test_one_group_of_all_rows():
    order = grouped.tile_order("nn", F32, "64x64", None, 130, 70, 64)
    assert sorted(t for t in order if t[0] >= 0) == sorted((0, m, 130, n) for m in (0, 64, 128) for n in (0, 1))


def test_tile_order_refusals():
    for bad in (dict(tile="16x16", form="nn"), dict(offsets=[0]), dict(M=-1), dict(M=1 << 30, tile="16x16")):
        args = dict(form="nt", dtype=BF16, tile="64x64", offsets=[0, 5], M=5, N=64, K=64, **{})
        args.update(bad)
        with pytest.raises(ValueError):
            grouped.tile_order(**args)


@pytest.mark.parametrize("tile", ["256x256", "128x128", "64x64", "16x32", "16x16"])
def test_offsets_out_of_order_never_leave_the_operands(tile):
    # Every tile is one of a group's: rows inside the group, columns inside N. Where
    # the groups count more whole tiles than the rows can have tiles, there is none at
    # all: sums would pass 32 bits (65536 groups of which every other one holds all).
    import random
    r = random.Random(ROWS[tile])
    for M in (5, 1000, 1 << 20, 150000001):
        for groups in (3, 64, 65, 1000, 65536):
            for tiles_n in (1, 3):
                if M // ROWS[tile] * tiles_n > 1 << 23:
                    continue  # more than a launch holds
                kinds = [[0 if e % 2 == 0 else M for e in range(groups + 1)],
                         [r.choice((-5, 0, M // 2, M, 1 << 30, r.randrange(M))) for _ in range(groups + 1)]]
                for off in kinds:
                    span = lambda e: (min(max(off[e], 0), M), min(max(off[e + 1], min(max(off[e], 0), M)), M))  # noqa: E731
                    whole = sum((hi - lo) // ROWS[tile] for lo, hi in map(span, range(groups)))
                    args = ("nt", BF16, tile, off, M, tiles_n * COLS[tile], 64)
                    for first in (0, r.randrange(1 << 16), 1 << 19):
                        for e, row, end, n in grouped.tile_order(*args, first, 64):
                            if e < 0:
                                continue
                            lo, hi = span(e)
                            assert 0 <= n < tiles_n and lo <= row < hi == end and (row - lo) % ROWS[tile] == 0
                            assert whole <= M // ROWS[tile] + min(groups, M)
