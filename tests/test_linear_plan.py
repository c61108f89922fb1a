"""Every kernel form that the planner of the linear and gated products can choose, held against
the fp64 oracle on the GPU; and, on the CPU, that the shapes here are all of them.

The shapes are ragged (rows odd, dimensions off every tile), and where a contraction is tiled a
workgroup has 10 steps of it at least, so that its ring of operands goes round.
"""
import random

import pytest

import linear_plans as P
from test_linear_gpu import check_glu, check_glu_backward, check_linear, check_linear_backward

# (call, type): shapes (rows, d_out, d_in)
SHAPES = {
    ("linear", "fp32"): [
        (1, 24, 24), (3, 24, 4112), (3, 4128, 24), (15, 88, 152), (17, 32, 4152), (17, 4336, 24), (27, 104, 72),
        (35, 24, 4056), (35, 4320, 32), (45, 112, 40), (49, 40, 312), (53, 24, 5800), (341, 17208, 312),
        (525, 3704, 1272), (643, 1496, 304), (663, 720, 1008), (941, 2200, 312), (985, 2072, 1048),
        (1091, 904, 1016), (1741, 2312, 1440), (1931, 3104, 304), (5611, 2416, 296)],
    ("linear", "bf16"): [
        (1, 24, 24), (3, 24, 8864), (3, 4128, 24), (15, 88, 152), (17, 24, 8616), (17, 4336, 24), (27, 104, 72),
        (35, 24, 9192), (35, 4320, 32), (45, 112, 40), (49, 24, 616), (49, 32, 10512), (283, 17832, 584),
        (335, 5896, 6168), (577, 1632, 3960), (725, 464, 4504), (1163, 3336, 7456), (1657, 2440, 600),
        (1685, 1192, 584), (1723, 608, 584), (2101, 3984, 592), (2807, 648, 5840)],
    ("glu", "fp32"): [
        (1, 24, 24), (3, 24, 4112), (3, 4128, 24), (15, 88, 152), (17, 32, 4152), (17, 4336, 24), (27, 104, 72),
        (35, 24, 4056), (35, 4320, 32), (45, 112, 40), (49, 40, 312), (53, 24, 5800), (291, 816, 952),
        (387, 1160, 304), (593, 3376, 1488), (643, 1496, 304), (817, 1376, 1048), (903, 584, 936),
        (1041, 3576, 360), (1091, 904, 1016), (3355, 1832, 352), (3485, 840, 296)],
    ("glu", "bf16"): [
        (1, 24, 24), (3, 24, 8864), (3, 4128, 24), (15, 88, 152), (17, 24, 8616), (17, 4336, 24), (27, 104, 72),
        (35, 24, 9192), (35, 4320, 32), (45, 112, 40), (49, 24, 616), (49, 32, 10512), (263, 3552, 5536),
        (385, 392, 4024), (449, 1032, 600), (649, 1560, 5816), (863, 584, 3800), (1087, 3424, 584),
        (1093, 2016, 7096), (1685, 1192, 584), (1723, 608, 584), (3343, 1224, 584)],
    ("linear_backward", "fp32"): [
        (1, 160, 6584), (1, 520, 2024), (17, 216, 5208), (17, 288, 3656), (297, 296, 1624), (311, 304, 24),
        (321, 352, 3688), (353, 2920, 1200), (437, 408, 14752), (453, 480, 6160), (525, 496, 1928),
        (999, 648, 152), (1259, 1776, 664), (1283, 664, 720), (1733, 952, 136), (2751, 328, 1240),
        (5073, 2576, 488)],
    ("linear_backward", "bf16"): [
        (1, 360, 5864), (1, 1712, 1232), (17, 1256, 1696), (21, 312, 6888), (33, 408, 14544), (33, 17584, 536),
        (33, 18896, 928), (35, 13776, 664), (37, 9960, 360), (65, 7504, 2712), (77, 656, 8968), (91, 4448, 344),
        (593, 616, 24), (631, 648, 856), (647, 592, 3376), (653, 88, 8504), (691, 584, 7960), (959, 592, 1312),
        (1889, 1240, 88), (2805, 40, 7656), (3089, 24, 864), (3781, 24, 2616), (4149, 24, 3368), (5089, 72, 536)],
    ("glu_backward", "fp32"): [
        (1, 40, 13160), (1, 168, 3144), (17, 96, 5784), (17, 288, 1832), (299, 152, 48), (309, 152, 3336),
        (315, 152, 10536), (385, 168, 1328), (415, 1512, 1144), (479, 240, 12968), (561, 328, 1696),
        (1057, 536, 216), (1097, 624, 432), (1327, 352, 72), (1375, 2568, 200), (2975, 248, 1176),
        (3219, 1632, 664)],
    ("glu_backward", "bf16"): [
        (1, 160, 6584), (1, 520, 2024), (17, 216, 5208), (17, 288, 3656), (35, 1888, 4472), (35, 3720, 928),
        (35, 8400, 552), (37, 7080, 656), (39, 6248, 288), (75, 2256, 328), (87, 312, 9440), (581, 296, 24),
        (637, 304, 776), (665, 40, 8288), (665, 400, 2704), (671, 304, 6544), (683, 312, 1568), (1909, 616, 88),
        (2453, 24, 3728), (3781, 24, 2616), (4017, 5208, 136), (4513, 48, 328), (5431, 40, 552)],
}
CHECKS = {"linear": check_linear, "glu": check_glu, "linear_backward": check_linear_backward,
          "glu_backward": check_glu_backward}
CALLS = [(call, dtype, s) for (call, dtype), shapes in SHAPES.items() for s in shapes]


def variants(so, call, dtype, shape, deep):
    f = P.gradient_variants if call.endswith("backward") else P.forward_variants
    return f(so, *shape, call.startswith("glu"), dtype, deep)


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    return P.compile_planner(str(tmp_path_factory.mktemp("planner")))


def test_the_shapes_reach_every_form(planner):
    """Whatever 40000 drawn shapes reach, over all sizes up to far past every threshold, the
    shapes of this file reach too."""
    rng = random.Random(20)

    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    reached = set()
    for _ in range(40000):
        shape = (spread(1, 16384), 8 * spread(1, 4096), 8 * spread(1, 4096))
        for call in CHECKS:
            for dtype in ("fp32", "bf16"):
                reached |= variants(planner, call, dtype, shape, False)
    covered = set().union(*(variants(planner, *c, True) for c in CALLS))
    assert reached <= covered, sorted(map(str, reached - covered))
    # the forms that there are: one row; few rows in 1 to 3 blocks with two waves, or more and
    # whole or split; six tiles whole or split; few-rows gradients; one grid or two
    tiles = {v[2:4] for v in covered if len(v) == 5 and isinstance(v[2], int)}
    assert tiles == {(256, 256), (256, 128), (128, 256), (128, 128), (64, 128), (64, 64)}
    for dtype in ("fp32", "bf16"):
        for name in ("linear", "glu", "dx", "dw", "glu dx", "glu dw"):
            for t in tiles:
                for cut in ("whole", "split"):
                    assert (dtype, name, *t, cut) in covered, (dtype, name, t, cut)


@pytest.mark.gpu
@pytest.mark.parametrize("call, dtype, shape", CALLS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_form(call, dtype, shape):
    CHECKS[call](*shape, dtype, "silu", seed=sum(shape))


# Gated gradients of 33 to 64 rows: the second block of 32 rows partly filled, the seam between the
# two weights inside it, d_out off the waves' rows.
TWO_BLOCKS = [(49, 648, 13064), (63, 2056, 4168), (34, 8536, 1000)]


def test_two_blocks_of_rows_stay_on_their_kernel(planner):
    for shape in TWO_BLOCKS:
        assert ("bf16", "glu dw", "few-rows gradients", 64, "whole") in P.gradient_variants(planner, *shape, True, "bf16")
    # 2 x 640 x 13064 is not large enough for it
    assert ("bf16", "glu dw", "few-rows gradients", 64, "whole") not in P.gradient_variants(planner, 49, 640, 13064, True,
                                                                                            "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", TWO_BLOCKS, ids=lambda s: "x".join(map(str, s)))
def test_gated_gradients_of_two_blocks_of_rows(shape):
    check_glu_backward(*shape, "bf16", "gelu", pad=8, seed=71)


# us on one MI355X of the few-rows kernel and of the tiles, where they are apart
TIMES = [("bf16", "linear", (16, 4096, 4096), 8.8, 13.4), ("bf16", "linear", (16, 11008, 4096), 18.7, 21.8),
         ("bf16", "linear", (24, 4096, 11008), 20.4, 26.9), ("bf16", "linear", (24, 4096, 4096), 9.7, 13.7),
         ("bf16", "linear", (32, 8192, 1024), 6.8, 9.1), ("bf16", "linear", (32, 5120, 8192), 28.9, 24.3),
         ("bf16", "linear", (32, 16384, 4096), 35.5, 26.8), ("bf16", "linear", (32, 28672, 8192), 103.6, 90.3),
         ("bf16", "linear", (30, 14176, 4096), 30.6, 25.6), ("bf16", "linear", (48, 4096, 4096), 12.1, 14.4),
         ("bf16", "linear", (48, 8192, 1024), 7.7, 9.4), ("bf16", "linear", (48, 8192, 8192), 39.9, 33.1),
         ("bf16", "linear", (48, 5120, 5560), 35.4, 24.0), ("bf16", "linear", (48, 11008, 4096), 32.3, 24.2),
         ("bf16", "glu", (24, 4096, 4096), 14.2, 21.0), ("bf16", "glu", (30, 8192, 4096), 24.7, 36.9),
         ("bf16", "glu", (32, 11008, 1024), 15.1, 13.6), ("bf16", "glu", (48, 4096, 8192), 30.0, 34.4),
         ("bf16", "glu", (48, 2048, 7168), 22.9, 19.8), ("bf16", "glu", (48, 5120, 8192), 46.4, 39.3),
         ("bf16", "glu", (48, 11008, 4096), 43.3, 38.7), ("fp32", "linear", (32, 11008, 4096), 48.5, 78.9),
         ("fp32", "linear", (48, 8192, 1024), 13.9, 19.1), ("fp32", "linear", (48, 11008, 1024), 24.9, 22.9),
         ("fp32", "glu", (32, 8192, 8192), 93.3, 164.4), ("fp32", "glu", (48, 11008, 4096), 100.6, 132.0),
         ("fp32", "glu", (48, 28672, 2048), 126.6, 156.7)]


def test_the_rule_for_few_rows_takes_the_faster_kernel(planner):
    for dtype, call, shape, few, tiles in TIMES:
        (form,) = variants(planner, call, dtype, shape, False)
        assert (form[2] == "few rows") == (few < tiles), (dtype, call, shape, form)


def test_the_rule_for_two_waves_takes_the_faster_one(planner):
    """... and of the few-rows kernel with two waves a workgroup, and with more."""
    for dtype, call, shape, two, more in [
            ("bf16", "linear", (8, 11008, 1024), 6.6, 10.2), ("bf16", "linear", (8, 14176, 6144), 33.0, 37.3),
            ("bf16", "linear", (8, 8192, 8192), 29.2, 25.7), ("bf16", "linear", (32, 8192, 1024), 6.8, 8.6),
            ("bf16", "glu", (16, 28672, 2048), 40.2, 48.8), ("bf16", "glu", (16, 8192, 8192), 48.9, 45.1),
            ("bf16", "glu", (30, 8192, 4096), 24.7, 27.3), ("fp32", "linear", (16, 14176, 2048), 23.6, 30.2),
            ("fp32", "linear", (24, 8192, 8192), 72.9, 55.8), ("fp32", "glu", (48, 28672, 2048), 126.6, 136.6)]:
        (form,) = variants(planner, call, dtype, shape, False)
        assert form[2] == "few rows" and (form[4] == 2) == (two < more), (dtype, call, shape, form)
