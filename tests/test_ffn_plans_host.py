"""The plans of the feed-forward block's products (host only): every way of launching them that
ordinary sizes reach is run by the sizes whose results the GPU tests compare."""
import ctypes
import math
import random

import pytest

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

from ffn_plans import SHAPES, plan, ways


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def test_the_compared_sizes_cover_every_way(lib):
    covered = {way for dtype, shapes in SHAPES.items() for s in shapes for way in ways(lib, *s, dtype)}
    rng = random.Random(11)

    def size(most, multiple=1):
        return max(1, int(math.exp(rng.uniform(0.0, math.log(most + 1)))) // multiple) * multiple

    missing = {}
    for _ in range(20000):
        e = rng.choice([1, 8])
        s = (size(10000), size(6000, e), size(14000, e), size(6000, e), rng.choice(["bf16", "f32"]))
        for way in ways(lib, *s) - covered:
            missing.setdefault(way, s)
    assert not missing, "ways that no compared size runs, with a size each: %s" % missing


def test_paths(lib):
    assert plan(lib, 0, 64, 128, 64, "bf16", 0).path == 0
    assert plan(lib, 1, 64, 128, 64, "bf16", 0).path == 1
    assert plan(lib, 16, 64, 128, 64, "bf16", 0).path == 1
    assert plan(lib, 32, 64, 128, 64, "f32", 0).path == 1
    assert plan(lib, 33, 64, 128, 64, "f32", 0).path == 2
    back = plan(lib, 1, 64, 128, 64, "bf16", 1)
    assert back.path == 2 and list(back.products) == [1, 4]
    assert plan(lib, 1, 64, (1 << 20) + 1, 64, "bf16", 0).path == 2        # sums too long for a few warps


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F,O", [(1 << 17, 64, 64, 64), ((1 << 17) + 1, 64, 64, 64), (1 << 20, 8, 8, 8), (1 << 24, 8, 8, 8),
                                     (40, 8, 1 << 24, 8), (1 << 14, 1 << 20, 64, 64)])
def test_no_sum_is_longer_than_2048_blocks(lib, M, D, F, O, dtype):
    """The tensor cores cut what an addition leaves over: sums of more than 131072 of K come in parts."""
    for backward, lengths in ((0, ([D], [F])), (1, ([O], [2 * F, M, M, M]))):
        info = plan(lib, M, D, F, O, dtype, backward)
        for parts, of in zip(info.parts, lengths):
            for n, K in zip(parts, of):
                blocks = -(-K // 64)
                assert -(-blocks // max(n, 1)) <= 2048, (K, n)


def test_plan_query_refusals(lib):
    info, p = gdn.GdnFfnPlanInfo(), ctypes.c_void_p(4096)
    good = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, 64, 40, 64, 128, 64, 0, 0)
    assert lib.gdn_gated_ffn_plan_query(None, 0, None, 0, info) == 1
    assert lib.gdn_gated_ffn_plan_query(good, 0, None, 0, None) == 1
    assert lib.gdn_gated_ffn_plan_query(good, 1, p, 63, info) == 1
    assert lib.gdn_gated_ffn_plan_query(good, 1, p, 1 << 37, info) == 2
    assert lib.gdn_gated_ffn_plan_query(good, 0, None, 0, info) == 0
    assert lib.gdn_gated_ffn_plan_query(gdn.GdnFfnDesc(4096, 4096, 4096, 4096, 64, (1 << 24) + 1, 64, 128, 64, 0, 0), 0, None, 0, info) == 2
