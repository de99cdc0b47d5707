"""CPU tests of how products of 4-bit matrices are cut into tiles and parts: the sizes that the GPU tests run reach every way through
the kernels, and stay there when the rule changes."""
import ctypes

import pytest

import streaming_causal_video_gb300 as sd
import test_gpu_project
from project_plans import FEW, PLANS, TILES


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def plan(size):
    M, N, K = size
    return sd.debug_mx4_plan(sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K))


@pytest.mark.parametrize("size", list(PLANS), ids=str)
def test_sizes_go_the_way_that_they_are_to_test(size):
    assert plan(size) == PLANS[size]


def test_every_way_is_taken_by_a_size():
    assert {p[:2] for p in FEW.values()} == {(w, n) for w in (16, 32, 64) for n in (1, 2, 4, 8)}
    several = {(w, n, rounds > 1) for w, n, rounds in TILES.values()}
    assert several == {(w, 1, more) for w in (128, 192, 256) for more in (False, True)} | {(128, 2, False), (128, 4, False)}
    # nothing else comes out of the rule
    for M in (1, 16, 17, 33, 64, 65, 130, 256, 300, 520, 1001, 2500, 4680, 10800):
        for N in (1, 130, 700, 1536, 2500, 6144, 20480):
            for K in (1, 300, 1536, 4096, 8200, 20480):
                width, parts, rounds = plan((M, N, K))
                if M <= 64:
                    assert (width, parts) in {p[:2] for p in FEW.values()} and rounds == 1 and M <= width
                else:
                    assert (width, parts, rounds > 1) in several


def test_parts_of_the_depth_of_the_older_sizes():
    """Two parts and four, and one where the exchange would cost more."""
    assert plan((700, 650, 8300)) == plan((300, 1030, 8200)) == (128, 2, 1)
    assert plan((512, 512, 8192)) == plan((90, 260, 9000)) == (128, 4, 1) and plan((512, 1536, 4096)) == (128, 1, 1)
    assert (300, 1030, 8200) in test_gpu_project.SHAPES and (700, 650, 8300) in test_gpu_project.DEEP


def test_the_query_refuses_what_the_product_refuses():
    out = (ctypes.c_int32 * 3)(7, 7, 7)
    L = sd.lib()
    for bad in (dict(rows=0), dict(depth=-1), dict(activation=3), dict(out_row_stride=1)):
        cfg = sd.Mx4ProductConfig.make(**{**dict(rows=6, cols=40, depth=100), **bad})
        with pytest.raises(sd.SDV2Error):
            sd.debug_mx4_plan(cfg)
        assert L.sdv2_debug_mx4_plan(cfg, out) == 1 and list(out) == [7, 7, 7]
    cfg = sd.Mx4ProductConfig.make(rows=6, cols=40, depth=100)
    assert L.sdv2_debug_mx4_plan(cfg, None) == 1 and L.sdv2_debug_mx4_plan(None, out) == 1
    assert b"NULL" in L.sdv2_last_error()
