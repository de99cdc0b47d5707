"""GPU tests of 4-bit products along every way through the kernels (project_plans.py): what test_gpu_project.py checks of a product,
at sizes whose tiles and parts are asserted before they run."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import streaming_causal_video_gb300 as sd
import test_gpu_project as base
from project_plans import FEW, PLANS, TILES
from test_gpu_project import gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32

# few rows in two, four and eight parts; tiles of 128 rows in two parts; several tiles of 256 of a pair
NEW = [(3, 10000, 3200), (3, 300, 3200), (16, 257, 9000), (17, 10000, 3200), (31, 1030, 3330), (64, 10000, 3200), (40, 300, 3200),
       (700, 650, 8300), (77, 4100, 8200), (5400, 2500, 300), (5400, 2501, 300), (1500, 8000, 1300)]


def on_its_way(size):
    M, N, K = size
    assert sd.debug_mx4_plan(sd.Mx4ProductConfig.make(rows=M, cols=N, depth=K)) == PLANS[size]


@pytest.mark.parametrize("out_dtype", [FP, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [*FEW, *(s for s in TILES if s[0] * s[1] < 14e6)], ids=str)
def test_products(size, out_dtype):
    on_its_way(size)
    base.test_products(size, out_dtype)


@pytest.mark.parametrize("out_dtype", [FP, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [s for s in TILES if TILES[s][2] > 1], ids=str)
def test_products_of_several_tiles_of_a_pair(size, out_dtype):
    on_its_way(size)
    base.test_products_of_several_tiles_of_a_pair(size, out_dtype)


@pytest.mark.parametrize("size", NEW, ids=str)
def test_sums_that_32_bits_hold_are_exact(size):
    """Partial sums are at most 6 * 6 * 2 * 2 * 9000 = 1.3 million ones, 5.2 million quarters: below 2^24."""
    on_its_way(size)
    base.test_sums_that_32_bits_hold_are_exact(size)


@pytest.mark.parametrize("size", NEW, ids=str)
def test_nan_stays_where_it_belongs(size):
    on_its_way(size)
    base.test_a_scale_of_nan_reaches_its_row_and_its_column_only(size)
    base.test_a_nan_leaves_its_neighbours_with_an_activation(size)


@pytest.mark.parametrize("size", NEW, ids=str)
def test_the_same_bits_again_from_graphs_at_once(size):
    on_its_way(size)
    base.test_products_are_deterministic_and_replay_from_graphs_that_share_a_workspace(size)


@pytest.mark.parametrize("size", NEW, ids=str)
def test_calls_write_only_their_outputs(size):
    on_its_way(size)
    base.test_calls_write_only_their_outputs(size)


@pytest.mark.parametrize("size,step", [((3, 300, 3200), 5), ((3, 10000, 3200), 12), ((17, 10000, 3200), 0), ((40, 300, 3200), 7),
                                       ((64, 10000, 3200), 6), ((77, 4100, 8200), 32), ((5400, 2500, 300), 1), ((1500, 8000, 1300), 4)], ids=str)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(size, step):
    on_its_way(size)
    base.test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(size, step)


def test_first_calls_of_a_process_inside_a_capture():
    was = "((3, 200, 2048), (70, 300, 2048), (90, 260, 9000), (600, 700, 2048))"
    assert was in base.FIRST_CALLS
    text = base.FIRST_CALLS.replace(was, "((3, 300, 3200), (64, 10000, 3200), (16, 257, 9000), (700, 650, 8300), (5400, 2500, 300))")
    run = subprocess.run([sys.executable, "-c", text, str(Path(__file__).resolve().parents[1])], capture_output=True, text=True, timeout=240)
    assert run.returncode == 0 and run.stdout.strip().endswith("same"), run.stderr[-2000:]


def test_calls_from_several_host_threads(monkeypatch):
    sizes = [(3, 10000, 3200), (40, 300, 3200), (17, 10000, 3200), (700, 650, 8300), (5400, 2500, 300), (3, 300, 3200), (77, 4100, 8200),
             (1500, 8000, 1300)]
    for size in sizes:
        on_its_way(size)
    monkeypatch.setattr(base, "SHAPES", sizes)
    base.test_calls_from_several_host_threads()
