"""The rule by which a linear layer's call takes its kernel (csrc/linear_shape.h), on 256
compute units: the GPU tests' sizes reach every shape and every height of its tiles."""
import pytest

import test_gpu_linear as plain
import test_gpu_linear_sums as sums
import test_gpu_linear_tiles as tiles
from linear_shapes import TILES, picked


def sizes_of(test, names):
    """The parameter sets of a test, in the order of `names`."""
    marks = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0].split(",")[:len(names)] == names]
    return [v[:len(names)] for v in marks[0].args[1]]


@pytest.mark.parametrize("op", ["forward", "grad_x"])
def test_sizes_reach_their_shape(op):
    for shape, cols, q in tiles.ROWS:
        N, K = (cols, q) if op == "forward" else (q, cols)
        for act in ("none", "gelu", "swiglu"):
            assert picked(op, tiles.R, tiles.E, N, K, act) == shape
    assert {s for s, _, _ in tiles.ROWS} == set(TILES)


def test_matrix_gradients_reach_their_shape():
    for shape, N, K in tiles.GRAD_W:
        assert picked("grad_w", tiles.R, tiles.E, N, K) == shape
    assert {s for s, _, _ in tiles.GRAD_W} == set(TILES) - {"288x256"}
    rows = sizes_of(sums.test_bias_gradient_of_one_sign, ["rows", "N", "K"])
    assert {picked("grad_w", r, 0, N, K) for r, N, K in rows} >= {"256x256", "128x128", "64x64 quad"}


@pytest.mark.parametrize("shape", TILES)
def test_ragged_rows_reach_every_height(shape):
    most, step = tiles.HEIGHTS[shape]
    assert tiles.rounds(shape) == set(range(1, most // step + 1))


def test_few_rows_reach_every_stream():
    seen = {picked("forward", T * k, E, N, K, act) for T, k, E, N, K, _, _ in plain.GROUPED for act in plain.ACTS}
    seen |= {picked("forward", rows, 0, N, K, act) for rows, N, K in plain.PLAIN for act in plain.ACTS}
    assert {s for s in seen if s.startswith("stream")} == {"stream 1.1", "stream 2.1", "stream 2.2", "stream 4.1"}


def test_rule():
    """Where the rule changes from one kernel to another."""
    assert picked("forward", 16, 0, 4096, 7168) == "stream 1.1" and picked("forward", 16, 0, 4096, 7168, "swiglu") == "stream 2.1"
    assert picked("forward", 32, 0, 4096, 7168) == "stream 2.2" and picked("forward", 33, 0, 4096, 7168) == "64x64 quad"
    # sorted rows: half as many an expert
    assert picked("forward", 64, 8, 4096, 7168) == "stream 4.1" and picked("forward", 128, 8, 4096, 7168) == "stream 2.2"
    assert picked("forward", 129, 8, 4096, 7168) not in ("stream 2.2", "stream 4.1")
    # experts of 256 rows, more or less, and plain rows
    assert picked("forward", 8192, 32, 7168, 2048) == "288x256" and picked("grad_x", 8192, 32, 4096, 7168) == "288x256"
    assert picked("forward", 8192, 0, 4096, 2048) == "256x256" and picked("grad_w", 8192, 0, 7168, 2048) == "256x256"
