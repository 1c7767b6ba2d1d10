"""Every tile shape of the linear layers at every number of rows that a tile of it can
have, each size held to the shape that it is meant for.  Bounds: linear_ref.py."""
import pytest
import torch

import test_gpu_linear_shapes as shapes
from linear_shapes import picked
from test_gpu_linear import TYPES, gen, lib  # noqa: F401 (lib: the fixture)

pytestmark = pytest.mark.gpu
E, R = len(shapes.RAGGED), sum(shapes.RAGGED)
#: shape: its rows, and those of a round of 16-row blocks over its waves
HEIGHTS = {"256x256": (256, 32), "128x128": (128, 32), "64x64 pair": (64, 32), "64x64 quad": (64, 32), "288x256": (288, 32)}
# the columns of the output, the values that a sum is over
ROWS = [("256x256", 1040, 264), ("256x256", 1296, 72), ("128x128", 528, 264), ("64x64 pair", 144, 520), ("64x64 quad", 48, 264),
        ("288x256", 1808, 72), ("288x256", 1808, 520), ("288x256", 5136, 264)]
GRAD_W = [("256x256", 1040, 520), ("128x128", 528, 264), ("64x64 pair", 144, 264), ("64x64 quad", 48, 72)]


def rounds(shape):
    """The rounds of blocks that RAGGED's tiles of this shape have."""
    most, step = HEIGHTS[shape]
    seen = set()
    for rows in filter(None, shapes.RAGGED):
        tiles = -(-rows // most)
        height = min(most, -(-(-(-rows // tiles)) // step) * step)
        seen |= {-(-(min(rows, m + height) - m) // step) for m in range(0, rows, height)}
    return seen


def here(op, N, K, act="none"):
    return picked(op, R, E, N, K, act, torch.cuda.get_device_properties(0).multi_processor_count)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,cols,q", ROWS)
def test_forward(lib, shape, cols, q, dtype):
    routing, off, _, _ = shapes.ragged(lib, cols)
    for act in ("none", "gelu", "swiglu"):
        assert here("forward", cols, q, act) == shape
        shapes.forward(lib, gen(cols + q), routing, 1, off, R, E, cols, q, act, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,cols,q", ROWS)
def test_gradient_of_the_rows(lib, shape, cols, q, dtype):
    routing, off, _, _ = shapes.ragged(lib, q)
    assert here("grad_x", q, cols) == shape
    for act in ("none", "silu", "swiglu"):
        shapes.grad_x(lib, gen(cols + q), routing, 1, off, R, E, q, cols, act, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,N,K", GRAD_W)
def test_gradient_of_the_matrices(lib, shape, N, K, dtype):
    routing, off, _, _ = shapes.ragged(lib, N)
    assert here("grad_w", N, K) == shape
    for out in (dtype, torch.float32):
        shapes.grad_w(lib, gen(N + K), routing, 1, off, R, E, N, K, out, dtype)
