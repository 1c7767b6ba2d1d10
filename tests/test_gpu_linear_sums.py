"""Long sums of the linear layers' gradients: the bias's over up to 2^24 rows
within a bound that does not grow with them."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import TYPES, gen, grouping, lib  # noqa: F401 (lib: the fixture)

pytestmark = pytest.mark.gpu

# dbias: eight values of a lane are added in a tree (3 roundings on a value's way), at most
# 128 such sums one after another (two of each of 64 stages), four lanes in two more; these
# sums are added in 64 bits (at most 2^18 of them: 2^-35) and rounded to fp32.  Every
# addition in between rounds to nearest: u = 2^-24 of a partial sum, which the sum of
# the magnitudes bounds.
BIAS_STEPS = 3 + 128 + 2 + 1 + 1


def bias_bound(size, want, out):
    return BIAS_STEPS * ref.U * size + ref.rounding(want, out)


def one_sign(g, rows, N, dtype):
    """A column of 0.1, one of -0.3, and columns of one value each, of either sign, the rest
    spread over an octave by row; and their sums in 64 bits."""
    dy = torch.empty(rows, N, dtype=dtype, device="cuda")
    for a in range(0, rows, 1 << 18):
        dy[a:a + (1 << 18)].uniform_(0.5, 1.5, generator=g)
    dy[:, 0], dy[:, 1] = 0.1, -0.3
    half = torch.empty(N - N // 2, device="cuda").uniform_(-2, 2, generator=g).to(dtype)
    dy[:, N // 2:] = half
    want = torch.zeros(N, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 1 << 16):
        want += dy[a:a + (1 << 16)].double().sum(0)
    return dy, want, want.abs()   # every column has one sign


# one matrix of each shape of tile, and the most rows
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,N,K", [(1 << 20, 4096, 4096), (1 << 20, 2048, 2048), ((1 << 22) - 77, 1024, 264), (1 << 24, 16, 8),
                                      (70001, 264, 264)])
def test_bias_gradient_of_one_sign(lib, rows, N, K, dtype):
    dy, want, size = one_sign(gen(rows + N), rows, N, dtype)
    x = torch.zeros(rows, K, dtype=dtype, device="cuda")
    _, db = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=torch.float32)
    ref.within(db, want, bias_bound(size, want, torch.float32), "dbias")
    before = db.clone()
    lib.moe_linear_grad_w(dy, x, dw=torch.zeros(N, K, device="cuda"), dbias=db, accumulate=True)
    ref.within(db, before.double() + want, bias_bound(size, before.double() + want, torch.float32), "added dbias")
    if dtype == torch.bfloat16:   # in the row type, whose range holds the sums
        _, db = lib.moe_linear_grad_w(dy, x, want_bias=True)
        ref.within(db, want, bias_bound(size, want, dtype), "rounded dbias")


@pytest.mark.parametrize("dtype", TYPES)
def test_bias_gradient_of_a_hot_expert(lib, dtype):
    """65536 sorted rows, two thirds of them and more on one expert."""
    T, k, E, N, K = 32768, 2, 3, 4112, 2064
    routing, off = grouping(lib, T, k, E, 3, 0.0, hot=True)
    dy, _, _ = one_sign(gen(7), T * k, N, dtype)
    x = torch.zeros(T * k, K, dtype=dtype, device="cuda")
    _, db = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, want_bias=True, dtype=torch.float32)
    want = torch.stack([dy[off[e]:off[e + 1]].double().sum(0) for e in range(E)])
    ref.within(db, want, bias_bound(want.abs(), want, torch.float32), "dbias by expert")
