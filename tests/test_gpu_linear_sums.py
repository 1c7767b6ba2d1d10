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


def ternary(g, rows, cols, dtype):
    """-1, 0 or 1: every partial sum of products over at most 2^24 rows is a whole number that fp32
    holds, so that sums are exact in any order and one row left out or taken twice is seen."""
    v = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for a in range(0, rows, 1 << 16):
        v[a:a + (1 << 16)] = torch.randint(-1, 2, v[a:a + (1 << 16)].shape, generator=g, device="cuda", dtype=torch.int8)
    return v


def whole_sums(dy, x, first, last):
    """dw and dbias over the rows [first, last) in 64 bits."""
    N, K = dy.shape[1], x.shape[1]
    dw, db = torch.zeros(N, K, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // max(N, K))
    for a in range(first, last, step):
        d, xe = dy[a:min(last, a + step)].double(), x[a:min(last, a + step)].double()
        dw += d.t().contiguous() @ xe
        db += d.sum(0)
    return dw, db


def rounded_once(want, dtype):
    """Whole numbers within fp32: the one rounding of the exact sum."""
    return want.float().to(dtype)


# `far`: the first row that a mistake would lose (an offset past 2^32 bytes, the end of many rows)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,N,K,far", [
    (1 << 24, 16, 8, (1 << 24) - 1),                       # the most rows; the last one of them
    ((1 << 24) - 33, 136, 136, (1 << 32) // 272),          # both operands past 2^32 bytes
    (70000, 32, 32768, 1 << 16),                           # x is
    (70000, 32768, 32, 1 << 16),                           # dy is
    (1 << 20, 2048, 2056, (1 << 32) // 4112),              # larger tiles
])
def test_every_row_counts(lib, rows, N, K, far, dtype):
    g = gen(rows + K)
    dy, x = ternary(g, rows, N, dtype), ternary(g, rows, K, dtype)
    dy[far:, 0], x[far:, 0] = 1, 1                         # what is checked below: the far rows add up
    near, nearb = whole_sums(dy, x, 0, far)
    rest, restb = whole_sums(dy, x, far, rows)
    assert float(rest[0, 0]) == rows - far and float(restb[0]) == rows - far
    want, wantb = near + rest, nearb + restb
    dw, db = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=torch.float32)
    assert torch.equal(dw.double(), want) and torch.equal(db.double(), wantb)
    assert not torch.equal(dw.double(), near) and not torch.equal(db.double(), nearb)
    assert torch.equal(lib.moe_linear_grad_w(dy, x, dtype=torch.float32), dw)
    if float(want.abs().max()) < torch.finfo(dtype).max:
        assert torch.equal(lib.moe_linear_grad_w(dy, x), rounded_once(want, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K", [(16, 34000), (34000, 16), (2064, 264)])
def test_every_sorted_row_counts(lib, N, K, dtype):
    """65536 rows of a few experts, the last ones' past 2^32 bytes."""
    T, k, E = 32768, 2, 5
    routing, off = grouping(lib, T, k, E, 4, 0.001, hot=True)
    g = gen(N)
    dy, x = ternary(g, T * k, N, dtype), ternary(g, T * k, K, dtype)
    n = off[E]
    dy[n:], x[n:] = float("nan"), float("nan")             # rows behind the last valid one take no part
    if max(N, K) == 34000:
        assert (n - 1) * 68000 > 1 << 32 and off[E - 1] < n
    dw, db = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, want_bias=True, dtype=torch.float32)
    for e in range(E):
        want, wantb = whole_sums(dy, x, off[e], off[e + 1])
        assert torch.equal(dw[e].double(), want) and torch.equal(db[e].double(), wantb), e
    base = torch.randint(-4, 5, dw.shape, generator=g, device="cuda").float()   # whole numbers too
    held = base.clone()
    lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dw=held, accumulate=True)
    assert torch.equal(held, base + dw)


@pytest.mark.parametrize("dtype", TYPES)
def test_accumulation_in_a_graph(lib, dtype):
    """Gradients added to what dw and dbias hold, captured and replayed over new rows between
    eager work: whole numbers, so that every replay's sums are exact."""
    T, k, E, N, K = 1500, 2, 7, 272, 136
    routing, off = grouping(lib, T, k, E, 6, 0.05, hot=True)
    dy, x = torch.empty(T * k, N, dtype=dtype, device="cuda"), torch.empty(T * k, K, dtype=dtype, device="cuda")
    dw, db = torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, device="cuda")
    dy.zero_(), x.zero_()
    call = lambda: lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dw=dw, dbias=db, accumulate=True)
    call()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        call()
    want, wantb = torch.zeros(E, N, K, dtype=torch.float64, device="cuda"), torch.zeros(E, N, dtype=torch.float64, device="cuda")
    for seed in range(4):
        g = gen(seed)
        dy.copy_(ternary(g, T * k, N, dtype)), x.copy_(ternary(g, T * k, K, dtype))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for e in range(E):
            a, b = whole_sums(dy, x, off[e], off[e + 1])
            want[e] += a
            wantb[e] += b
        assert torch.equal(dw.double(), want) and torch.equal(db.double(), wantb), seed


def test_bias_gradient_keeps_nan_in_its_column(lib):
    """An Inf or NaN of dy over several folds of the sum, in the gradient of its own bias alone."""
    dtype, rows, N, K = torch.bfloat16, 70001, 264, 264
    g = gen(8)
    dy, x = ternary(g, rows, N, dtype), torch.zeros(rows, K, dtype=dtype, device="cuda")
    _, clean = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=torch.float32)
    dy[5, 3], dy[rows - 1, 200], dy[40000, 100], dy[7, 100] = float("nan"), float("inf"), float("inf"), float("-inf")
    _, db = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=torch.float32)
    assert bool(db[3].isnan()) and float(db[200]) == float("inf") and bool(db[100].isnan())
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[3, 100, 200]] = False
    assert torch.equal(db[keep], clean[keep])
