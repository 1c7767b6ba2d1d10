"""The linear layers at sizes that reach every tile shape and row count of the
kernels: experts with none to several tiles of rows and every partial height
between, hot experts on the path of few rows, products of few and of many
tiles, and outputs that are stored past the caches.  Bounds: linear_ref.py."""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import ACTS, TYPES, gen, grouping, lib, normal  # noqa: F401 (lib: the fixture)

pytestmark = pytest.mark.gpu
#: rows by expert: every height of a partial tile, one row to several tiles, none in between
RAGGED = [1, 16, 17, 32, 33, 0, 64, 65, 96, 97, 128, 129, 160, 161, 192, 193, 224, 0, 225, 256, 257, 320, 385, 512, 513, 770,
          288, 289, 576, 577, 600, 500]


def ragged(lib, seed):
    """Routing of one pair a token onto RAGGED, in mixed order."""
    E = len(RAGGED)
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor(RAGGED))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(seed))].to(torch.int32).view(-1, 1)
    routing = lib.alloc_routing(len(ids), 1, E, 128, 128)
    lib.moe_build_routing_bf16(ids.cuda(), E, 128, 128, routing)
    off = [0]
    for n in RAGGED:
        off.append(off[-1] + n)
    return routing, off, len(ids), E


def forward(lib, g, routing, k, off, R, E, N, K, act, dtype):
    x, w, bias = normal(g, R, K, dtype=dtype), normal(g, E, N, K, dtype=dtype), normal(g, E, N, dtype=dtype)
    M = N // 2 if act == "swiglu" else N
    res = normal(g, R, M, dtype=dtype)
    y, z = lib.moe_grouped_linear(x, w, routing, k, bias=bias, act=act, residual=res, want_z=True)
    want, ez = ref.product(x, w, off, bias)
    n = off[E]
    ref.within(z[:n], want, ez + ref.rounding(want, dtype), "z")
    v, ev = ref.value(want, ez, act)
    v = v + res[:n].double()
    ref.within(y[:n], v, ev + 2 * ref.U * v.abs() + ref.rounding(v, dtype), "y")


def grad_x(lib, g, routing, k, off, R, E, N, K, act, dtype):
    Z = 2 * K if act == "swiglu" else K
    dy, w, z = normal(g, R, N, dtype=dtype), normal(g, E, N, K, dtype=dtype), 2 * normal(g, R, Z, dtype=dtype)
    dx = lib.moe_grouped_linear_grad_x(dy, w, routing, k, z=None if act == "none" else z, act=act)
    n = off[E]
    d, ed = ref.product(dy, w.transpose(1, 2), off)
    want, e = ref.upstream(d, ed, z[:n].double(), act)
    ref.within(dx[:n], want, e + ref.rounding(want, dtype), "dx")


def grad_w(lib, g, routing, k, off, R, E, N, K, out, dtype):
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    dw, db = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, want_bias=True, dtype=out)
    want, ew, wantb, eb = ref.outer(dy, x, off, E)
    ref.within(dw, want, ew + ref.rounding(want, out), "dw")
    ref.within(db, wantb, eb + ref.rounding(wantb, out), "dbias")
    assert torch.equal(dw, lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dtype=out))
    lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dw=dw, accumulate=True)   # twice the sums
    ref.within(dw, 2 * want, 2 * ew + ref.rounding(want, out) + 4 * ref.U * want.abs() + ref.rounding(2 * want, out), "dw added")


# wide and narrow: the largest tiles, and small ones, for the product and for its gradient
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K", [(4112, 264), (2816, 264), (272, 136), (528, 1032)])
def test_every_height(lib, N, K, dtype):
    routing, off, R, E = ragged(lib, N)
    for act in ACTS:
        forward(lib, gen(N), routing, 1, off, R, E, N, K, act, dtype)
        grad_x(lib, gen(K), routing, 1, off, R, E, K if act == "none" else N, N if act == "none" else K, act, dtype)
    grad_x(lib, gen(K), routing, 1, off, R, E, K, N, "swiglu", dtype)
    for out in (dtype, torch.float32):
        grad_w(lib, gen(N + 1), routing, 1, off, R, E, N, K, out, dtype)


# T, k, E, N, K, drop, hot
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,N,K,p_drop,hot", [
    (3000, 2, 6, 4112, 1048, 0.02, False),
    (1600, 4, 24, 2064, 1048, 0.0, True),
    (100, 8, 40, 272, 264, 0.0, False),      # about 20 rows an expert
    (300, 2, 60, 1040, 136, 0.05, True),     # few rows an expert, hundreds of one
    (40, 2, 70, 2064, 72, 0.0, True),
    (64, 4, 64, 4112, 72, 0.0, False),       # four rows an expert, many columns
    (2048, 2, 16, 2816, 264, 0.0, False),    # 256 rows an expert, more or less
    (2048, 2, 16, 272, 2816, 0.0, False),
])
def test_many_tiles(lib, T, k, E, N, K, p_drop, hot, dtype):
    routing, off = grouping(lib, T, k, E, T, p_drop, hot)
    for act in ("none", "swiglu"):
        forward(lib, gen(T), routing, k, off, T * k, E, N, K, act, dtype)
        grad_x(lib, gen(T), routing, k, off, T * k, E, N, K, act, dtype)
    grad_w(lib, gen(T), routing, k, off, T * k, E, N, K, torch.float32, dtype)


@pytest.mark.parametrize("rows,N,K", [(8200, 4104, 264), (4100, 520, 1032), (520, 2064, 2056), (9000, 1032, 520), (40, 4112, 1048), (33, 272, 72)])
def test_plain_products(lib, rows, N, K):
    dtype, off = torch.bfloat16, [0, rows]
    g = gen(rows)
    x, w, dy = normal(g, rows, K), normal(g, N, K), normal(g, rows, N)
    for act in ("none", "gelu"):
        want, ez = ref.product(x, w[None], off)
        v, ev = ref.value(want, ez, act)
        ref.within(lib.moe_linear(x, w, act=act), v, ev + ref.rounding(v, dtype), "y")
    want, e = ref.product(dy, w.t()[None], off)
    ref.within(lib.moe_linear_grad_x(dy, w), want, e + ref.rounding(want, dtype), "dx")
    for out in (dtype, torch.float32):
        dw, db = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=out)
        want, ew, wantb, eb = ref.outer(dy, x, off, 1)
        ref.within(dw, want[0], ew[0] + ref.rounding(want[0], out), "dw")
        ref.within(db, wantb[0], eb[0] + ref.rounding(wantb[0], out), "dbias")


def test_outputs_past_the_caches(lib):
    """More than 256 MiB read and written: stored with another instruction."""
    dtype = torch.bfloat16
    T, k, E, N, K = 1500, 4, 16, 4112, 2064
    routing, off = grouping(lib, T, k, E, 8, 0.01)
    for act in ACTS:
        grad_x(lib, gen(3), routing, k, off, T * k, E, N, K, act, dtype)
    grad_w(lib, gen(4), routing, k, off, T * k, E, N, K, torch.float32, dtype)
    grad_w(lib, gen(5), routing, k, off, T * k, E, N, K, dtype, dtype)


def test_most_rows(lib):
    """2^24 plain rows, and 65536 sorted ones of 511 experts."""
    dtype, rows = torch.bfloat16, 1 << 24
    g = gen(6)
    x, w = normal(g, rows, 8), normal(g, 16, 8)
    y = lib.moe_linear(x, w, act="swiglu")
    at = torch.tensor([0, 1, 4095, rows // 2, rows - 65, rows - 1], device="cuda")
    want, ez = ref.product(x[at], w[None], [0, len(at)])
    v, ev = ref.value(want, ez, "swiglu")
    ref.within(y[at], v, ev + ref.rounding(v, dtype), "y")
    dx = lib.moe_linear_grad_x(y, w[:8].contiguous())
    want, e = ref.product(y[at], w[:8].t()[None], [0, len(at)])
    ref.within(dx[at], want, e + ref.rounding(want, dtype), "dx")
    dw, db = lib.moe_linear_grad_w(y, x, want_bias=True, dtype=torch.float32)
    want, ew, wantb, eb = ref.outer(y, x, [0, rows], 1)
    ref.within(dw, want[0], ew[0] + ref.rounding(want[0], torch.float32), "dw")
    ref.within(db, wantb[0], eb[0] + ref.rounding(wantb[0], torch.float32), "dbias")
    with pytest.raises(lib.MoeError) as err:
        lib.moe_act_grad(torch.empty(rows + 1, 8, dtype=dtype, device="cuda"), torch.empty(rows + 1, 8, dtype=dtype, device="cuda"), "silu")
    assert err.value.status == -2
    T, k, E, N, K = 4096, 16, 511, 136, 72
    routing, off = grouping(lib, T, k, E, 9, 0.01)
    forward(lib, gen(7), routing, k, off, T * k, E, N, K, "gelu", dtype)
    grad_x(lib, gen(8), routing, k, off, T * k, E, N, K, "silu", dtype)
    grad_w(lib, gen(9), routing, k, off, T * k, E, N, K, dtype, dtype)


def test_back_to_back_calls(lib):
    """Calls of different shapes one after another on one stream, none waited for: each result is
    that of the call alone."""
    dtype = torch.bfloat16
    cases = []
    for rows, N, K in ((1, 4096, 1032), (300, 528, 264), (40, 4112, 1048), (2000, 2064, 520), (17, 144, 200)):
        g = gen(rows)
        cases.append((normal(g, rows, K), normal(g, N, K), normal(g, rows, N)))
    run = lambda x, w, dy: (lib.moe_linear(x, w, act="swiglu"), lib.moe_linear_grad_x(dy, w), lib.moe_linear_grad_w(dy, x, dtype=torch.float32))
    alone = []
    for c in cases:
        alone.append(run(*c))
        torch.cuda.synchronize()
    for _ in range(3):
        together = [run(*c) for c in cases]
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
