"""GPU parity of the linear layers over rows in expert order and plain rows, of
their gradients and of the activation's, against plain fp64 forms and differences
of them, within the bounds of linear_ref.py."""
import pytest
import torch

import linear_ref as ref
import mxfp4_ref
from moe_inputs import random_ids

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
ACTS = ["none", "silu", "gelu", "swiglu"]


@pytest.fixture(scope="module")
def lib():
    import mixture_experts_layer_lds_amd as m
    return m


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def grouping(lib, T, k, E, seed, p_drop, hot=False, kind="bf16"):
    """A routing buffer and the experts' offsets."""
    ids = random_ids(T, k, E, seed=seed, p_drop=p_drop)
    if hot:   # two thirds of all pairs on one expert
        ids[torch.rand(T, k, generator=torch.Generator().manual_seed(seed)) < 0.67] = E // 2
    routing = lib.alloc_routing(T, k, E, 128, 128, kind)
    lib.build_routing(ids.cuda(), E, 128, 128, routing, kind)
    _, _, off = mxfp4_ref.sorted_order(ids, E)
    return routing, [int(v) for v in off]


# T, k, E, N, K, p_drop, hot
GROUPED = [
    (1, 1, 1, 16, 8, 0.0, False),
    (1, 8, 256, 512, 128, 0.1, False),
    (2, 2, 5, 32, 2056, 0.0, False),
    (5, 3, 7, 48, 40, 0.3, False),
    (64, 8, 64, 160, 264, 0.05, False),
    (33, 16, 40, 1008, 72, 0.5, False),
    (129, 5, 511, 32, 64, 1.0, False),
    (700, 2, 8, 272, 520, 0.02, False),
    (900, 4, 5, 416, 136, 0.0, True),
    (4099, 4, 16, 64, 192, 0.1, False),
    (513, 8, 8, 528, 328, 0.0, True),
]
# rows, N, K
PLAIN = [(1, 16, 8), (1, 4096, 1032), (2, 48, 7168), (15, 80, 64), (17, 144, 200), (64, 1536, 2048), (100, 1008, 1000),
         (257, 256, 256), (1000, 272, 328), (2049, 2064, 72)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,k,E,N,K,p_drop,hot", GROUPED)
def test_grouped_forward(lib, T, k, E, N, K, p_drop, hot, act, dtype):
    g = gen(T + N)
    routing, off = grouping(lib, T, k, E, T + 1, p_drop, hot)
    n, R, M = off[E], T * k, N // 2 if act == "swiglu" else N
    x, w = normal(g, R, K, dtype=dtype), normal(g, E, N, K, dtype=dtype)
    bias, res = normal(g, E, N, dtype=dtype), normal(g, R, M, dtype=dtype)
    x[n:] = float("nan")                     # rows behind the last valid one are not read
    for e in range(E):
        if off[e] == off[e + 1]:
            w[e] = float("nan")              # nor are matrices without rows
    y, z = torch.full_like(res, 7), torch.full((R, N), 7, dtype=dtype, device="cuda")
    out = lib.moe_grouped_linear(x, w, routing, k, bias=bias, act=act, residual=res, z=z, out=y)
    assert out[0] is y and out[1] is z
    assert bool((y[n:] == 7).all()) and bool((z[n:] == 7).all()), "rows behind the valid ones changed"
    want, ez = ref.product(x, w, off, bias)
    ref.within(z[:n], want, ez + ref.rounding(want, dtype), "z")
    v, ev = ref.value(want, ez, act)
    v = v + res[:n].double()
    ref.within(y[:n], v, ev + 2 * ref.U * v.abs() + ref.rounding(v, dtype), "y")
    # without bias, residual and z; the same again bit for bit
    want, ez = ref.product(x, w, off)
    v, ev = ref.value(want, ez, act)
    a = lib.moe_grouped_linear(x, w, routing, k, act=act)
    ref.within(a[:n], v, ev + ref.rounding(v, dtype), "bare y")
    assert torch.equal(a[:n], lib.moe_grouped_linear(x, w, routing, k, act=act)[:n])
    # the residual's buffer as the output
    res2 = res.clone()
    assert lib.moe_grouped_linear(x, w, routing, k, bias=bias, act=act, residual=res2, out=res2) is res2
    assert torch.equal(res2[:n], y[:n]) and torch.equal(res2[n:], res[n:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,k,E,N,K,p_drop,hot", GROUPED)
def test_grouped_grad_x(lib, T, k, E, N, K, p_drop, hot, act, dtype):
    g = gen(T + N + 1)
    routing, off = grouping(lib, T, k, E, T + 2, p_drop, hot, "fp8")
    n, R, Z = off[E], T * k, 2 * K if act == "swiglu" else K
    dy, w = normal(g, R, N, dtype=dtype), normal(g, E, N, K, dtype=dtype)
    z = 2 * normal(g, R, Z, dtype=dtype)
    dy[n:] = float("nan")
    for e in range(E):
        if off[e] == off[e + 1]:
            w[e] = float("nan")
    dx = torch.full((R, Z), 7, dtype=dtype, device="cuda")
    assert lib.moe_grouped_linear_grad_x(dy, w, routing, k, z=None if act == "none" else z, act=act, dx=dx) is dx
    assert bool((dx[n:] == 7).all())
    d, ed = ref.product(dy, w.transpose(1, 2), off)
    want, e = ref.upstream(d, ed, z[:n].double(), act)
    ref.within(dx[:n], want, e + ref.rounding(want, dtype), "dx")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,E,N,K,p_drop,hot", GROUPED)
def test_grouped_grad_w(lib, T, k, E, N, K, p_drop, hot, wide, dtype):
    g = gen(T + N + 2)
    routing, off = grouping(lib, T, k, E, T + 3, p_drop, hot, "mxfp4")
    n, R, out = off[E], T * k, torch.float32 if wide else dtype
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    dy[n:], x[n:] = float("nan"), float("nan")
    dw, db = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, want_bias=True, dtype=out)
    want, ew, wantb, eb = ref.outer(dy, x, off, E)
    ref.within(dw, want, ew + ref.rounding(want, out), "dw")
    ref.within(db, wantb, eb + ref.rounding(wantb, out), "dbias")
    assert torch.equal(dw, lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dtype=out))
    # added to what is there
    base, baseb = normal(g, E, N, K, dtype=out), normal(g, E, N, dtype=out)
    sw, sb = base.clone(), baseb.clone()
    lib.moe_grouped_linear_grad_w(dy, x, routing, k, E, dw=sw, dbias=sb, accumulate=True)
    want, wantb = want + base.double(), wantb + baseb.double()
    ref.within(sw, want, ew + 2 * ref.U * want.abs() + ref.rounding(want, out), "accumulated dw")
    ref.within(sb, wantb, eb + 2 * ref.U * wantb.abs() + ref.rounding(wantb, out), "accumulated dbias")
    for e in range(E):
        if off[e] == off[e + 1]:
            assert torch.equal(sw[e], base[e]) and not dw[e].any() and not db[e].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,N,K", PLAIN)
def test_plain_rows(lib, rows, N, K, act, dtype):
    g = gen(rows + N)
    off = [0, rows]
    M, Z = N // 2 if act == "swiglu" else N, 2 * K if act == "swiglu" else K
    x, w = normal(g, rows, K, dtype=dtype), normal(g, N, K, dtype=dtype)
    bias, res = normal(g, N, dtype=dtype), normal(g, rows, M, dtype=dtype)
    y, z = lib.moe_linear(x, w, bias=bias, act=act, residual=res, want_z=True)
    want, ez = ref.product(x, w[None], off, bias[None])
    ref.within(z, want, ez + ref.rounding(want, dtype), "z")
    v, ev = ref.value(want, ez, act)
    v = v + res.double()
    ref.within(y, v, ev + 2 * ref.U * v.abs() + ref.rounding(v, dtype), "y")
    dy, zi = normal(g, rows, N, dtype=dtype), 2 * normal(g, rows, Z, dtype=dtype)
    dx = lib.moe_linear_grad_x(dy, w, z=None if act == "none" else zi, act=act)
    d, ed = ref.product(dy, w.t()[None], off)
    want, e = ref.upstream(d, ed, zi.double(), act)
    ref.within(dx, want, e + ref.rounding(want, dtype), "dx")
    if act == "none":
        for out in (dtype, torch.float32):
            dw, db = lib.moe_linear_grad_w(dy, x, want_bias=True, dtype=out)
            want, ew, wantb, eb = ref.outer(dy, x, off, 1)
            ref.within(dw, want[0], ew[0] + ref.rounding(want[0], out), "dw")
            ref.within(db, wantb[0], eb[0] + ref.rounding(wantb[0], out), "dbias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("rows,M", [(1, 8), (3, 1000), (100, 640), (2049, 264)])
def test_act_grad(lib, rows, M, act, dtype):
    g = gen(rows + M)
    Z = 2 * M if act == "swiglu" else M
    dy, z = normal(g, rows, M, dtype=dtype), 3 * normal(g, rows, Z, dtype=dtype)
    z[0, :4] = torch.tensor([0.0, -0.0, 60.0, -30.0], dtype=dtype)
    dz = lib.moe_act_grad(dy, z, act)
    zero = torch.zeros(rows, M, dtype=torch.float64, device="cuda")
    want, e = ref.upstream(dy.double(), zero, z.double(), act)
    ref.within(dz, want, e + ref.rounding(want, dtype), "dz")
    # central differences of the forward's definition: h^2 / 6 times a third derivative below 1
    # (times the up value), and what 64 bits lose in the quotient
    h = 1e-4
    zd = z.double()
    if act == "swiglu":
        gate, up = zd.chunk(2, 1)
        diff = torch.cat(((ref.act(gate + h, "silu") - ref.act(gate - h, "silu")) / (2 * h) * up, ref.act(gate, "silu")), 1)
        scale = torch.cat((up.abs(), torch.ones_like(up)), 1) * dy.double().abs().repeat(1, 2)
        diff = diff * dy.double().repeat(1, 2)
    else:
        diff = (ref.act(zd + h, act) - ref.act(zd - h, act)) / (2 * h) * dy.double()
        scale = dy.double().abs()
    ref.within(dz, diff, e + ref.rounding(want, dtype) + scale * (h * h + (1 + z.double().abs().amax()) * 2.0 ** -52 / h), "differences")
    # grouped: the same for the valid rows, the others untouched
    T, k, E = rows, 2, 9
    routing, off = grouping(lib, T, k, E, rows, 0.3)
    dy2, z2 = dy.repeat(2, 1), z.repeat(2, 1)
    out = torch.full((2 * rows, Z), 7, dtype=dtype, device="cuda")
    assert lib.moe_grouped_act_grad(dy2, z2, routing, k, E, act, dz=out) is out
    assert torch.equal(out[:off[E]], dz.repeat(2, 1)[:off[E]]) and bool((out[off[E]:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_far_arguments(lib, dtype):
    """Activations and slopes where e^-|z| leaves fp32, at both ends of the type, and at infinity."""
    far = torch.tensor([-1e4, -300.0, -104.0, -88.0, -80.0, -20.0, -9.0, -5.0, -1.28125, 1.28125, 5.0, 9.0, 88.0, 104.0, 300.0, 1e4],
                       dtype=dtype, device="cuda")
    x = torch.zeros(16, 64, dtype=dtype, device="cuda")
    x[:, 0] = far
    w = torch.zeros(32, 64, dtype=dtype, device="cuda")
    w[:, 0] = 1
    one = torch.ones(16, 32, dtype=dtype, device="cuda")
    z = far[:, None].repeat(1, 32)
    for act in ("silu", "gelu"):
        y = lib.moe_linear(x, w, act=act)
        want, e = ref.value(z.double(), torch.zeros_like(z, dtype=torch.float64), act)
        ref.within(y, want, e + ref.rounding(want, dtype), act)
        want, e = ref.upstream(one.double(), torch.zeros_like(one, dtype=torch.float64), z.double(), act)
        ref.within(lib.moe_act_grad(one, z, act), want, e + ref.rounding(want, dtype), act + " slope")
    inf = torch.full((1, 8), float("inf"), dtype=dtype, device="cuda")
    for act in ("silu", "gelu"):
        assert bool((lib.moe_act_grad(torch.ones_like(inf), -inf, act).isnan()).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_stays_in_its_row(lib, dtype):
    g = gen(5)
    T, k, E, N, K = 300, 2, 6, 144, 200
    routing, off = grouping(lib, T, k, E, 6, 0.1)
    n, R = off[E], T * k
    x, w, dy = normal(g, R, K, dtype=dtype), normal(g, E, N, K, dtype=dtype), normal(g, R, N, dtype=dtype)
    clean = lib.moe_grouped_linear(x, w, routing, k), lib.moe_grouped_linear_grad_x(dy, w, routing, k)
    cleanw = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E)
    bad = off[2]                             # the first row of an expert: behind another's last
    x[bad, 3], dy[bad, N - 1] = float("nan"), float("inf")
    y, dx = lib.moe_grouped_linear(x, w, routing, k), lib.moe_grouped_linear_grad_x(dy, w, routing, k)
    dw = lib.moe_grouped_linear_grad_w(dy, x, routing, k, E)
    keep = torch.arange(R, device="cuda") != bad
    keep[n:] = False
    assert bool(y[bad].isnan().all()) and torch.equal(y[keep], clean[0][keep])
    assert not bool(dx[bad].isfinite().any()) and torch.equal(dx[keep], clean[1][keep])
    others = [e for e in range(E) if e != 2]
    assert torch.equal(dw[others], cleanw[others])
    assert bool(dw[2][:, 3].isnan().all()) and not bool(dw[2][N - 1].isfinite().any())
    fine = torch.ones(N, K, dtype=torch.bool, device="cuda")
    fine[:, 3], fine[N - 1] = False, False
    assert torch.equal(dw[2][fine], cleanw[2][fine])


def test_no_rows(lib):
    w = torch.ones(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    x, dy = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    routing = lib.alloc_routing(0, 2, 3, 64, 64)
    assert lib.moe_grouped_linear(x, w, routing, 2).shape == (0, 16) and lib.moe_linear(x, w[0], act="swiglu").shape == (0, 8)
    assert lib.moe_grouped_linear_grad_x(dy, w, routing, 2).shape == (0, 24)
    assert lib.moe_act_grad(dy, dy, "silu").shape == (0, 16)
    for dw, db in (lib.moe_grouped_linear_grad_w(dy, x, routing, 2, 3, want_bias=True), lib.moe_linear_grad_w(dy, x, want_bias=True)):
        assert not dw.any() and not db.any()
    kept = w.clone()
    lib.moe_grouped_linear_grad_w(dy, x, routing, 2, 3, dw=kept, accumulate=True)
    assert torch.equal(kept, w)


def test_past_32_bit_offsets(lib):
    g = gen(9)
    dtype = torch.bfloat16
    # rows past 2^32 bytes of both sides
    rows, N, K = 70000, 32, 32768
    x = torch.empty(rows, K, dtype=dtype, device="cuda").normal_(generator=g)
    w = normal(g, N, K, dtype=dtype)
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, 69000, 69999], device="cuda")
    y = lib.moe_linear(x, w)
    want, e = ref.product(x[at], w[None], [0, 8])
    ref.within(y[at], want, e + ref.rounding(want, dtype), "rows of x")
    dx = lib.moe_linear_grad_x(y, w)
    want, e = ref.product(y[at], w.t()[None], [0, 8])
    ref.within(dx[at], want, e + ref.rounding(want, dtype), "rows of dx")
    dw = lib.moe_linear_grad_w(y, x, dtype=torch.float32)
    cols = torch.tensor([0, 8, 16383, 32767], device="cuda")
    want, ew, _, _ = ref.outer(y, x[:, cols], [0, rows], 1)
    ref.within(dw[:, cols], want[0], ew[0] + ref.rounding(want[0], torch.float32), "dw over rows past 2^32 bytes")
    del x, dx
    # matrices past 2^32 bytes, the last expert's rows among them
    T, k, E, N, K = 64, 4, 40, 8192, 8192
    routing, off = grouping(lib, T, k, E, 10, 0.0)
    w = torch.empty(E, N, K, dtype=dtype, device="cuda").normal_(generator=g)
    x = normal(g, T * k, K, dtype=dtype)
    y = lib.moe_grouped_linear(x, w, routing, k)
    dx = lib.moe_grouped_linear_grad_x(x, w, routing, k)
    dw = lib.moe_grouped_linear_grad_w(x, x, routing, k, E)
    e = max(i for i in range(E) if off[i] < off[i + 1])
    a, b = off[e], off[e + 1]
    for got, m, what in ((y, w[e], "y"), (dx, w[e].t(), "dx")):
        want, bound = ref.product(x[a:b], m[None], [0, b - a])
        ref.within(got[a:b], want, bound + ref.rounding(want, dtype), what + " of the last expert")
    want, ew, _, _ = ref.outer(x[a:b], x[a:b], [0, b - a], 1)
    ref.within(dw[e], want[0], ew[0] + ref.rounding(want[0], dtype), "dw of the last expert")
    # one matrix of 2^30 values
    N, K = 16384, 65536
    w = torch.empty(N, K, dtype=dtype, device="cuda").normal_(generator=g)
    x, dy = normal(g, 3, K, dtype=dtype), normal(g, 3, N, dtype=dtype)
    y, dx = lib.moe_linear(x, w, act="swiglu"), lib.moe_linear_grad_x(dy, w)
    pick = torch.tensor([0, 5, N // 2 - 1], device="cuda")
    both = torch.cat((pick, pick + N // 2))
    z, ez = ref.product(x, w[both][None], [0, 3])
    v, ev = ref.value(z, ez, "swiglu")
    ref.within(y[:, pick], v, ev + ref.rounding(v, dtype), "y of 2^30 values")
    pick = torch.tensor([0, 5, K - 1], device="cuda")
    want, e = ref.product(dy, w[:, pick].t().contiguous()[None], [0, 3])
    ref.within(dx[:, pick], want, e + ref.rounding(want, dtype), "dx of 2^30 values")


def layer(lib, x, ids_routing, k, E, topk_w, W1, b1, W2, S1, S2, dout):
    """A layer of a program's own experts with a shared one, forward and backward: every
    tensor on the way."""
    r = ids_routing
    t = {}
    t["xs"] = lib.moe_dispatch(x, r, k, E)
    t["h"], t["z"] = lib.moe_grouped_linear(t["xs"], W1, r, k, bias=b1, act="swiglu", want_z=True)
    t["y"] = lib.moe_grouped_linear(t["h"], W2, r, k)
    t["routed"] = lib.moe_combine(t["y"], r, k, E, topk_w=topk_w)
    t["sh"], t["sz"] = lib.moe_linear(x, S1, act="gelu", want_z=True)
    t["out"] = lib.moe_linear(t["sh"], S2, residual=t["routed"])
    t["dy"], t["dw"] = lib.moe_combine_grad(dout, r, k, E, y=t["y"], topk_w=topk_w)
    t["dz"] = lib.moe_grouped_linear_grad_x(t["dy"], W2, r, k, z=t["z"], act="swiglu")
    t["dW2"] = lib.moe_grouped_linear_grad_w(t["dy"], t["h"], r, k, E, dtype=torch.float32)
    t["dxs"] = lib.moe_grouped_linear_grad_x(t["dz"], W1, r, k)
    t["dW1"], t["db1"] = lib.moe_grouped_linear_grad_w(t["dz"], t["xs"], r, k, E, want_bias=True, dtype=torch.float32)
    t["dx"] = lib.moe_dispatch_grad(t["dxs"], r, k, E)
    t["dsz"] = lib.moe_linear_grad_x(dout, S2, z=t["sz"], act="gelu")
    t["dS2"] = lib.moe_linear_grad_w(dout, t["sh"])
    t["dxsh"] = lib.moe_linear_grad_x(t["dsz"], S1)
    t["dS1"] = lib.moe_linear_grad_w(t["dsz"], x)
    return t


def layer_case(lib, seed, dtype):
    g = gen(seed)
    T, k, E, H, I, J = 203, 3, 9, 136, 72, 64
    ids = random_ids(T, k, E, seed=seed, p_drop=0.05)
    routing = lib.alloc_routing(T, k, E, 128, 128)
    lib.moe_build_routing_bf16(ids.cuda(), E, 128, 128, routing)
    pos, _, off = mxfp4_ref.sorted_order(ids, E)
    args = (normal(g, T, H, dtype=dtype), routing, k, E, torch.rand(T, k, generator=g, device="cuda"),
            normal(g, E, 2 * I, H, dtype=dtype) / 8, normal(g, E, 2 * I, dtype=dtype), normal(g, E, H, I, dtype=dtype) / 8,
            normal(g, J, H, dtype=dtype) / 8, normal(g, H, J, dtype=dtype) / 8, normal(g, T, H, dtype=dtype))
    return ids, pos, [int(v) for v in off], args


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_of_own_experts(lib, dtype):
    """Dispatch, products with SwiGLU, combine and a shared expert, and back: every step against its
    formula on the step's inputs, and the whole step against 64-bit autograd."""
    ids, pos, off, args = layer_case(lib, 31, dtype)
    x, routing, k, E, tw, W1, b1, W2, S1, S2, dout = args
    t = layer(lib, *args)
    n = off[E]
    z, ez = ref.product(t["xs"], W1, off, b1)
    h, eh = ref.value(z, ez, "swiglu")
    ref.within(t["h"][:n], h, eh + ref.rounding(h, dtype), "h")
    for got, a, m, kind, zz in (("dz", "dy", W2, "swiglu", "z"), ("dxs", "dz", W1, "none", None)):
        d, ed = ref.product(t[a], m.transpose(1, 2), off)
        want, e = ref.upstream(d, ed, t[zz][:n].double() if zz else None, kind)
        ref.within(t[got][:n], want, e + ref.rounding(want, dtype), got)
    for got, a, b in (("dW1", "dz", "xs"), ("dW2", "dy", "h")):
        want, ew, wantb, eb = ref.outer(t[a], t[b], off, E)
        ref.within(t[got], want, ew + ref.rounding(want, torch.float32), got)
        if got == "dW1":
            ref.within(t["db1"], wantb, eb + ref.rounding(wantb, torch.float32), "db1")
    s, es = ref.product(t["sh"], S2[None], [0, x.shape[0]])
    want = s + t["routed"].double()
    ref.within(t["out"], want, es + 2 * ref.U * want.abs() + ref.rounding(want, dtype), "out")

    # the whole: every stored tensor between is rounded once to the row type, at most seven in a
    # row on any path (xs is exact), each by half a step of the norm through maps of bounded gain;
    # 32 half steps cover paths that add and slopes above one
    leaves = [v.double().requires_grad_() for v in (x, tw, W1, b1, W2, S1, S2)]
    T, H = x.shape
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    rows = torch.zeros(T * k, dtype=torch.long, device="cuda")
    rows[pos.cuda()] = torch.arange(T * k, device="cuda")   # the pair of every sorted row

    def forward(xd, wd, A1, c1, A2, B1, B2):
        xs, ys = xd[token[rows]], []
        for e, a, b in ref.spans(off):
            gate, up = (xs[a:b] @ A1[e].t() + c1[e]).chunk(2, 1)
            ys.append((gate * torch.sigmoid(gate) * up) @ A2[e].t())
        y = torch.cat(ys) * wd.flatten()[rows[:n]][:, None]
        v = xd @ B1.t()
        return torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add(0, token[rows[:n]], y) + (v * ref.cdf(v)) @ B2.t()

    out = forward(*leaves)
    out.backward(dout.double())
    got = (t["dx"].double() + t["dxsh"].double(), t["dw"], t["dW1"], t["db1"], t["dW2"], t["dS1"], t["dS2"])
    out = out.detach()
    bound = 32 * ref.half_step(dtype)
    assert float((t["out"].double() - out).norm() / out.norm()) < bound
    # and central differences of the whole along a direction of each leaf, h small against the
    # leaf and large against 64 bits: h^2 times a third derivative is far below the bound
    g = gen(77)
    for name, a, leaf in zip(("x", "w", "W1", "b1", "W2", "S1", "S2"), got, leaves):
        rel = float((a.double() - leaf.grad).norm() / leaf.grad.norm())
        assert rel < bound, (name, rel)
        d = torch.randn(leaf.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        with torch.no_grad():
            ends = [float((forward(*[v + s * h * d if v is leaf else v for v in leaves]) * dout.double()).sum()) for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(float((a.double() * d).sum()) - slope) < bound * float(leaf.grad.norm() * d.norm()), name


def test_layer_in_a_graph(lib):
    """Captured on a stream of its own, replayed over new inputs between eager work."""
    dtype = torch.bfloat16
    ids, pos, off, args = layer_case(lib, 41, dtype)
    n = off[args[3]]
    first = layer(lib, *args)                      # warm-up
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        held = layer(lib, *args)
    for seed in (1, 2, 3, 4):
        g = gen(seed)
        args[0].copy_(normal(g, *args[0].shape, dtype=dtype))
        args[-1].copy_(normal(g, *args[-1].shape, dtype=dtype))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = layer(lib, *args)
        for name, v in eager.items():
            m = n if name in ("xs", "h", "z", "y", "dy", "dz", "dxs") else len(v)
            assert torch.equal(held[name][:m], v[:m]), (seed, name)


def test_two_streams_at_once(lib):
    """Two layers on two streams, each over its own routing, give what each gives alone."""
    cases = [layer_case(lib, s, torch.float16) for s in (51, 52)]
    alone = [layer(lib, *c[3]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            both.append([layer(lib, *c[3]) for _ in range(3)])
    torch.cuda.synchronize()
    for c, want, runs in zip(cases, alone, both):
        n = c[2][c[3][3]]
        for t in runs:
            for name, v in want.items():
                m = n if name in ("xs", "h", "z", "y", "dy", "dz", "dxs") else len(v)
                assert torch.equal(t[name][:m], v[:m]), name
    # a stream argument beside the current stream
    x, w = cases[0][3][0], cases[0][3][8]
    want = lib.moe_linear(x, w, act="gelu")
    torch.cuda.synchronize()
    got = lib.moe_linear(x, w, act="gelu", stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(got, want)


def test_foreign_routing_stays_in_bounds(lib):
    """A routing buffer whose ranges do not fit the rows is cut to them."""
    T, k, E, N, K = 16, 2, 4, 32, 64
    routing = lib.alloc_routing(T, k, E, 64, 64)
    lay = lib.moe_routing_layout(T, k, E, 64, 64)
    routing.zero_()
    at = lay["expert_offsets"] // 4
    routing.view(torch.int32)[at:at + E + 1] = torch.tensor([-5, 40, 20, 1 << 30, 1 << 30], dtype=torch.int32, device="cuda")
    x, w = torch.ones(T * k, K, dtype=torch.bfloat16, device="cuda"), torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda")
    big = torch.full((3, T * k, N), 7, dtype=torch.bfloat16, device="cuda")
    lib.moe_grouped_linear(x, w, routing, k, out=big[1])
    torch.cuda.synchronize()
    assert bool((big[0] == 7).all()) and bool((big[2] == 7).all()) and bool((big[1] == K).all())
    dw = lib.moe_grouped_linear_grad_w(big[1], x, routing, k, E)
    assert bool(dw.isfinite().all())


def test_refusals(lib):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: lib.moe_linear(x.cpu(), w), lambda: lib.moe_linear(x, w.half()), lambda: lib.moe_linear(x.float(), w),
                lambda: lib.moe_linear(x, w, act="tanh"), lambda: lib.moe_linear(x, w[:, :32]), lambda: lib.moe_linear(x.t(), w),
                lambda: lib.moe_linear(x, w, bias=torch.zeros(31, dtype=torch.bfloat16, device="cuda")),
                lambda: lib.moe_linear(x, w, act="swiglu", residual=torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.MoeError) as e:
        lib.moe_linear(x[:, :12].contiguous(), w[:, :12].contiguous())
    assert e.value.status == -2
