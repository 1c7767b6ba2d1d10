"""GPU parity of the expert-order row operators (moe_dispatch, moe_combine and
their gradients) and of the router's gradient against plain fp64 forms, and a
training step through all of them against torch's fp64 autograd.

Tolerances: products and sums run in fp32 and a result rounds once to its row
type, so with u = 2^-24 (half a step of fp32) and eps / 2 of the row type
  rows to experts   |w x| (u + eps / 2)
  rows to tokens    (k + 1) u sum_j |w y| + eps / 2 |out|
  dw                (n + 13) u sum |x y|, n = ceil(H / 512 / waves) * 8 columns a
                    lane and 13 further additions over lanes and waves
"""
import math

import pytest
import torch

import mxfp4_ref as ref
from moe_inputs import random_ids, random_weights_w, router_logits
from moe_testlib import log

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def lib():
    import mixture_experts_layer_lds_amd as m
    return m


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def case(lib, T, k, E, H, dtype, seed, p_drop, kind="bf16"):
    g = torch.Generator().manual_seed(seed)
    ids = random_ids(T, k, E, seed=seed + 1, p_drop=p_drop)
    w = torch.randn(T, k, generator=g)
    # a dropped pair's weight is never used
    w[(ids < 0) | (ids >= E)] = float("nan")
    routing = lib.alloc_routing(T, k, E, 128, 128, kind)
    lib.build_routing(ids.cuda(), E, 128, 128, routing, kind)
    pos, order, off = ref.sorted_order(ids, E)
    n = int(off[E])
    x = torch.randn(T, H, generator=g).to(dtype)
    y = torch.randn(T * k, H, generator=g).to(dtype)
    y[n:] = float("nan")         # rows behind the last valid one are not read
    valid = ((ids >= 0) & (ids < E)).flatten()
    return ids, w, routing, pos, n, valid, x, y


def within(got, want, bound, what):
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((err / bound.clamp(min=1e-300)).max())} of the bound"


def to_tokens(rows, pos, valid, w, T, k):
    take = torch.where(valid.unsqueeze(1), rows.double()[pos], 0.0).view(T, k, -1)
    ww = torch.where(valid.view(T, k), w, 0.0).unsqueeze(2)
    return (take * ww).sum(1), (take.abs() * ww.abs()).sum(1)


def dots(rows, tokens, pos, valid, T, k):
    r = torch.where(valid.unsqueeze(1), rows.double()[pos], 0.0).view(T, k, -1)
    t = tokens.double().unsqueeze(1)
    return (r * t).sum(2), (r * t).abs().sum(2)


# T, k, E, H, p_drop
SHAPES = [
    (1, 1, 1, 8, 0.0),
    (1, 8, 256, 7168, 0.1),
    (5, 3, 7, 40, 0.3),
    (64, 8, 64, 520, 0.05),
    (33, 16, 40, 1000, 0.5),
    (700, 2, 8, 2056, 0.02),
    (129, 5, 511, 512, 1.0),
    (4099, 4, 16, 64, 0.1),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,p_drop", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_and_combine(lib, T, k, E, H, p_drop, dtype, weighted):
    ids, w, routing, pos, n, valid, x, y = case(lib, T, k, E, H, dtype, T + k, p_drop)
    dw = w.cuda() if weighted else None
    wd = w.double() if weighted else torch.ones(T, k, dtype=torch.float64)
    mark = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    xs = lib.moe_dispatch(x.cuda(), routing, k, E, topk_w=dw, out=mark)
    assert xs is mark and bool((xs[n:] == 7).all()), "rows behind the valid ones changed"
    want = torch.zeros(T * k, H, dtype=torch.float64)
    want[pos] = x.double().repeat_interleave(k, 0) * wd.flatten().unsqueeze(1)
    if weighted:
        within(xs[:n], want[:n], want[:n].abs() * (U + half_step(dtype)) + 2.0 ** -25, "dispatch")
    else:
        assert torch.equal(xs[:n].cpu().double(), want[:n])
    out = lib.moe_combine(y.cuda(), routing, k, E, topk_w=dw)
    want, mag = to_tokens(y, pos, valid, wd, T, k)
    within(out, want, (k + 1) * U * mag + half_step(dtype) * want.abs() + 2.0 ** -25, "combine")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,p_drop", SHAPES)
def test_gradients(lib, T, k, E, H, p_drop, dtype):
    ids, w, routing, pos, n, valid, x, y = case(lib, T, k, E, H, dtype, T + k + 1, p_drop)
    steps = math.ceil(H / 512) * 8 + 13
    # dispatch: dx and dw from dxs (y) and x
    dx, dw = lib.moe_dispatch_grad(y.cuda(), routing, k, E, x=x.cuda(), topk_w=w.cuda())
    want, mag = to_tokens(y, pos, valid, w.double(), T, k)
    within(dx, want, (k + 1) * U * mag + half_step(dtype) * want.abs() + 2.0 ** -25, "dx")
    wantw, magw = dots(y, x, pos, valid, T, k)
    within(dw, wantw, steps * U * magw, "dispatch dw")
    assert not dw.cpu().flatten()[~valid].any()
    # without the weights' gradient: the sum alone
    alone = lib.moe_dispatch_grad(y.cuda(), routing, k, E, topk_w=w.cuda())
    within(alone, want, (k + 1) * U * mag + half_step(dtype) * want.abs() + 2.0 ** -25, "dx alone")
    # combine: dy and dw from dout (x) and y
    mark = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    dy, dw = lib.moe_combine_grad(x.cuda(), routing, k, E, y=y.cuda(), topk_w=w.cuda(), dy=mark)
    assert bool((dy[n:] == 7).all())
    want = torch.zeros(T * k, H, dtype=torch.float64)
    want[pos] = x.double().repeat_interleave(k, 0) * w.double().flatten().unsqueeze(1)
    within(dy[:n], want[:n], want[:n].abs() * (U + half_step(dtype)) + 2.0 ** -25, "dy")
    within(dw, wantw, steps * U * magw, "combine dw")
    assert torch.equal(lib.moe_combine_grad(x.cuda(), routing, k, E, topk_w=w.cuda())[:n], dy[:n])


def test_past_32_bit_offsets(lib):
    # the largest count of pairs on the widest rows: 2^32 values of sorted rows
    T, k, E, H = 4096, 16, 40, 65536
    ids = random_ids(T, k, E, seed=3, p_drop=0.01)
    w = torch.randn(T, k)
    routing = lib.alloc_routing(T, k, E, 128, 128, "bf16")
    lib.build_routing(ids.cuda(), E, 128, 128, routing, "bf16")
    pos, _, off = ref.sorted_order(ids, E)
    n, valid = int(off[E]), ((ids >= 0) & (ids < E))
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    xs = lib.moe_dispatch(x, routing, k, E, topk_w=w.cuda())
    dx, dw = lib.moe_dispatch_grad(xs, routing, k, E, x=x, topk_w=w.cuda())
    out = lib.moe_combine(xs, routing, k, E)
    dy, dv = lib.moe_combine_grad(x, routing, k, E, y=xs, topk_w=w.cuda())
    u = half_step(torch.bfloat16)
    order = torch.argsort(pos)
    for r in (0, 1, 32767, 32768, 65535 - (T * k - n), n // 2, n - 1):
        p = int(order[r])
        want = x[p // k].cpu().double() * w.double().flatten()[p]
        within(xs[r], want, want.abs() * (U + u) + 2.0 ** -133, f"dispatch row {r}")
        assert torch.equal(dy[r], xs[r]), f"combine gradient row {r}"
    for t in (0, 2047, 2048, T - 1):
        ok = valid[t]
        rows = xs[pos.view(T, k)[t].clamp(max=n - 1).cuda()].cpu().double() * ok.unsqueeze(1)
        ww = w[t].double().unsqueeze(1) * ok.unsqueeze(1)
        for got, f, what in ((dx[t], ww, "dispatch gradient"), (out[t], torch.ones_like(ww), "combine")):
            want, mag = (rows * f).sum(0), (rows * f).abs().sum(0)
            within(got, want, (k + 1) * U * mag + u * want.abs() + 2.0 ** -133, f"{what} of token {t}")
        prod = rows * x[t].cpu().double()
        for got in (dw[t], dv[t]):   # four waves or more: H / 512 / 4 * 8 columns a lane
            within(got, prod.sum(1), (H // 256 + 13) * U * prod.abs().sum(1), f"weight gradient of token {t}")


def test_gradients_against_differences(lib):
    # fp32 rows: a step of one input along a direction changes <out, r> by the gradient's product with it
    T, k, E, H = 19, 4, 12, 264
    ids, w, routing, pos, n, valid, x, y = case(lib, T, k, E, H, torch.float32, 3, 0.2)
    w = torch.nan_to_num(w)
    g = torch.Generator().manual_seed(9)
    r = torch.randn(T, H, generator=g)
    y[n:] = 0
    dy, dw = lib.moe_combine_grad(r.cuda(), routing, k, E, y=y.cuda(), topk_w=w.cuda(), dy=torch.zeros(T * k, H, device="cuda"))

    def value(yy, ww):
        return float((lib.moe_combine(yy.cuda(), routing, k, E, topk_w=ww.cuda()).cpu().double() * r.double()).sum())

    # combine is linear in y and in w, so the difference over a whole step is the
    # gradient but for rounding: (k + 2) u of every |w y r| on either side
    size = float((to_tokens(y, pos, valid, w.double(), T, k)[1] * r.double().abs()).sum())
    step = torch.randn(T * k, H, generator=g)
    got = value(y + step, w) - value(y, w)
    big = float((to_tokens(y + step, pos, valid, w.double(), T, k)[1] * r.double().abs()).sum())
    assert abs(got - float((dy.cpu().double() * step.double()).sum())) <= 2 * (k + 2) * U * (size + big)
    step = torch.randn(T, k, generator=g)
    got = value(y, w + step) - value(y, w)
    big = float((to_tokens(y, pos, valid, (w + step).double(), T, k)[1] * r.double().abs()).sum())
    assert abs(got - float((dw.cpu().double() * step.double()).sum())) <= 2 * (H + k + 2) * U * (size + big)


def test_any_dtypes_routing_serves(lib):
    # the order does not depend on the tile height that a dtype's build cuts
    T, k, E, H = 50, 4, 9, 256
    outs = []
    for kind in ("bf16", "fp8", "mxfp4", "int4"):
        *_, routing, pos, n, valid, x, y = case(lib, T, k, E, H, torch.bfloat16, 5, 0.1, kind)
        outs.append(lib.moe_dispatch(x.cuda(), routing, k, E, out=torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")))
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_repeats_streams_and_graphs(lib):
    T, k, E, H = 257, 6, 32, 1032
    ids, w, routing, pos, n, valid, x, y = case(lib, T, k, E, H, torch.bfloat16, 11, 0.1)
    x, y, w = x.cuda(), y.cuda(), w.cuda()
    y[n:] = 0
    out, dy = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(T, k, device="cuda")

    def step(stream=None):
        lib.moe_combine(y, routing, k, E, topk_w=w, out=out, stream=stream)
        lib.moe_combine_grad(x, routing, k, E, y=y, topk_w=w, dy=dy, dtopk_w=dw, stream=stream)

    step()
    first = [t.clone() for t in (out, dy, dw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        for t in (out, dy, dw):
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(dy[:n], first[1][:n]) and torch.equal(dw, first[2])
        # other inputs in the same buffers
        y.mul_(-1)
        first[0], first[2] = -first[0], -first[2]
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(dw, first[2])
    s.wait_stream(torch.cuda.current_stream())
    out.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    s.synchronize()
    assert torch.equal(out, first[0])


# ---- the router's gradient

def router_ref(logits, ids, dw, renorm):
    """fp64: the derivative of sum dw w of a softmax top-k choice; NaN scores as -infinity."""
    l = torch.where(logits.isnan(), -math.inf, logits.double())
    chosen = torch.zeros_like(l, dtype=torch.bool).scatter_(1, ids.long(), True)
    up = torch.zeros_like(l).scatter_(1, ids.long(), dw.double())
    p = torch.softmax(l.masked_fill(~chosen, -math.inf) if renorm else l, 1)
    return p * (up - (p * up).sum(1, keepdim=True)), p, up


@pytest.mark.parametrize("T,E,k,n_shared", [(1, 1, 1, 0), (3, 8, 8, 0), (5, 17, 3, 2), (64, 64, 8, 0), (257, 130, 4, 1), (1000, 256, 16, 0)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kind", ["normal", "ties", "const", "nan"])
def test_router_gradient(lib, T, E, k, n_shared, renorm, kind):
    logits = router_logits(T, E, seed=T + E, kind=kind)
    if kind == "nan":    # at least k scores are left to choose
        logits[:, :k] = torch.nan_to_num(logits[:, :k], nan=0.25)
    ids, w = lib.moe_router_topk(logits.cuda(), k, renormalize=renorm, n_shared=n_shared)
    g = torch.Generator().manual_seed(T)
    dw = torch.randn(T, k + n_shared, generator=g)
    got = lib.moe_router_topk_grad(logits.cuda(), ids, w, dw.cuda(), renormalize=renorm, n_shared=n_shared)
    want, p, up = router_ref(logits, ids[:, :k].cpu(), dw[:, :k], renorm)
    # w and p are within 16 u + 2e-6 relative (the bound of the forward's weights, held here for
    # both), and s sums k products: every term of the difference carries that, and a few u more
    rel = 2e-6 + (16 + k) * U
    mag = p * (up.abs() + 2 * (p * up.abs()).sum(1, keepdim=True))
    within(got, want, rel * 2 * mag + 1e-37, f"router gradient {kind}")


def test_router_gradient_against_differences(lib):
    # the fp64 rule that the kernel is held to, against central differences of the weights in fp64
    T, E, k = 4, 12, 3
    logits = router_logits(T, E, seed=2).double()
    ids = torch.topk(logits, k, dim=1).indices
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    for renorm in (True, False):
        def value(l):
            p = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1).gather(1, ids)
            return (p * dw).sum()

        want, _, _ = router_ref(logits, ids, dw, renorm)
        h = 1e-5
        for t in range(T):
            for e in range(E):
                d = torch.zeros_like(logits)
                d[t, e] = h
                diff = (value(logits + d) - value(logits - d)) / (2 * h)
                assert abs(diff - want[t, e]) <= 1e-9   # h^2 of third derivatives below 1, and 1e-16 / h


# ---- all of them together

def test_training_step_matches_autograd(lib):
    """Router top-k -> dispatch -> experts (a plain fp32 matrix each) -> combine, and back to the
    inputs and the router scores, against torch's fp64 autograd of the same step."""
    T, k, E, H = 96, 4, 8, 64
    g = torch.Generator().manual_seed(21)
    x = torch.randn(T, H, generator=g)
    logits = torch.randn(T, E, generator=g)
    A = torch.randn(E, H, H, generator=g) / H ** 0.5
    r = torch.randn(T, H, generator=g)

    xd, ld, Ad = x.double().requires_grad_(), logits.double().requires_grad_(), A.double().requires_grad_()
    top, idd = torch.topk(ld, k, dim=1)
    wd = torch.softmax(top, 1)
    yd = torch.tanh(torch.einsum("th,tkgh->tkg", xd, Ad[idd]))
    (wd.unsqueeze(2) * yd).sum(1).backward(r.double())

    lg = logits.cuda()
    ids, w = lib.moe_router_topk(lg, k)
    routing = lib.alloc_routing(T, k, E, H, H)
    lib.build_routing(ids, E, H, H, routing)
    xs = lib.moe_dispatch(x.cuda(), routing, k, E)
    off = lib.read_routing(routing, T, k, E, H, H)["offsets"].tolist()
    Ac = A.cuda()
    y = torch.empty_like(xs)
    for e in range(E):
        y[off[e]:off[e + 1]] = torch.tanh(xs[off[e]:off[e + 1]] @ Ac[e].t())
    out = lib.moe_combine(y, routing, k, E, topk_w=w)
    dy, dw = lib.moe_combine_grad(r.cuda(), routing, k, E, y=y, topk_w=w)
    dz = dy * (1 - y * y)
    dxs, dA = torch.empty_like(xs), torch.empty_like(Ac)
    for e in range(E):
        dxs[off[e]:off[e + 1]] = dz[off[e]:off[e + 1]] @ Ac[e]
        dA[e] = dz[off[e]:off[e + 1]].t() @ xs[off[e]:off[e + 1]]
    dx = lib.moe_dispatch_grad(dxs, routing, k, E)
    dl = lib.moe_router_topk_grad(lg, ids, w, dw)
    # a chain of fp32 sums of at most H + k + T/2 terms of size about 1 each
    for name, a, b in (("out", out, (wd.unsqueeze(2) * yd).sum(1).detach()), ("dx", dx, xd.grad), ("dA", dA, Ad.grad),
                       ("dlogits", dl, ld.grad)):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        log(f"  {name} rel {rel:.1e}")
        assert rel <= (H + k + T) * U, name
