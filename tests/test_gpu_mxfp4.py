"""GPU parity of the MXFP4 operators against the plain fp64 forms.

* Quantisation and its inverse are exact: every code and every value equal.
* The layer in two steps, so that a rounding of the intermediate that sits at
  a border of the format does not blur the check:
  - the intermediate codes: x's codes are decided on exact inputs, and the
    MFMA adds the exact products of a unit and rounds its fp32 sum once a
    unit, and at most 8 waves' sums are added, so gate and up are within
    (units + 8) * 2^-23 * sum |w x| of the fp64 values and h = silu(g) u within
    |silu'| < 1.1 times that, plus 2^-20 |h| for SiLU and its product.  Each
    code has to be the rounding of some value that close to the fp64 one.
  - the output against the fp64 product of the library's own intermediate
    codes: the down sums (at T = 1 with the weighted sum over k rows, 4 lane
    steps and 8 waves) are within (units + k + 12) * 2^-23 * sum |W2 h|, each
    stored row rounds to bf16 (2^-8 relative; not at T = 1), the weighted sum
    of k rows to fp32 and the output to bf16 (2^-8).
"""
import pytest
import torch

import mxfp4_ref as ref
from moe_inputs import make_tokens, random_ids, random_weights_w, WORKLOADS
from moe_testlib import log

pytestmark = pytest.mark.gpu

U23 = 2.0 ** -23
BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def lib():
    import mixture_experts_layer_lds_amd as m
    return m


def weights(E, rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    return ref.quantize(torch.randn(E, rows, cols, generator=g) / cols ** 0.5)


# ---- quantisation

def special_rows(dtype):
    """Rows of 64 values: ties, zeros, subnormals, the largest values, NaN and Inf."""
    tiny = torch.finfo(dtype).smallest_normal
    big = torch.finfo(dtype).max
    tie = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 5.5, 7, .5, -0.0, -.25, -5, -7, 0])
    rows = []
    for k in (0, 3, -5, 10):
        rows.append(torch.cat((tie * 2.0 ** k, torch.zeros(16), -tie * 2.0 ** -k, torch.ones(16))))
    rows.append(torch.zeros(64))
    rows.append(torch.full((64,), tiny))
    rows.append(torch.linspace(-tiny, tiny, 64))
    rows.append(torch.cat((torch.full((32,), big), torch.full((32,), -big / 2))))
    for at, bad in ((0, float("nan")), (31, float("inf")), (32, -float("inf")), (63, float("nan"))):
        r = torch.linspace(-3, 5, 64)
        r[at] = bad
        rows.append(r)
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (7, 4128), (130, 640), (1000, 2048)])
def test_quantize_is_exact(lib, dtype, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(dtype)
    codes, scales = lib.moe_quantize_mxfp4(x.cuda())
    rc, rs = ref.quantize(x)
    assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)
    back = lib.moe_dequantize_mxfp4(codes, scales, dtype)
    assert torch.equal(back.cpu().double(), ref.dequantize(rc, rs).to(dtype).double())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize_special_values(lib, dtype):
    x = special_rows(dtype)
    codes, scales = lib.moe_quantize_mxfp4(x.cuda())
    rc, rs = ref.quantize(x)
    assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)


def test_quantize_strided_rows(lib):
    x = torch.randn(37, 512, device="cuda").bfloat16()
    for part in (x[:, :96], x[:, 64:480], x[::3, 8:40]):
        codes, scales = lib.moe_quantize_mxfp4(part)
        rc, rs = ref.quantize(part.cpu())
        assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)


def test_quantize_past_32_bit_offsets(lib):
    rows, cols = 66001, 65536        # 4.3e9 values
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = lib.moe_quantize_mxfp4(x)
    back = lib.moe_dequantize_mxfp4(codes, scales)
    for r in (0, 32767, 32768, 65535, 65536, rows - 1):
        rc, rs = ref.quantize(x[r:r + 1].cpu())
        assert torch.equal(codes[r:r + 1].cpu(), rc) and torch.equal(scales[r:r + 1].cpu(), rs), r
        assert torch.equal(back[r:r + 1].cpu().double(), ref.dequantize(rc, rs)), r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_dequantize_every_code_and_scale(lib, dtype):
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(1).view(256, 1)
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 1) * 17      # every code, twice a block
    out = lib.moe_dequantize_mxfp4(codes.cuda(), scales.cuda(), dtype).cpu()
    want = ref.dequantize(codes, scales).to(dtype)   # one rounding from the exact value
    assert torch.equal(out.isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(out[ok], want[ok])


@pytest.mark.parametrize("E,rows,cols", [(3, 64, 512), (2, 32, 256), (2, 96, 640), (1, 32, 128)])
def test_pack_weights_layout(lib, E, rows, cols):
    g = torch.Generator().manual_seed(rows)
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0, 256, (E, rows, cols // 32), generator=g, dtype=torch.uint8)
    p = lib.moe_pack_weights_mxfp4(codes.cuda(), scales.cuda())
    c, s = ref.unpack_weights(p.tensor.cpu(), E, rows, cols)
    assert torch.equal(c, codes) and torch.equal(s, scales)
    again = p.clone()
    assert torch.equal(again.tensor, p.tensor)
    for f in ("dtype", "experts", "rows", "cols"):
        assert getattr(again.desc, f) == getattr(p.desc, f)


# ---- the layer

def check_layer(lib, x, ids, w, W, out, routing, ws, sizes, what):
    """The two-step check of the module's comment, rows of NaN-free tokens."""
    T, k, E, H, I = sizes
    (c1, s1), (c2, s2) = W
    xq = ref.dequantize(*ref.quantize(x.cpu().bfloat16()))
    hc, hs, R = ref.read_h(lib, ws, routing, T, k, E, H, I)
    pos, order, off = ref.sorted_order(ids.cpu(), E)
    assert torch.equal(R["pos"].long(), pos) and torch.equal(R["offsets"].long(), off)
    hq = ref.dequantize(hc, hs)
    y, ymag = torch.zeros(T * k, H, dtype=torch.float64), torch.zeros(T * k, H, dtype=torch.float64)
    worst = 0.0
    for e in range(E):
        r = torch.arange(int(off[e]), int(off[e + 1]))
        if not r.numel():
            continue
        w1, w2 = ref.dequantize(c1[e], s1[e]), ref.dequantize(c2[e], s2[e])
        xt = xq[order[r] // k]
        gu = xt @ w1.t()
        d = (H // 128 + 8) * U23 * (xt.abs() @ w1.abs().t())
        g, u = gu[:, :I], gu[:, I:]
        h = ref.silu(g) * u
        dh = 1.1 * u.abs() * d[:, :I] + ref.silu(g).abs() * d[:, I:] + 1.1 * d[:, :I] * d[:, I:] + 2.0 ** -20 * h.abs()
        # scale codes: of some amax within the bound of the fp64 one
        top = h.abs().unflatten(1, (-1, 32)).amax(2)
        dt = dh.unflatten(1, (-1, 32)).amax(2)
        lo, hi = ref.scale_exponents((top - dt).clamp(min=0).repeat_interleave(32, 1))[0], ref.scale_exponents((top + dt).repeat_interleave(32, 1))[0]
        s = hs[r].long() - 127
        assert ((s >= lo) & (s <= hi)).all(), f"{what}: scale codes of expert {e}"
        # codes: between the roundings of the bound's ends, at the library's scale
        inv = ref.two_to(-s).repeat_interleave(32, 1)
        got = torch.stack((hc[r] & 15, hc[r] >> 4), -1).flatten(1).long()
        signed = torch.where(got > 7, -(got & 7), got)

        def ends(v):
            c = ref.round_codes((v * inv).abs())
            return torch.where(v < 0, -c, c)

        bad = (signed < ends(h - dh)) | (signed > ends(h + dh))
        assert not bad.any(), f"{what}: {int(bad.sum())} codes of expert {e}"
        worst = max(worst, float((dh * inv).max()))
        y[r] = hq[r] @ w2.t()
        ymag[r] = hq[r].abs() @ w2.abs().t()
    wt = (w.cpu().double() * ((ids.cpu() >= 0) & (ids.cpu() < E))).unsqueeze(2)
    y, ymag = y[pos].view(T, k, H), ymag[pos].view(T, k, H)
    want = (y * wt).sum(1)
    dy = (I // 128 + k + 12) * U23 * ymag + (BF16 * y.abs() if T > 1 else 0.0)
    bound = ((dy + (k + 1) * U23 * y.abs()) * wt.abs()).sum(1)
    bound = bound * (1 + BF16) + BF16 * want.abs() + 2.0 ** -133
    err = (out.cpu().double() - want).abs()
    log(f"  {what}: intermediate bound {worst:.1e} steps, output max err/bound {float((err / bound).max()):.2f}")
    assert (err <= bound).all(), f"{what}: output"


def run_layer(lib, T, k, E, H, I, seed, p_drop=0.0, ids=None, x=None, W=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) if x is None else x
    ids = random_ids(T, k, E, seed=seed + 1, p_drop=p_drop) if ids is None else ids
    w = random_weights_w(T, k, seed=seed + 2)
    W = W or (weights(E, 2 * I, H, seed + 3), weights(E, H, I, seed + 4))
    P = lib.pack_weights({"w1": W[0][0].cuda(), "w1_scale": W[0][1].cuda(), "w2": W[1][0].cuda(), "w2_scale": W[1][1].cuda()},
                         "mxfp4")
    out, routing, ws = lib.moe_layer(x.cuda().bfloat16(), ids.cuda(), w.cuda(), P, dtype="mxfp4")
    torch.cuda.synchronize()
    return x, ids, w, W, P, out, routing, ws


# E, H, I, k, T, p_drop, tile rows.  Register streaming on 16- and 32-row
# tiles, strips on 64, 96, 128, 160 and 192; reductions in groups of 4, 2 and 1 units
# and every stage length of the strips (units 4, 6, 2, 5, 3, 1); H not a
# multiple of 256; down reductions in 2, 4 and 8 slices.
SHAPES = [
    (8, 512, 512, 2, 5, 0.0, 16),
    (16, 256, 384, 4, 33, 0.1, 32),
    (64, 1024, 640, 8, 60, 0.05, 16),
    (32, 256, 128, 8, 40, 0.0, 32),
    (3, 896, 128, 1, 7, 0.0, 16),
    (256, 384, 256, 8, 40, 0.02, 16),
    (8, 128, 1152, 3, 40, 0.0, 32),
    (1, 128, 128, 1, 1, 0.0, 16),
    (8, 512, 768, 2, 100, 0.0, 64),
    (8, 768, 512, 2, 130, 0.1, 64),
    (4, 640, 256, 2, 60, 0.0, 64),
    (4, 256, 640, 2, 150, 0.0, 128),
    (5, 384, 896, 3, 120, 0.2, 96),
    (4, 896, 384, 2, 160, 0.0, 128),
    (2, 1536, 768, 2, 90, 0.0, 128),
    (4, 512, 512, 2, 130, 0.0, 96),
    (4, 768, 640, 2, 220, 0.1, 160),
    (3, 1280, 768, 3, 110, 0.0, 160),
    (4, 512, 2048, 2, 130, 0.0, 96),
    (8, 384, 1024, 2, 100, 0.1, 64),
    (2, 256, 2048, 1, 300, 0.0, 192),
    (192, 1024, 640, 2, 1200, 0.0, 64),
    (4, 512, 512, 2, 300, 0.0, 192),
    (3, 768, 640, 2, 310, 0.1, 192),
    (2, 384, 1280, 1, 400, 0.0, 192),
    (1, 128, 384, 1, 260, 0.0, 192),
]


@pytest.mark.parametrize("E,H,I,k,T,p_drop,bm", SHAPES)
def test_layer_parity(lib, E, H, I, k, T, p_drop, bm):
    log(f"mxfp4 layer E={E} H={H} I={I} k={k} T={T} p_drop={p_drop}")
    assert lib.moe_routing_layout(T, k, E, H, I, "mxfp4")["block_m"] == bm
    x, ids, w, W, _, out, routing, ws = run_layer(lib, T, k, E, H, I, E + T, p_drop)
    check_layer(lib, x, ids, w, W, out, routing, ws, (T, k, E, H, I), f"E={E} T={T}")


@pytest.mark.parametrize("T,k,E,H,I", [(5000, 1, 16, 256, 128), (8192, 8, 64, 128, 256), (65536, 1, 128, 128, 128)])
def test_thousands_of_tokens(lib, T, k, E, H, I):
    # token indices over the whole range of pairs
    x, ids, w, W, _, out, routing, ws = run_layer(lib, T, k, E, H, I, 70 + k, p_drop=0.01)
    check_layer(lib, x, ids, w, W, out, routing, ws, (T, k, E, H, I), f"T={T}")


@pytest.mark.parametrize("k,E,H,I", [(1, 4, 256, 256), (16, 1, 256, 384), (8, 64, 512, 512), (16, 40, 384, 768), (5, 5, 640, 640)])
def test_one_token(lib, k, E, H, I):
    # the down launch adds the token's rows; one pair dropped, and two pairs of one expert
    ids = random_ids(1, k, E, seed=k)
    if k > 4:   # (one expert: sixteen rows of it, one dropped)
        ids[0, 1] = -1
        ids[0, 3] = ids[0, 2]
    x, ids, w, W, _, out, routing, ws = run_layer(lib, 1, k, E, H, I, 50 + k, ids=ids)
    check_layer(lib, x, ids, w, W, out, routing, ws, (1, k, E, H, I), f"one token k={k}")


@pytest.mark.parametrize("T,k,E", [(200, 2, 16), (700, 3, 8), (20, 4, 64)])
def test_one_expert_takes_every_token(lib, T, k, E):
    H, I = 256, 256
    ids = random_ids(T, k, E, seed=T)
    ids[ids == 3] = 4
    ids[:, 0] = 3
    x, ids, w, W, _, out, routing, ws = run_layer(lib, T, k, E, H, I, T, ids=ids)
    check_layer(lib, x, ids, w, W, out, routing, ws, (T, k, E, H, I), f"hot expert T={T}")


@pytest.mark.parametrize("T", [1, 30, 300])
def test_all_pairs_dropped(lib, T):
    E, H, I, k = 8, 256, 256, 2
    ids = torch.full((T, k), E, dtype=torch.int32)
    ids[::2] = -1
    *_, out, _, _ = run_layer(lib, T, k, E, H, I, T, ids=ids)
    assert not out.any()


@pytest.mark.parametrize("T,k,E", [(1, 4, 8), (24, 4, 16), (200, 2, 16), (400, 2, 4)])
def test_nan_and_inf_stay_in_their_token(lib, T, k, E):
    # a NaN or Inf of x reaches every output of its token and no other token's
    H, I = 384, 256
    g = torch.Generator().manual_seed(T)
    clean = torch.randn(T, H, generator=g)
    x = clean.clone()
    rows = sorted({0, T // 2, T - 1})
    for i, t in enumerate(rows):
        x[t, 17 + 40 * i] = float("inf") if i % 2 else float("nan")
    a = run_layer(lib, T, k, E, H, I, T, x=x)
    b = run_layer(lib, T, k, E, H, I, T, x=clean)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[rows] = True
    assert a[5].cpu()[bad].isnan().all()
    assert torch.equal(a[5].cpu()[~bad], b[5].cpu()[~bad])


@pytest.mark.parametrize("T,k,E,H,I", [(1, 8, 32, 512, 512), (7, 8, 32, 512, 640), (32, 2, 64, 256, 256), (33, 2, 64, 256, 256),
                                       (300, 4, 8, 512, 256)])
def test_route_forward_equals_the_two_calls(lib, T, k, E, H, I):
    x, ids, w, W, P, out, routing, ws = run_layer(lib, T, k, E, H, I, 7 * T, p_drop=0.1)
    r2, ws2 = torch.full_like(routing, 0xEE), torch.full_like(ws, 0xEE)
    out2 = torch.full_like(out, float("nan"))
    lib.route_forward(ids.cuda(), x.cuda().bfloat16(), w.cuda(), r2, P, ws2, out2, "mxfp4")
    torch.cuda.synchronize()
    a, b = (lib.read_routing(r, T, k, E, H, I, "mxfp4") for r in (routing, r2))   # (the bytes between the parts are not set)
    assert all(torch.equal(a[n], b[n]) for n in ("header", "offsets", "sorted", "pos", "tasks"))
    assert torch.equal(out2, out)


def test_results_do_not_depend_on_buffers_or_repeats(lib):
    # stale workspace contents (all ones: NaN scale codes and values) change nothing
    for T, k, E, H, I in ((1, 4, 16, 512, 512), (9, 4, 16, 512, 256), (100, 4, 16, 256, 512), (500, 2, 4, 512, 256)):
        x, ids, w, W, P, out, routing, ws = run_layer(lib, T, k, E, H, I, T)
        for fill in (0xFF, 0x00, 0x7F):
            ws.fill_(fill)
            again = torch.full_like(out, float("nan"))
            lib.moe_forward_mxfp4(x.cuda().bfloat16(), w.cuda(), routing, P["w1"], P["w2"], ws, again)
            assert torch.equal(again, out)


def test_graph_replays_and_another_stream(lib):
    # two graphs of differing sizes on one workspace, replayed in turn with eager
    # work between; then a call on a stream of its own
    E, H, I, k = 32, 512, 256, 4
    W = (weights(E, 2 * I, H, 1), weights(E, H, I, 2))
    P = lib.pack_weights({"w1": W[0][0].cuda(), "w1_scale": W[0][1].cuda(), "w2": W[1][0].cuda(), "w2_scale": W[1][1].cuda()},
                         "mxfp4")
    ws = lib.alloc_workspace(600, k, E, H, I, "mxfp4")
    made = []
    for T in (1, 12, 600):
        assert lib.moe_workspace_layout(T, k, E, H, I, "mxfp4")["total_bytes"] <= ws.numel()
        st = dict(T=T, x=torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"),
                  ids=torch.zeros(T, k, dtype=torch.int32, device="cuda"), w=torch.zeros(T, k, device="cuda"),
                  routing=lib.alloc_routing(T, k, E, H, I, "mxfp4"),
                  out=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))

        def step(st=st, out=None, stream=None):
            lib.route_forward(st["ids"], st["x"], st["w"], st["routing"], P, ws, st["out"] if out is None else out, "mxfp4", stream)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        made.append((st, step, g))
    for rep in range(3):
        for st, step, g in made:
            T = st["T"]
            st["x"].copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(rep + T)))
            st["ids"].copy_(random_ids(T, k, E, seed=rep + T, p_drop=0.1))
            st["w"].copy_(random_weights_w(T, k, seed=rep + T))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            got = st["out"].clone()
            eager = torch.empty_like(got)
            step(out=eager)
            torch.cuda.synchronize()
            assert torch.equal(got, eager), f"replay {rep} T={T}"
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            other = torch.empty_like(got)
            step(out=other, stream=side)
            side.synchronize()
            assert torch.equal(got, other)


def test_dsv3_shape(lib):
    # the DeepSeek-V3-shaped layer at full width, 24 of its experts: decode, a
    # small batch and strips
    wl = WORKLOADS["dsv3"]
    E, H, I, k = 24, wl.H, wl.I, wl.k
    W = (weights(E, 2 * I, H, 8), weights(E, H, I, 9))
    for T in (1, 6, 80):
        x, _, _ = make_tokens(wl, T)
        x, ids, w, _, _, out, routing, ws = run_layer(lib, T, k, E, H, I, 90 + T, x=x.float(), W=W)
        check_layer(lib, x, ids, w, W, out, routing, ws, (T, k, E, H, I), f"dsv3 width T={T}")
