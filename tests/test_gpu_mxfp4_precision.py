"""What the MXFP4 layer keeps in fp32: the down rows up to the weighted sum over
a token's experts, and SiLU(gate) * up up to its codes, over the whole range of
gates that fp32 holds.

Tolerances:
* output, against the fp64 product of the library's own intermediate codes: the
  MFMA adds the exact products of a unit (128 values) and rounds its fp32 sum
  once a unit, at most 8 waves or slices are added, the sum over k rows rounds
  each product and each addition, and the output rounds once to bf16 (half a
  step, 2^-8):
      E = ((units + 8) 2^-23 + (k + 1) 2^-23) sum_j |w_j| sum |W2 h_j|
      |error| <= E + 2^-8 (|out| + E)
  A row rounded to bf16 before the sum is off by up to 2^-8 of itself, which the
  sum of rows of differing signs does not forgive.
* SiLU(gate) * up: seven fp32 roundings of at most 2^-23 and the rounded
  exponent's rest stay under 2^-20 of the value.  The gates and ups here are
  exact in fp32 (sums of a few powers of two), so a value 2^-19 of itself away
  from the border between two codes has to fall on its own side.
"""
import math

import pytest
import torch

import mxfp4_ref as ref
from moe_testlib import log
from test_gpu_mxfp4 import BF16, SHAPES, U23, lib, run_layer   # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,H,I,k,T,p_drop,bm", [s for s in SHAPES if s[3] > 1])
def test_rows_are_summed_in_fp32(lib, E, H, I, k, T, p_drop, bm):   # noqa: F811
    assert lib.moe_routing_layout(T, k, E, H, I, "mxfp4")["block_m"] == bm
    x, ids, w, W, _, out, routing, ws = run_layer(lib, T, k, E, H, I, E + T, p_drop)
    hc, hs, _ = ref.read_h(lib, ws, routing, T, k, E, H, I)
    hq = ref.dequantize(hc, hs)
    pos, _, off = ref.sorted_order(ids, E)
    y, mag = torch.zeros(T * k, H, dtype=torch.float64), torch.zeros(T * k, H, dtype=torch.float64)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        w2 = ref.dequantize(W[1][0][e], W[1][1][e])
        y[r], mag[r] = hq[r] @ w2.t(), hq[r].abs() @ w2.abs().t()
    wt = (w.double() * ((ids >= 0) & (ids < E))).unsqueeze(2)
    want = (y[pos].view(T, k, H) * wt).sum(1)
    sums = (I // 128 + 8 + k + 1) * U23 * (mag[pos].view(T, k, H) * wt.abs()).sum(1)
    bound = sums + BF16 * (want.abs() + sums) + 2.0 ** -133
    err = (out.cpu().double() - want).abs()
    log(f"  mxfp4 E={E} T={T}: output max err/bound {float((err / bound).max()):.2f}")
    bad = err > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs, worst {float((err / bound).max()):.1f} of the bound"


# ---- SiLU(gate) * up

def terms(v, n, low, high):
    """v (fp64 [...]) as n e2m1 values times powers of two 2^low .. 2^high, the
    largest first: (magnitude codes with sign, exponents), and their sum."""
    codes, exps, rest = [], [], v.clone()
    for _ in range(n):
        _, e = torch.frexp(rest.abs())
        e = torch.where(rest == 0, low, (e - 1).clamp(low, high))      # 2^e <= |rest| < 2^(e + 1)
        u = rest * ref.two_to(-e)
        c = torch.where(u.abs() >= 1.75, 4, torch.where(u.abs() >= 1.25, 3, torch.where(u.abs() >= 0.75, 2, 0)))   # 2, 3/2, 1, 0
        sign = torch.where(rest < 0, -1.0, 1.0)
        rest = rest - sign * ref.GRID[c] * ref.two_to(e)
        codes.append(c + 8 * (sign < 0))
        exps.append(e)
    return torch.stack(codes, -1), torch.stack(exps, -1), v - rest


def rows_of(codes, exps, H):
    """Weight rows [..., H]: one value at the first column of each 32-value block."""
    full = torch.zeros(*codes.shape[:-1], H // 32, 32, dtype=torch.uint8)
    full[..., :codes.shape[-1], 0] = codes.to(torch.uint8)
    scales = torch.full((*codes.shape[:-1], H // 32), 127, dtype=torch.uint8)
    scales[..., :exps.shape[-1]] = (exps + 127).to(torch.uint8)
    c = full.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scales


# tokens an expert: streaming on 16- and 32-row tiles, strips
@pytest.mark.parametrize("T,bm", [(1, 16), (5, 16), (12, 32), (30, 64), (50, 96), (100, 160)])
def test_silu_over_the_range_of_gates(lib, T, bm):   # noqa: F811
    """Token rows of ones at the first column of each block, so that a weight row's
    sum is its gate or up.  A block of 32 intermediate columns has one column
    that sets its scale (gate 32, whose SiLU is 32 to fp32, times up 1/8) and 31
    whose SiLU(gate) * up is 2^-19 of itself above or below a border."""
    E, H, I, k = 1, 1024, 1024, 1
    assert lib.moe_routing_layout(T, k, E, H, I, "mxfp4")["block_m"] == bm
    g = torch.Generator().manual_seed(T)
    n = I
    # gates of 20 bits, of every magnitude up to 88 and both signs; those whose SiLU is largest beside
    gate = torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * (math.log(88.0) + 9) - 9)
    gate = torch.where(torch.rand(n, generator=g) < 0.75, -gate, gate)
    gate[1::64] = -torch.linspace(70, 88, gate[1::64].numel(), dtype=torch.float64)
    _, e = torch.frexp(gate)
    step = ref.two_to(e - 20)
    gate = torch.round(gate / step) * step
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5], dtype=torch.float64)[torch.randint(6, (n,), generator=g)]
    side = torch.where(torch.rand(n, generator=g) < 0.5, 1.0, -1.0)
    up = border * (1 + side * 2.0 ** -19) / ref.silu(gate)
    _, e = torch.frexp(up)
    step = ref.two_to(e - 23)      # 23 bits: 2^-23 of itself at most
    up = torch.round(up / step) * step
    first = torch.arange(n) % 32 == 0
    gate[first], up[first] = 32.0, 1 / 8
    gc, ge, gate = terms(gate, H // 32, -60, 8)
    uc, ue, up = terms(up, H // 32, -60, 126)
    c1, s1 = rows_of(torch.cat((gc, uc)).unsqueeze(0), torch.cat((ge, ue)).unsqueeze(0), H)
    c2 = torch.zeros(E, H, I // 2, dtype=torch.uint8)
    s2 = torch.full((E, H, I // 32), 127, dtype=torch.uint8)
    exact = ref.dequantize(c1[0], s1[0])[:, 0::32].sum(1)
    assert torch.equal(exact, torch.cat((gate, up))) and torch.equal(exact, exact.float().double())
    x = torch.zeros(T, H)
    x[:, 0::32] = 1
    ids = torch.zeros(T, k, dtype=torch.int32)
    _, _, _, _, _, out, routing, ws = run_layer(lib, T, k, E, H, I, T, ids=ids, x=x, W=((c1, s1), (c2, s2)))
    assert not out.any()
    hc, hs, _ = ref.read_h(lib, ws, routing, T, k, E, H, I)
    assert (hs == 127).all()
    got = torch.stack((hc & 15, hc >> 4), -1).flatten(1).long()
    h = ref.silu(gate) * up
    away = (h.abs() / border - 1).abs()
    assert (away[~first] > 2.0 ** -20).all()
    want = ref.round_codes(h.abs()) + 8 * (h < 0)
    bad = got != want
    assert not bad.any(), f"{int(bad[0].sum())} of {n} codes, gates {gate[bad[0]][:8].tolist()}"
    assert torch.equal(hc, hc[:1].expand_as(hc))


@pytest.mark.parametrize("T", [1, 12, 50])
def test_silu_of_extreme_gates(lib, T):   # noqa: F811
    """Gates whose e^-g fp32 does not hold, or whose exponent's product with log2(e)
    it does not: SiLU is the gate itself or 0 there, never NaN."""
    E, H, I, k = 1, 128, 128, 1
    # (gate code, its exponent, up's exponent, SiLU(gate) * up)
    cases = [(3, 126, -126, 1.5), (11, 126, -126, 0.0), (2, 127, -127, 1.0), (10, 127, 126, 0.0), (3, 7, -7, 1.5), (11, 7, 60, 0.0),
             (2, 10, -9, 2.0), (10, 10, 100, 0.0), (0, 0, 100, 0.0), (2, -126, 126, 0.5), (3, 40, -39, 3.0), (2, 3, 0, 8 / (1 + math.exp(-8.0)))]
    c1 = torch.zeros(E, 2 * I, H, dtype=torch.uint8)
    s1 = torch.full((E, 2 * I, H // 32), 127, dtype=torch.uint8)
    want = torch.zeros(I, dtype=torch.float64)
    for i, (gc, ge, ue, h) in enumerate(cases):
        c1[0, i, 0], s1[0, i, 0] = gc, ge + 127
        c1[0, I + i, 0], s1[0, I + i, 0] = 2, ue + 127
        want[i] = h
    c1 = c1[..., 0::2] | (c1[..., 1::2] << 4)
    c2, s2 = torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.full((E, H, I // 32), 127, dtype=torch.uint8)
    x = torch.zeros(T, H)
    x[:, 0] = 1
    _, _, _, _, _, _, routing, ws = run_layer(lib, T, k, E, H, I, T, ids=torch.zeros(T, k, dtype=torch.int32), x=x, W=((c1, s1), (c2, s2)))
    hc, hs, _ = ref.read_h(lib, ws, routing, T, k, E, H, I)
    assert (hs[:, 0] == 127).all()       # the largest is 7.997
    got = torch.stack((hc & 15, hc >> 4), -1).flatten(1).long() & 7
    assert torch.equal(got, ref.round_codes(want).expand_as(got))


def test_down_rows_past_32_bit_offsets(lib):   # noqa: F811
    # 65536 down rows of 16640 fp32 values: 4.4 GB of them
    T, k, E, H, I = 8192, 8, 8, 16640, 128
    x, ids, w, W, _, out, routing, ws = run_layer(lib, T, k, E, H, I, 5, p_drop=0.01)
    W_ = lib.moe_workspace_layout(T, k, E, H, I, "mxfp4")
    assert W_["y"] + 4 * T * k * H <= W_["total_bytes"] and 4 * T * k * H > 1 << 32
    hc, hs, _ = ref.read_h(lib, ws[:W_["y"]], routing, T, k, E, H, I)
    pos, _, off = ref.sorted_order(ids, E)
    for p in (0, 1, 32767, 40000, int(off[E]) - 2, int(off[E]) - 1):
        t = int((pos == p).nonzero()) // k       # the token of sorted row p, with its other rows
        rows = pos.view(T, k)[t]
        want, sums = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                h, w2 = ref.dequantize(hc[rows[j]], hs[rows[j]]), ref.dequantize(W[1][0][e], W[1][1][e])
                want += w[t, j].double() * (w2 @ h)
                sums += w[t, j].double().abs() * (w2.abs() @ h.abs())
        sums = (I // 128 + 8 + k + 1) * U23 * sums
        err = (out[t].cpu().double() - want).abs()
        assert (err <= sums + BF16 * (want.abs() + sums) + 2.0 ** -133).all(), f"token {t}"
