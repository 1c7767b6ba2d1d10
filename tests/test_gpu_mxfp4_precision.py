"""What the MXFP4 layer keeps in fp32: the down rows up to the weighted sum over
a token's experts.

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
"""
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
