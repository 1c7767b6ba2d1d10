"""The row passes on the paths that other sizes leave out: quantisers of four
runs a wave whose last workgroup is partly filled, also over strided rows, and
gradients on sixteen waves a token for every pair count.  Tolerances: exact,
and those of test_gpu_rows.py (the bound there of a dw's additions, columns a
lane on one wave and 13, covers sixteen waves: a sixteenth of the columns a
lane, 6 exchanges and 15 additions over the waves)."""
import math

import pytest
import torch

import mxfp4_ref as ref
from test_gpu_rows import TYPES, U, case, dots, half_step, lib, to_tokens, within   # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("strided", [False, True])
def test_quantisers_with_a_remainder(lib, dtype, strided):   # noqa: F811
    rows, cols = 4099, 544
    vectors = rows * cols * torch.finfo(dtype).bits // 8 // 16
    assert vectors >= 1 << 18 and vectors % 1024 % 64     # four runs a wave; a partly filled wave in the last workgroup
    g = torch.Generator().manual_seed(cols)
    wide = (torch.randn(rows, cols + 96, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(dtype)
    x = wide[:, 64:64 + cols]
    given = wide.cuda()[:, 64:64 + cols] if strided else x.contiguous().cuda()
    assert given.is_contiguous() != strided
    mark_c, mark_s = torch.full((rows + 1, cols // 2), 0xEE, dtype=torch.uint8), torch.full((rows + 1, cols // 32), 0xEE, dtype=torch.uint8)
    codes, scales = mark_c.cuda(), mark_s.cuda()
    lib.moe_quantize_mxfp4(given, codes[:rows], scales[:rows])
    rc, rs = ref.quantize(x)
    assert torch.equal(codes[:rows].cpu(), rc) and torch.equal(scales[:rows].cpu(), rs)
    back = torch.full((rows + 1, cols), 7.0, dtype=dtype, device="cuda")
    lib.moe_dequantize_mxfp4(codes[:rows], scales[:rows], out=back[:rows])
    assert torch.equal(back[:rows].cpu().double(), ref.dequantize(rc, rs).to(dtype).double())
    # what lies behind the rows is left as it was
    assert bool((codes[rows] == 0xEE).all()) and bool((scales[rows] == 0xEE).all()) and bool((back[rows] == 7).all())


# rows of eight 1 KiB runs and more, up to 512 tokens: sixteen waves a token, for 2, 4, 8 and 16 pairs
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,p_drop", [(130, 2, 8, 4096, 0.1), (300, 3, 9, 7168, 0.2), (61, 6, 61, 4104, 0.05),
                                            (37, 16, 40, 4104, 0.3), (512, 1, 4, 4096, 0.0), (513, 5, 16, 4160, 0.1)])
def test_gradients_of_long_rows(lib, T, k, E, H, p_drop, dtype):   # noqa: F811
    ids, w, routing, pos, n, valid, x, y = case(lib, T, k, E, H, dtype, T + k, p_drop)
    steps = math.ceil(H / 512) * 8 + 13
    wantw, magw = dots(y, x, pos, valid, T, k)
    dx, dw = lib.moe_dispatch_grad(y.cuda(), routing, k, E, x=x.cuda(), topk_w=w.cuda())
    want, mag = to_tokens(y, pos, valid, w.double(), T, k)
    within(dx, want, (k + 1) * U * mag + half_step(dtype) * want.abs() + 2.0 ** -25, "dx")
    within(dw, wantw, steps * U * magw, "dispatch dw")
    assert not dw.cpu().flatten()[~valid].any()
    mark = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    dy, dv = lib.moe_combine_grad(x.cuda(), routing, k, E, y=y.cuda(), topk_w=w.cuda(), dy=mark)
    assert bool((dy[n:] == 7).all())
    want = torch.zeros(T * k, H, dtype=torch.float64)
    want[pos] = x.double().repeat_interleave(k, 0) * w.double().flatten().unsqueeze(1)
    within(dy[:n], want[:n], want[:n].abs() * (U + half_step(dtype)) + 2.0 ** -25, "dy")
    within(dv, wantw, steps * U * magw, "combine dw")
    assert not dv.cpu().flatten()[~valid].any()
