"""Plain fp64 forms of the MXFP4 layer and of the expert-order row operators
(torch on the CPU, no code of the library), and readers of the library's
MXFP4 buffers.  tests/test_mxfp4_ref.py pins them."""
from __future__ import annotations

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def two_to(e):
    """2^e in fp64, exact, for whole e of [-1022, 1023]."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def scale_exponents(v):
    """Shared exponent s of every 32-value block of v [..., cols] (fp64), and
    whether the block holds Inf or NaN."""
    top = v.unflatten(-1, (-1, 32)).abs().amax(-1)
    bad = ~torch.isfinite(v.unflatten(-1, (-1, 32))).all(-1)
    _, e = torch.frexp(torch.where(bad, 1.0, top))
    return torch.where(top > 0, (e - 3).clamp(min=-127), -127), bad


def round_codes(a):
    """e2m1 magnitude codes of a >= 0: the nearest of GRID, a tie to the even
    code, at most 6."""
    border = (GRID[1:] + GRID[:-1]) / 2
    low, high = torch.bucketize(a, border), torch.bucketize(a, border, right=True)
    return torch.where(low % 2 == 0, low, high)


def quantize(v):
    """(codes uint8 [..., cols / 2], scale codes uint8 [..., cols / 32]) of v."""
    v = v.double()
    s, bad = scale_exponents(v)
    u = v.unflatten(-1, (-1, 32)) * two_to(-s).unsqueeze(-1)
    u = torch.where(bad.unsqueeze(-1), 0.0, u)
    c = round_codes(u.abs()) + 8 * torch.signbit(u).long()
    c = c.flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.where(bad, 255, s + 127).to(torch.uint8)


def dequantize(codes, scales):
    """fp64 values [..., cols]."""
    both = torch.cat((GRID, -GRID))
    v = torch.stack((both[(codes & 15).long()], both[(codes >> 4).long()]), -1).flatten(-2)
    s = torch.where(scales == 255, float("nan"), two_to(scales.int() - 127))
    return v * s.repeat_interleave(32, -1)


def silu(g):
    return g / (1 + torch.exp(-g))


def sorted_order(ids, E):
    """(pos [P], order [P], offsets [E + 1]) of the stable expert order: pair
    p at sorted row pos[p], dropped pairs behind the valid ones."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel())
    return pos, order, torch.searchsorted(key[order], torch.arange(E + 1))


# ---- the library's buffers

def group_of(K):
    units = K // 128
    return 4 if units % 4 == 0 else 2 if units % 2 == 0 else 1


def read_blocks(raw, n, K):
    """(codes [n, 16, K / 2], scale codes [n, 16, K / 32]) of n blocks of 16
    rows x K values: groups of G units, each G KiB of 1 KiB chunks (16-byte
    piece 16 kb + row) and 64 G scale codes (code G (16 kb + row) + unit)."""
    units, G = K // 128, group_of(K)
    raw = raw[:n * units * 1088].view(n, units // G, G * 1088)
    c = raw[..., :G * 1024].reshape(n, units // G, G, 4, 16, 16).permute(0, 4, 1, 2, 3, 5)   # n, row, group, u, kb, byte
    s = raw[..., G * 1024:].reshape(n, units // G, 4, 16, G).permute(0, 3, 1, 4, 2)          # n, row, group, u, kb
    return c.reshape(n, 16, K // 2), s.reshape(n, 16, K // 32)


def unpack_weights(packed, E, rows, K):
    """Row-major (codes, scales) of a packed weight tensor: row 4 g + i of
    16-row block b is row 32 (b / 2) + 8 g + 4 (b % 2) + i."""
    c, s = read_blocks(packed.flatten(), E * rows // 16, K)

    def rows_of(t):
        t = t.view(E, rows // 32, 2, 4, 4, t.shape[-1])             # expert, 32-row group, block, g, i
        return t.permute(0, 1, 3, 2, 4, 5).reshape(E, rows, t.shape[-1])

    return rows_of(c), rows_of(s)


def read_h(lib, ws, routing, T, k, E, H, I):
    """(codes [P, I / 2], scale codes [P, I / 32]) of the intermediate, sorted
    rows; rows behind the valid ones are zero."""
    W = lib.moe_workspace_layout(T, k, E, H, I, "mxfp4")
    R = lib.read_routing(routing, T, k, E, H, I, "mxfp4")
    mb = R["block_m"] // 16
    n = R["layout"]["max_tasks"] * mb
    c, s = read_blocks(ws.cpu()[W["h"]:], n, I)
    c, s = c.reshape(n * 16, -1), s.reshape(n * 16, -1)
    codes, scales = torch.zeros(T * k, I // 2, dtype=torch.uint8), torch.zeros(T * k, I // 32, dtype=torch.uint8)
    for ti, (_, begin, rows, _) in enumerate(R["tasks"].tolist()):
        codes[begin:begin + rows] = c[ti * mb * 16:ti * mb * 16 + rows]
        scales[begin:begin + rows] = s[ti * mb * 16:ti * mb * 16 + rows]
    return codes, scales, R
