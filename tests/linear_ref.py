"""Plain fp64 forms of the linear layers over rows in expert order, with error bounds.

Bounds.  Products of bf16 or fp16 values are exact in fp32.  Every addition of a
sum of q of them errs by at most one step of fp32 (2 u, u = 2^-24) of a partial
sum, whatever the order and whether the unit rounds or truncates, so a sum errs
by at most 2 u (q + 8) S, S the sum of the magnitudes; eight more cover the
bias, the groups' sums and a residual.  A function's value f(z) adds the error
of z times the largest slope (1.13 for GELU, 1.1 for SiLU) and its own
evaluation: relative, a few u times 1 + |z| (2^x of a rounded argument) or
1 + z^2 (erfc of a rounded argument).  The result rounds once, by half a step
of its type or of its subnormals.
"""
import torch

U = 2.0 ** -24
SLOPE = 1.13


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(want, dtype):
    info = torch.finfo(dtype)
    return want.abs() * half_step(dtype) + info.tiny * info.eps


def cdf(z):
    """The normal distribution function; torch.special.ndtr loses its digits below -6 on the GPU."""
    return 0.5 * torch.erfc(z * -0.5 ** 0.5)


def act(z, kind):
    """fp64 act(z) without a gate."""
    if kind == "none":
        return z
    return z * (torch.sigmoid(z) if kind == "silu" else cdf(z))


def slope(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * torch.sigmoid(-z))
    return cdf(z) + z * torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5


def evaluation(z, kind):
    """Error of act(z) or act'(z) evaluated in fp32 at an exact fp32 z."""
    if kind == "none":
        return torch.zeros_like(z)
    a = z.abs()
    if kind == "silu":
        size = torch.sigmoid(z) * (1 + a)
        return (16 + 4 * a) * U * size + 2.0 ** -126 * (1 + a)
    size = cdf(z) + a * torch.exp(-0.5 * z * z)
    return (48 + 4 * z * z) * U * size * (1 + a) + 2.0 ** -126 * (1 + a)


def value(z, ez, kind):
    """act of the sums z known to ez: (value, its error before rounding)."""
    if kind == "swiglu":
        gate, up = z.chunk(2, 1)
        eg, eu = ez.chunk(2, 1)
        s = act(gate, "silu")
        es = SLOPE * eg + evaluation(gate, "silu")
        return s * up, es * (up.abs() + eu) + s.abs() * eu + 2 * U * (s * up).abs()
    return act(z, kind), SLOPE * ez + evaluation(z, kind)


def upstream(d, ed, z, kind):
    """d act'(z) for d known to ed and exact z: (value, error)."""
    if kind == "none":
        return d, ed
    if kind == "swiglu":
        gate, up = z.chunk(2, 1)
        a, b = slope(gate, "silu"), act(gate, "silu")
        ea = eb = evaluation(gate, "silu")
        dg, du = d * up * a, d * b
        eg = (ed * a.abs() + (d.abs() + ed) * ea) * up.abs() + 4 * U * dg.abs()
        eu = ed * b.abs() + (d.abs() + ed) * eb + 4 * U * du.abs()
        return torch.cat((dg, du), 1), torch.cat((eg, eu), 1)
    a = slope(z, kind)
    return d * a, ed * a.abs() + (d.abs() + ed) * evaluation(z, kind) + 4 * U * (d * a).abs()


def spans(off):
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def product(x, w, off, bias=None):
    """x w^T + bias by expert in fp64 for the valid rows: (sums, their error)."""
    n, q = off[-1], x.shape[1]
    z = torch.zeros(n, w.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(z)
    for e, a, b in spans(off):
        xe, we = x[a:b].double(), w[e].double()
        z[a:b] = xe @ we.t()
        size[a:b] = xe.abs() @ we.abs().t()
        if bias is not None:
            z[a:b] += bias[e].double()
            size[a:b] += bias[e].double().abs()
    return z, 2 * U * (q + 8) * size


def outer(dy, x, off, E):
    """dw and dbias by expert in fp64, with their errors."""
    N, K = dy.shape[1], x.shape[1]
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=x.device)
    ew, db = torch.zeros_like(dw), torch.zeros(E, N, dtype=torch.float64, device=x.device)
    eb = torch.zeros_like(db)
    for e, a, b in spans(off):
        d, xe = dy[a:b].double(), x[a:b].double()
        dw[e], ew[e] = d.t() @ xe, 2 * U * (b - a + 8) * (d.abs().t() @ xe.abs())
        db[e], eb[e] = d.sum(0), 2 * U * (b - a + 8) * d.abs().sum(0)
    return dw, ew, db, eb


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, worst "
                           f"{float((err / bound.clamp(min=1e-300)).nan_to_num(float('inf')).max())} of the bound")
