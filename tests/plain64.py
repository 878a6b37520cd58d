"""Plain binary64 forms of the norm and feed-forward operators (test-only), and the unit
roundings that their tolerances count.  Inputs are torch tensors on any device; everything is
computed in torch.float64 from the formulas in include/fp8q.h."""
import math

import torch

U = 2.0 ** -24                                   # half a step of fp32, relative
FMAX = {0: 448.0, 1: 57344.0}
HALF = {0: 2.0 ** -4, 1: 2.0 ** -3}              # half a step of e4m3 / e5m2, relative
TINY = {0: 2.0 ** -10, 1: 2.0 ** -17}            # half a step of their subnormals, absolute
FP8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


def half_step(t):
    """Half a step of a torch type, relative to the value."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step of its subnormals, absolute."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


def norm(x, w, res, eps):
    """r (as stored, in 64 bits), rstd, v."""
    r = x.double() if res is None else (x.double() + res.double()).to(x.dtype).double()
    rstd = (r.square().mean(1, keepdim=True) + eps).rsqrt()
    return r, rstd, r * rstd * w.double()


def norm_grad(r, w, rstd, dy, dres):
    """dx, dw and the magnitudes that their rounding errors scale with."""
    t, xhat = dy.double() * w.double(), r * rstd
    mean = (t * xhat).mean(1, keepdim=True)
    dx = rstd * (t - xhat * mean)
    mag = rstd * (t.abs() + xhat.abs() * (t * xhat).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        mag = mag + dres.double().abs()
    g = dy.double() * xhat
    return dx, g.sum(0), mag, g.abs().sum(0)


def check_groups(q, s, v, width, fmt, rel):
    """Codes and scales of 1 x width groups (the last one may be short) against the values v in 64
    bits that the library knows to a relative error `rel` of the group's largest (a number, or one
    per group): each code is at most half a step, and that error, away from v scaled to the
    format's maximum."""
    m, n = v.shape
    nb = -(-n // width)
    rel = torch.zeros((m, nb), dtype=torch.float64, device=v.device) + rel
    p = torch.zeros((m, nb * width), dtype=torch.float64, device=v.device)
    p[:, :n] = v
    amax = p.view(m, nb, width).abs().amax(2).clamp(min=float(torch.tensor(1e-4)))
    want = amax / FMAX[fmt]
    bad = ~((s.double().view(m, nb) - want).abs() <= (rel + 2 * U) * want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} scales off"
    z = v * (FMAX[fmt] / amax).repeat_interleave(width, 1)[:, :n]
    got = q.view(m, n).view(FP8[fmt]).double()
    tol = torch.clamp(z.abs() * HALF[fmt], min=TINY[fmt]) * (1 + 8 * U) + ((rel + 4 * U) * FMAX[fmt]).repeat_interleave(width, 1)[:, :n]
    bad = ~((got - z).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes off"


GELU = 2 * math.sqrt(2 / math.pi)


def act(g, name):
    """act(g) and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def exponent(g, name):
    """p(g) of act(g) = g * sigmoid(p(g)), and p'(g)."""
    if name == "silu":
        return g, torch.ones_like(g)
    return GELU * (g + 0.044715 * g ** 3), GELU * (1 + 3 * 0.044715 * g * g)


def spread(s, rows, k):
    """One scale per 128 x 128 block (or, for a scale per row, per 1 x 128 group) for each element."""
    s = s.double()
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :k]


def gated(a, wg, wu, name, err):
    """h in 64 bits from the operands' values, and the bound of its error when gate and up are known
    to err times the sum of their products' magnitudes: |act'| is at most 1.13, and e^-p, the
    quotient and the products take at most 16 roundings and 8 of p."""
    gate, up = a @ wg.t(), a @ wu.t()
    eg, eu = err * (a.abs() @ wg.abs().t()), err * (a.abs() @ wu.abs().t())
    v = act(gate, name)[0]
    h = v * up
    e = 1.13 * eg * (up.abs() + eu) + v.abs() * eu + (16 + 8 * exponent(gate, name)[0].abs()) * U * h.abs()
    return gate, up, h, eg, eu, e
