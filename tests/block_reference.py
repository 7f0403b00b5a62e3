"""The transformer block's operators from their formulas in 64 bits, with bounds on how far a correct
kernel's results may be: fp32 sums (a relative error of 2^-24 per addition, times the sum of the terms'
magnitudes) and one rounding, at most finfo(dtype).eps / 2 of the value, to the I/O type."""
from __future__ import annotations

import math

import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def layer_norm(x, weight, bias, eps, add):
    """(y, h, stats), and the bounds of y and stats."""
    td, C = x.dtype, x.shape[1]
    h = x if add is None else (x.float() + add.float()).to(td)
    hd = h.double()
    mean = hd.mean(1, keepdim=True)
    d = hd - mean
    var = d.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    w = torch.ones(C, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    y = d * r * w + b
    # a thread adds at most 64 values, then a tree and the warps' sums: 80 additions; rstd is off by
    # half the variance's relative error (80 additions of squares, and the mean's error squared)
    e_mean = 80 * F32 * hd.abs().mean(1, keepdim=True)
    e_r = (0.5 * (84 * F32 * var + e_mean.square()) / (var + eps) + 6 * F32)
    ey = w.abs() * r * (e_mean + d.abs() * (e_r + 4 * F32)) + 2 * F32 * (b.abs() + y.abs()) + \
        half_step(td) * y.abs()
    stats = torch.stack([mean[:, 0], r[:, 0]])
    return (y, h, stats), (ey, torch.stack([e_mean[:, 0] + 2 * F32 * mean[:, 0].abs(), (e_r * r)[:, 0]]))


def layer_norm_backward(h, weight, stats, dy, add):
    """(dx, dw, db) with the given stats, and their bounds."""
    td, (rows, C) = h.dtype, h.shape
    mean, r = stats.double()[0][:, None], stats.double()[1][:, None]
    w = torch.ones(C, dtype=torch.float64, device=h.device) if weight is None else weight.double()
    d = dy.double()
    xh = (h.double() - mean) * r
    g = d * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    e = F32 * r * (8 * g.abs() + 90 * g.abs().mean(1, keepdim=True) +
                   xh.abs() * 100 * (g * xh).abs().mean(1, keepdim=True))
    if add is not None:
        dx = dx + add.double()
        e = e + 2 * F32 * dx.abs()
    e = e + half_step(td) * dx.abs()
    depth = rows + 80  # additions of a column's sum, in whatever grouping
    return (dx, (d * xh).sum(0), d.sum(0)), (e, depth * F32 * (d * xh).abs().sum(0),
                                             depth * F32 * d.abs().sum(0))


def rotary(x, dims, axes, first, start, step, base, interleaved, backward):
    F, Hp, Wp = dims
    rows, _, dh = x.shape
    n = first + torch.arange(rows, device=x.device)
    idx = (n // (Hp * Wp), n // Wp % Hp, n % Wp)
    ang = []
    for a in range(3):
        pos = start[a] + step[a] * idx[a].double()
        j = torch.arange(axes[a] // 2, device=x.device, dtype=torch.float64)
        ang.append(pos[:, None] * base ** (-2.0 * j / max(axes[a], 1)))
    ang = torch.cat(ang, 1) * (-1.0 if backward else 1.0)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    R, xd, out = sum(axes), x.double(), x.double().clone()
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    out[..., lo] = xd[..., lo] * c - xd[..., hi] * s
    out[..., hi] = xd[..., lo] * s + xd[..., hi] * c
    # the fp32 angle (pi 2^-25), sine and cosine (2 units), two products and a sum
    e = torch.zeros_like(out)
    e[..., lo] = e[..., hi] = 12 * F32 * (xd[..., lo].abs() + xd[..., hi].abs())
    e[..., :R] += half_step(x.dtype) * out[..., :R].abs()
    return out, e


def act(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.erfc(-g / math.sqrt(2.0))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _hidden(x, wg, wu, name, u):
    """h and the parts a backward needs, with the error of g and u (C products summed in fp32; the
    activations and their derivatives change by at most 1.13 and 1 per unit of g)."""
    C = x.shape[1]
    g, up = x @ wg, x @ wu
    eg, eu = (C + 8) * F32 * (x.abs() @ wg.abs()), (C + 8) * F32 * (x.abs() @ wu.abs())
    a, da = act(g, name)
    # relative error of the exponentials at |g| up to about 20 (bf16: approximate ones, of 2^-22 of their
    # argument's magnitude), reciprocals and erfc
    e_fn = 2.0 ** -17 if u > 1e-5 else 2.0 ** -20
    ea, eda = 1.13 * eg + e_fn * (a.abs() + 1e-3), eg + e_fn * (da.abs() + 1e-3)
    h = a * up
    eh = ea * up.abs() + a.abs() * eu + u * h.abs()
    return g, up, a, da, h, eu, ea, eda, eh


def gated_ffn(x, wg, wu, wd, name, add):
    u = half_step(x.dtype)
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    *_, h, _, _, _, eh = _hidden(x, wg, wu, name, u)
    y = h @ wd
    e = eh @ wd.abs() + (wd.shape[0] + 8) * F32 * (h.abs() @ wd.abs())
    if add is not None:
        y = y + add.double()
    return y, e + (u + 2 * F32) * y.abs()


def gated_ffn_backward(x, wg, wu, wd, dy, name):
    u = half_step(x.dtype)
    N, C = x.shape
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    g, up, a, da, h, eu, ea, eda, eh = _hidden(x, wg, wu, name, u)
    dh = dy @ wd.t()
    edh = (C + 8) * F32 * (dy.abs() @ wd.abs().t())
    dg, du = dh * up * da, dh * a
    edg = edh * (up * da).abs() + dh.abs() * (eu * da.abs() + up.abs() * eda) + (u + 4 * F32) * dg.abs()
    edu = edh * a.abs() + dh.abs() * ea + (u + 2 * F32) * du.abs()
    K = (2 * wg.shape[1] + 8) * F32
    dx = dg @ wg.t() + du @ wu.t()
    edx = edg @ wg.abs().t() + edu @ wu.abs().t() + K * (dg.abs() @ wg.abs().t() + du.abs() @ wu.abs().t())
    out, err = [dx], [edx + u * dx.abs()]
    T = (N + 80) * F32
    for A, B, eA, eB in ((x, dg, None, edg), (x, du, None, edu), (h, dy, eh, None)):
        r = A.t() @ B
        e = T * (A.abs().t() @ B.abs()) + u * r.abs()
        e = e + (A.abs().t() @ eB if eA is None else eA.t() @ B.abs())
        out.append(r)
        err.append(e)
    return out, err


def check(name, got, ref, bound):
    """got within bound of ref, element by element; where ref is not finite, the same value."""
    got, ref, bound = got.double(), ref.double(), bound.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{name}: finiteness differs"
    over = (got - ref).abs()[fin] - bound[fin] - 1e-30
    assert over.numel() == 0 or over.max().item() <= 0, \
        f"{name}: {over.max().item():.3e} over the bound (largest |ref| {ref[fin].abs().max().item():.3g})"
