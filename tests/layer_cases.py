"""Plain 64-bit forms of the norms, the gated recurrence and the 4-bit products, and the tolerances of their tests.

Tolerances count roundings: U = 2^-24 is half a step of fp32 relative to the value, eps(t) / 2 that of the stored type.
"""
from __future__ import annotations

import torch

from attention_cases import EPS, cu, gen, offsets, randn  # noqa: F401

U = 2.0 ** -24


# ---- norms ----------------------------------------------------------------------------------------------

def norm(x, weight, eps, offset):
    """y and, per value, a size of its fp32 roundings: the sum of squares is added in at most 80 + cols / 1024 steps in a
    row (half of that reaches the root), then mean, eps, root, quotient, offset and two products."""
    cols = x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    y = x * r * (1.0 if weight is None else offset + weight)
    mag = (x * r).abs() * (1.0 if weight is None else abs(offset) + weight.abs())
    return y, mag * (40 + cols / 2048 + 9) * U


def norm_grad(x, weight, dout, dsum, eps, offset):
    cols = x.shape[-1]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    f = torch.ones(cols, dtype=torch.float64) if weight is None else offset + weight
    fmag = f.abs() if weight is None else abs(offset) + weight.abs()
    c = (f * dout * x).mean(-1, keepdim=True) * r * r
    dx = (f * dout - x * c) * r
    cmag = (fmag * dout.abs() * x.abs()).mean(-1, keepdim=True) * r * r
    mag = (fmag * dout.abs() + x.abs() * cmag) * r
    steps = 2.5 * (80 + cols / 1024) + 12  # r (to the third power) and the second sum
    if dsum is not None:
        dx, mag = dx + dsum, mag + dsum.abs()
    dw, wmag = (dout * x * r).reshape(-1, cols), (dout * x * r).abs().reshape(-1, cols)
    # dw: a block's rows in a row, its groups of lanes, then the blocks in runs
    return dx, mag * steps * U, dw.sum(0), wmag.sum(0) * (x.numel() / cols / 152 + 40 + cols / 2048 + 150) * U


def eight(y, tol, values, exps, group):
    """Whether values (float8 bits) and exponents are those of y within tol: the exponent is the smallest that fits, and a
    value is off by half an 8-bit step and tol."""
    rows, cols = y.reshape(-1, y.shape[-1]).shape
    width = group or cols
    y, tol = y.reshape(rows, -1, width), tol.reshape(rows, -1, width)
    e = exps.cpu().reshape(rows, -1).double() - 127
    unit = torch.exp2(e)[..., None]
    top, slack = y.abs().amax(-1), tol.amax(-1)
    fits = 448 * unit[..., 0] >= top - slack
    least = (224 * unit[..., 0] < top + slack) | (e == -127)
    v = values.cpu().view(torch.float8_e4m3fn).double().reshape(rows, -1, width) * unit
    half = torch.maximum(y.abs() * 2.0 ** -4, unit * 2.0 ** -10)
    near = (v - y).abs() <= half + 2 * tol + slack[..., None] * 2.0 ** -3
    return bool(fits.all()), bool(least.all()), bool(near.all())


# ---- the gated recurrence -------------------------------------------------------------------------------

def recurrence(g, x, lens, group, h0=None, dout=None, dh_last=None):
    """The rows one after another in float64, and the sizes of their errors in fp32: e = exp(g) - 1 is off by 4 U of
    itself and takes two roundings of a row; exp(g), which a run with a gate below -ln 2 uses, is off by up to 7 U of itself
    and takes one: a row adds at most 8 U of the same recurrence over magnitudes (a run's map, once for 8 rows or more, is
    off by less than those rows may be), and earlier errors pass on through the gates.  (Where e is used it is above -1/2,
    so that e h, which is rounded, is no larger than exp(g) h.)"""
    n, c = x.shape
    a = g.exp().repeat_interleave(group, 1) if group > 1 else g.exp()
    h, mag, err = (torch.zeros(n + 1, c, dtype=torch.float64) for _ in range(3))
    before = torch.zeros(n, c, dtype=torch.float64)
    berr = torch.zeros(n, c, dtype=torch.float64)
    h_last = torch.zeros(len(lens), c, dtype=torch.float64) if h0 is None else h0.clone()
    last_err = torch.zeros_like(h_last)
    cu_ = offsets(lens)
    for s in range(len(lens)):
        y, m, e = h_last[s].clone(), h_last[s].abs(), torch.zeros(c, dtype=torch.float64)
        for t in range(cu_[s], cu_[s + 1]):
            before[t], berr[t] = y, e
            y = a[t] * y + x[t]
            m = a[t] * m + x[t].abs()
            e = a[t] * e + 8 * U * m
            h[t], mag[t], err[t] = y, m, e
        h_last[s], last_err[s] = y, e
    out = {"out": (h[:n], err[:n]), "h_last": (h_last, last_err)}
    if dout is None:
        return out
    dx, xerr = torch.zeros(n, c, dtype=torch.float64), torch.zeros(n, c, dtype=torch.float64)
    dh0 = torch.zeros(len(lens), c, dtype=torch.float64) if dh_last is None else dh_last.clone()
    herr = torch.zeros_like(dh0)
    for s in range(len(lens)):
        y, m, e = dh0[s].clone(), dh0[s].abs(), torch.zeros(c, dtype=torch.float64)
        for t in range(cu_[s + 1] - 1, cu_[s] - 1, -1):
            l, lm = dout[t] + y, dout[t].abs() + m
            le = e + 4 * U * lm
            dx[t], xerr[t] = l, le
            y, m, e = a[t] * l, a[t] * lm, a[t] * (le + 8 * U * lm)
        dh0[s], herr[s] = y, e
    u = a * before
    dg = dx * u
    gerr = xerr * u.abs() + dx.abs() * (a * berr + 6 * U * u.abs()) + 2 * U * dg.abs()
    if group > 1:
        gerr = gerr.view(n, -1, group).sum(-1) + 10 * U * dg.abs().view(n, -1, group).sum(-1)
        dg = dg.view(n, -1, group).sum(-1)
    out.update(g=(dg, gerr), x=(dx, xerr), h0=(dh0, herr))
    return out


def close(got, ref, err):
    """got (fp32 or bf16, on the GPU) against ref in float64: err of fp32 roundings and one of the stored type."""
    want = err + (ref.abs() + err) * EPS[got.dtype] / 2
    off = (got.detach().cpu().double() - ref).abs()
    assert (off <= want).all(), (float((off - want).max()), float((off / want.clamp(min=1e-300)).max()))


# ---- products with 4-bit weights ------------------------------------------------------------------------

def unpack4(w, scales, offs, group):
    n = w.shape[0]
    q = torch.stack([w & 15, w >> 4], -1).reshape(n, -1, group).double() - 8
    y = q * scales.double()[..., None]
    mag = y.abs()
    if offs is not None:
        y, mag = y + offs.double()[..., None], mag + offs.double().abs()[..., None]
    return y.reshape(n, -1), mag.reshape(n, -1)


def linear4(x, w, scales, offs, group, parts):
    """y and its error: exact products; a group's sum takes 16 more products and a truncated sum per step (taken as 4 U
    of the magnitudes each), then one step per group of a warp, the scales, and eight warps."""
    y, mag = unpack4(w, scales, offs, group)
    steps = 4 * (group // 16) * parts + y.shape[1] / group / 8 + 20
    return x @ y.T, (x.abs() @ mag.T) * steps * U
