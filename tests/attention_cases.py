"""Plain 64-bit forms of the full softmax layers' operators, and the tolerances of their tests.

Tolerances count roundings.  eps(t) = finfo(t).eps; a rounding is off by at most eps / 2 of the value.
"""
from __future__ import annotations

import math

import torch

EPS = {torch.float32: torch.finfo(torch.float32).eps, torch.bfloat16: torch.finfo(torch.bfloat16).eps}


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def cu(lens, device="cuda"):
    return torch.tensor(offsets(lens), dtype=torch.int32, device=device)


def gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(seed, *shape, dtype=torch.float64, device="cpu"):
    return torch.randn(*shape, generator=gen(seed), dtype=torch.float64).to(device=device, dtype=dtype)


# ---- rotary positions -----------------------------------------------------------------------------------

def rope(x, positions, w, gain, rot, interleaved, back=False):
    """x [T, H, d] float64, w [rot / 2]: pairs turned by positions * w, times gain."""
    t = positions.double()[:, None, None] * torch.as_tensor(w, dtype=torch.float64)
    c, s = gain * t.cos(), gain * t.sin() * (-1 if back else 1)
    y = x.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ---- attention ------------------------------------------------------------------------------------------

def attention(q, k, v, q_lens, k_lens, scale=None, dout=None):
    """Causal attention in float64: out, lse and (dout given) dq, dk, dv.  Rows that see no key: 0, -inf, 0.

    Also returns, per output, a size of its rounding errors: `mag`, the same sums with every product replaced
    by its magnitude (out: sum p |v|; dq: sum p (|dp| + |D|) |k|, ...)."""
    q, k, v = q.double(), k.double(), v.double()
    Hq, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    G, scale = Hq // Hkv, (1.0 / math.sqrt(d) if scale is None else scale)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    grads = {"q": torch.zeros_like(q), "k": torch.zeros_like(k), "v": torch.zeros_like(v)}
    mag = {"out": torch.zeros_like(q), "q": torch.zeros_like(q), "k": torch.zeros_like(k), "v": torch.zeros_like(v)}
    a = b = 0
    for lq, lk in zip(q_lens, k_lens):
        see = torch.arange(lk, device=q.device)[None] <= torch.arange(lq, device=q.device)[:, None] + (lk - lq)
        for h in range(Hq):
            kv = h // G
            qq, kk, vv = q[a:a + lq, h], k[b:b + lk, kv], v[b:b + lk, kv]
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            ls = torch.logsumexp(s, 1) if lk else torch.full((lq,), -math.inf, dtype=torch.float64,
                                                                     device=q.device)
            p = torch.where(see, (s - ls[:, None]).exp(), 0.0)
            lse[a:a + lq, h] = ls
            # a masked key adds nothing, whatever its value holds
            o = torch.stack([p[i, see[i]] @ vv[see[i]] for i in range(lq)]) if lq and not vv.isfinite().all() else p @ vv
            out[a:a + lq, h] = o
            mag["out"][a:a + lq, h] = p @ vv.abs()
            if dout is None:
                continue
            do = dout[a:a + lq, h].double()
            dp = do @ vv.T
            D = (do * o).sum(1, keepdim=True)
            ds = p * (dp - D) * scale
            grads["q"][a:a + lq, h] = ds @ kk
            grads["k"][b:b + lk, kv] += ds.T @ qq
            grads["v"][b:b + lk, kv] += p.T @ do
            dm = p * ((do.abs() @ vv.abs().T) + (do.abs() * o.abs()).sum(1, keepdim=True)) * scale
            mag["q"][a:a + lq, h] = dm @ kk.abs()
            mag["k"][b:b + lk, kv] += dm.T @ qq.abs()
            mag["v"][b:b + lk, kv] += p.T @ do.abs()
        a, b = a + lq, b + lk
    return out, lse, grads, mag


# ---- cache ----------------------------------------------------------------------------------------------

def e4m3_values():
    """All finite non-negative 8-bit floats (4 exponent, 3 mantissa bits): m 2^-9, then (8 + m) 2^(e - 10)."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    norm = [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(sub + norm[:-1], dtype=torch.float64)  # the last code is NaN


def quantise(x):
    """Rows of x (last axis, finite, float64) kept as 8-bit floats times a power of two: (value, exponent byte)."""
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -127.0, dtype=torch.float64)
    for k in range(-126, 121):
        e = torch.where(top > 448.0 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
    y = (x.abs() / torch.exp2(e)[..., None]).flatten()
    vals = e4m3_values()
    hi = torch.searchsorted(vals, y).clamp(max=len(vals) - 1)
    lo = (hi - 1).clamp(min=0)
    up = vals[hi] - y
    down = y - vals[lo]
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))  # halves to the even code
    r = torch.where(take_lo, vals[lo], vals[hi]).reshape(x.shape) * x.sign()
    return r * torch.exp2(e)[..., None], (e + 127).to(torch.uint8)


def decode(q, k_rows, v_rows, scale=None):
    """q [Hq, d], k_rows, v_rows [L, Hkv, d] float64: one token's attention over L keys (0 if none)."""
    Hq, d = q.shape
    if k_rows.shape[0] == 0:
        return torch.zeros_like(q)
    G = Hq // k_rows.shape[1]
    kk, vv = k_rows.repeat_interleave(G, 1), v_rows.repeat_interleave(G, 1)
    w = torch.softmax(torch.einsum("hd,lhd->hl", q, kk) * (1.0 / math.sqrt(d) if scale is None else scale), -1)
    return torch.einsum("hl,lhd->hd", w, vv)


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    got, ref = got.detach().double().cpu(), ref.double().cpu()
    n = float(ref.norm())
    return float((got - ref).norm()) / n if n else float((got - ref).norm())
