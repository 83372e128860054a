"""Operators around the mixing layers of a linearised backbone, as cases that can be timed.

The gated linear recurrence (packed sequences, its gradients, one token per sequence), the root-mean-square norm with
the residual's addition (outputs in the layer's type or in 8 bits with exponents, its gradients), and products of a few
tokens with frozen weights kept in 4 bits.  `run` computes a case in elementary torch operations, or, where `own` is
true, by the calls a user makes of linearized_attention_rope_gb300.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---- the cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 sequences: the state of every channel takes one token
        dict(name="recurrence_step", op="step", tokens=64, channels=4096, gate_dim=1, dtype="bf16", gates="f32"),
        # a batch of short prompts packed together, one gate per head: launch latency and ragged ends
        dict(name="recurrence_short", op="recurrence", lens="5,64,1,130,33,0,200,77", channels=512, gate_dim=64,
             dtype="bf16", gates="f32", carried=False, gradient=False),
        # one long prompt on few channels: the work is spread over time
        dict(name="recurrence_long", op="recurrence", lens="131071", channels=1024, gate_dim=1, dtype="bf16",
             gates="bf16", carried=True, gradient=False),
        # training on a ragged pack of a 4096 wide layer, a gate per channel
        dict(name="recurrence_train", op="recurrence", lens="1024,2999,4096,8190", channels=4096, gate_dim=1,
             dtype="bf16", gates="f32", carried=False, gradient=True),
        # the fp32 layer that numerics are checked on, with its gradients, a gate per head
        dict(name="recurrence_f32", op="recurrence", lens="4096,301", channels=1024, gate_dim=128, dtype="f32",
             gates="f32", carried=True, gradient=True),
        # one decode step's rows into 8 bits for the projections behind them
        dict(name="norm_tokens", op="norm", tokens=64, heads=1, cols=4096, dtype="bf16", out="e4m3", group=32,
             residual=True, gradient=False),
        # a long prompt's rows with the residual stream, 5120 wide
        dict(name="norm_prompt", op="norm", tokens=32767, heads=1, cols=5120, dtype="bf16", out="bf16", group=0,
             residual=True, gradient=False),
        # the gradient of the norm of every query head, behind a packed batch
        dict(name="norm_heads", op="norm", tokens=8193, heads=64, cols=128, dtype="bf16", out="bf16", group=0,
             residual=False, gradient=True),
        # the gradient of a 4096 wide fp32 norm with what the residual stream brings
        dict(name="norm_gradient", op="norm", tokens=4097, heads=1, cols=4096, dtype="f32", out="f32", group=0,
             residual=True, gradient=True),
        # one token through a square projection
        dict(name="linear4_token", op="linear4", tokens=1, n_in=4096, n_out=4096, group=128, dtype="bf16", x="bf16",
             x_group=0, offsets=False),
        # a small batch's 8-bit rows through the widest projection, weights with offsets
        dict(name="linear4_batch", op="linear4", tokens=16, n_in=8192, n_out=28672, group=128, dtype="bf16",
             x="e4m3", x_group=32, offsets=True),
        # a full batch's rows, odd in number, through a 5120 wide layer's projection
        dict(name="linear4_wide", op="linear4", tokens=61, n_in=5120, n_out=10240, group=64, dtype="bf16", x="bf16",
             x_group=0, offsets=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(values):
    return ",".join(str(int(v)) for v in values)


def draw(rng):
    op = rng.choice(["step", "recurrence", "recurrence", "norm", "norm", "linear4", "linear4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("step", "recurrence"):
        gate_dim = rng.choice([1, 1, 64, 128])
        channels = _spread(rng, 1, 8192) if gate_dim == 1 else gate_dim * _spread(rng, 1, 64)
        gates = rng.choice(["f32", "bf16"])
        if op == "step":
            return dict(op=op, tokens=_spread(rng, 1, 1024), channels=channels, gate_dim=gate_dim, dtype=dtype,
                        gates=gates)
        n = _spread(rng, 1, 12)
        total = _spread(rng, 16, min(131072, 35000000 // channels))
        lens = [max(0, int(total / n * rng.uniform(0.0, 1.4))) for _ in range(n)]
        lens[rng.randrange(n)] += 1
        return dict(op=op, lens=_text(lens), channels=channels, gate_dim=gate_dim, dtype=dtype, gates=gates,
                    carried=rng.random() < 0.5, gradient=rng.random() < 0.5)
    if op == "norm":
        heads = rng.choice([1, 1, 1, 8, 32, 64])
        cols = rng.choice([64, 128, 256]) if heads > 1 else rng.choice([_spread(rng, 8, 16384),
                                                                       128 * _spread(rng, 1, 128)])
        out = dtype if cols % 128 else rng.choice([dtype, dtype, "e4m3"])
        tokens = _spread(rng, 1, min(65536, 80000000 // (heads * cols)))
        gradient = rng.random() < 0.4
        if gradient:
            out = dtype
        return dict(op=op, tokens=tokens, heads=heads, cols=cols, dtype=dtype, out=out,
                    group=rng.choice([0, 32, 128]) if out == "e4m3" else 0,
                    residual=heads == 1 and rng.random() < 0.7, gradient=gradient)
    group = rng.choice([32, 64, 128])
    x = rng.choice([dtype, dtype, "e4m3"])
    n_in = 128 * _spread(rng, 1, 112)
    return dict(op=op, tokens=_spread(rng, 1, 64), n_in=n_in, n_out=_spread(rng, 1, min(28672, 60000000 // n_in)),
                group=group, dtype=dtype, x=x, x_group=rng.choice([0, 32, 128]) if x == "e4m3" else 0,
                offsets=rng.random() < 0.5)


def _numbers(text):
    return [int(x) for x in text.split(",")]


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _exponents(cols, group):
    return -(-cols // group) if group else 1


def work(case):
    op, b = case["op"], SIZES[case["dtype"]]
    if op in ("step", "recurrence"):
        rows = case["tokens"] if op == "step" else sum(_numbers(case["lens"]))
        seqs = rows if op == "step" else len(_numbers(case["lens"]))
        x = rows * case["channels"] * b
        g = rows * (case["channels"] // case["gate_dim"]) * SIZES[case["gates"]]
        h = seqs * case["channels"] * 4
        if op == "step":  # gates, inputs, states in; states, outputs out
            return {"bytes": g + 2 * x + 2 * h, "flops": 3 * rows * case["channels"]}
        if case["gradient"]:  # g, x, dout, dh_last in; out, h_last, dg, dx out
            return {"bytes": 2 * g + 4 * x + 2 * h + (2 * h if case["carried"] else 0),
                    "flops": 10 * rows * case["channels"]}
        return {"bytes": g + 2 * x + h + (h if case["carried"] else 0), "flops": 3 * rows * case["channels"]}
    if op == "norm":
        n, c = case["tokens"] * case["heads"], case["cols"]
        if case["gradient"]:  # the rows, dout (and the residual stream's gradient) in; dx and dweight out
            return {"bytes": n * c * b * (4 if case["residual"] else 3) + c * (b + 4), "flops": 8 * n * c}
        kept = c * SIZES[case["out"]] + (_exponents(c, case["group"]) if case["out"] == "e4m3" else 0)
        return {"bytes": n * c * b * (3 if case["residual"] else 1) + n * kept + c * b, "flops": 5 * n * c}
    m, k, n = case["tokens"], case["n_in"], case["n_out"]
    weights = n * k // 2 + n * (k // case["group"]) * b * (2 if case["offsets"] else 1)
    x = m * k * SIZES[case["x"]] + (m * _exponents(k, case["x_group"]) if case["x"] == "e4m3" else 0)
    return {"bytes": weights + x + m * n * b, "flops": 2 * m * n * k}


# ---- inputs ---------------------------------------------------------------------------------------------

class _Source:
    """Seeded tensors."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def nibbles(self, *shape):
        """Bytes of two 4-bit numbers each, gathered around the middle as rounded weights are."""
        def half():
            return (self.normal(*shape) * 2.5 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
        return half() | (half() << 4)

    def gates(self, n, width):
        """Logarithms of gates: every channel has a rate of its own, with memories of a few to a thousand tokens."""
        rate = torch.exp(torch.rand(width, generator=self.g, device="cuda") * 6.0 - 7.0)
        return -rate * torch.nn.functional.softplus(self.normal(n, width))


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    src = _Source(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = {"case": case}
    if op in ("step", "recurrence"):
        lens = [1] * case["tokens"] if op == "step" else _numbers(case["lens"])
        n, c = sum(lens), case["channels"]
        s["g"] = src.gates(n, c // case["gate_dim"]).to(TYPES[case["gates"]])
        s["x"] = src.normal(n, c).to(dt)
        s["h0"] = src.normal(len(lens), c) if op == "step" or case["carried"] else None
        s["cu"] = _offsets(lens)
        s["cu_seqlens"] = _int32(s["cu"])
        if op == "step":
            s["h"] = s["h0"].clone()
        elif case["gradient"]:
            s["dout"] = src.normal(n, c).to(dt)
            s["dh_last"] = src.normal(len(lens), c)
        if own:
            from linearized_attention_rope_gb300 import hla
            kind = {"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16}
            s["params"] = hla.RecurrenceParams(c, gate_dim=case["gate_dim"], dtype=kind[case["dtype"]],
                                               gate_dtype=kind[case["gates"]])
            if op == "recurrence":
                s["ws"] = hla.alloc_recurrence_workspace(s["params"], n)
                if case["gradient"]:
                    s["states"] = hla.alloc_recurrence_states(s["params"], n)
        return s
    if op == "norm":
        shape = (case["tokens"], case["heads"], case["cols"]) if case["heads"] > 1 else (case["tokens"], case["cols"])
        # rows of a residual stream: tokens differ in size, a few channels are far larger than the rest
        size = torch.exp2(src.normal(case["tokens"], *[1] * (len(shape) - 1)))
        loud = 1.0 + 20.0 * (torch.rand(case["cols"], generator=src.g, device="cuda") < 0.01)
        s["x"] = (src.normal(*shape) * size * loud).to(dt)
        s["weight"] = (1.0 + 0.3 * src.normal(case["cols"])).to(dt)
        s["residual"] = (src.normal(*shape) * size).to(dt) if case["residual"] else None
        if case["gradient"]:
            s["dout"] = src.normal(*shape).to(dt)
        if own:
            from linearized_attention_rope_gb300 import hla
            kind = {"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16, "e4m3": hla.DTYPE_E4M3}
            s["params"] = hla.NormParams(case["cols"], n_heads=case["heads"], dtype=kind[case["dtype"]],
                                         out_dtype=kind[case["out"]], group=case["group"], eps=1e-6)
            if case["gradient"]:
                s["ws"] = hla.alloc_norm_workspace(s["params"])
        return s
    m, k, n = case["tokens"], case["n_in"], case["n_out"]
    x = src.normal(m, k) * torch.exp2(src.normal(m, 1))
    s["x"], s["x_exp"] = _to_8_bits(x, case["x_group"]) if case["x"] == "e4m3" else (x.to(dt), None)
    s["w"] = src.nibbles(n, k // 2)
    s["scales"] = (torch.exp2(0.5 * src.normal(n, k // case["group"])) / (3.0 * math.sqrt(k))).to(dt)
    s["offsets"] = (s["scales"].float() * src.normal(n, k // case["group"])).to(dt) if case["offsets"] else None
    if own:
        from linearized_attention_rope_gb300 import hla
        kind = {"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16, "e4m3": hla.DTYPE_E4M3}
        s["params"] = hla.Linear4Params(k, n, group=case["group"], dtype=kind[case["dtype"]], x_dtype=kind[case["x"]],
                                        x_group=case["x_group"])
    return s


# ---- the plain forms ------------------------------------------------------------------------------------

def _rows(case, s):
    """Per row of a packed batch, whether it is its sequence's first and its last."""
    n = s["x"].shape[0]
    cu = s["cu_seqlens"].long()
    some = cu[1:] > cu[:-1]
    first = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
    first[torch.where(some, cu[:-1], n)] = True
    first = first[:n, None]
    return first, torch.cat([first[1:], torch.ones_like(first[:1])])


def _scan(a, b, longest):
    """y_t = a_t y_{t-1} + b_t over rows, by doubling: after each step a row has taken in twice as many before it."""
    a, b, k = a.clone(), b.clone(), 1
    while k < longest:
        b[k:] += a[k:] * b[:-k]
        a[k:] *= a[:-k].clone()
        k *= 2
    return b


def _recurrence(s):
    case = s["case"]
    n, c, group = s["x"].shape[0], case["channels"], case["gate_dim"]
    cu = s["cu_seqlens"].long()
    some = (cu[1:] > cu[:-1])[:, None]
    lens = [b - a for a, b in zip(s["cu"], s["cu"][1:])]
    first, last = _rows(case, s)
    a = torch.exp(s["g"].double())  # in 64 bits: products and sums over thousands of rows
    a = a.repeat_interleave(group, 1) if group > 1 else a
    h0 = torch.zeros(len(lens), c, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    before = torch.zeros(n + 1, c, dtype=torch.float64, device="cuda")  # the state that a sequence's first row meets
    before[torch.where(some[:, 0], cu[:-1], n)] = h0
    before = before[:n]
    h = _scan(a.masked_fill(first, 0.0), s["x"].double() + a * before, max(lens))
    out = h.to(s["x"].dtype)
    end = (cu[1:] - 1).clamp(min=0)
    h_last = torch.where(some, h[end], h0).float()
    if not case["gradient"]:
        return {"out": out, "h_last": h_last}
    # backwards: the state's gradient takes the next row's, through the next row's gate
    seed = s["dout"].double()
    at_end = torch.zeros(n + 1, c, dtype=torch.float64, device="cuda")
    at_end[torch.where(some[:, 0], cu[1:] - 1, n)] = s["dh_last"].double()
    seed += at_end[:n]
    after = torch.cat([a[1:], torch.zeros_like(a[:1])]).masked_fill_(last, 0.0)
    dh = _scan(after.flip(0), seed.flip(0), max(lens)).flip(0)
    prior = torch.where(first, before, torch.cat([before[:1], h[:-1]]))
    dg = dh * a * prior
    if group > 1:
        dg = dg.view(n, -1, group).sum(-1)
    got = {"out": out, "h_last": h_last, "g": dg.to(s["g"].dtype), "x": dh.to(s["x"].dtype)}
    if case["carried"]:
        start = cu[:-1].clamp(max=n - 1)
        got["h0"] = torch.where(some, (a * dh)[start], s["dh_last"].double()).float()
    return got


def _step(s):
    case = s["case"]
    a = torch.exp(s["g"].float())
    if case["gate_dim"] > 1:
        a = a.repeat_interleave(case["gate_dim"], 1)
    h = a * s["h"] + s["x"].float()
    s["h"].copy_(h)
    return {"out": h.to(s["x"].dtype), "h": s["h"]}


def _to_8_bits(x, group):
    """Groups of a row (0: the whole row) as 8-bit floats and a power of two: the smallest that keeps them within 448."""
    rows, cols = x.shape
    width = group or cols
    y = torch.nn.functional.pad(x, (0, -cols % width)).view(rows, -1, width)
    part, power = torch.frexp(y.abs().amax(-1))
    e = torch.where(part == 0, -127, power - 9 + (part > 0.875).int()).clamp(min=-127)
    y = torch.ldexp(y, -e[..., None]).float().to(torch.float8_e4m3fn).view(rows, -1)[:, :cols]
    return y.contiguous().view(torch.uint8), (e + 127).to(torch.uint8)


def _from_8_bits(x, e, group):
    rows, cols = x.shape
    e = e.int().repeat_interleave(group or cols, 1)[:, :cols] - 127
    return torch.ldexp(x.view(torch.float8_e4m3fn).float(), e)


def _norm(s):
    case = s["case"]
    dt = s["x"].dtype
    w = s["weight"].float()
    x = s["x"].float()
    if case["gradient"]:
        dy = s["dout"].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        y, wd = x * r, w * dy
        dx = (wd - y * (wd * y).mean(-1, keepdim=True)) * r
        if case["residual"]:
            dx += s["residual"].float()  # here: the gradient that the residual stream brings
        dw = (dy * y).view(-1, case["cols"]).sum(0, dtype=torch.float64)
        return {"x": dx.to(dt), "weight": dw.float()}
    got = {}
    if case["residual"]:
        got["sum"] = (x + s["residual"].float()).to(dt)
        x = got["sum"].float()
    if case["out"] == "e4m3":  # in 64 bits: values next to a border between two 8-bit floats
        x, w = x.double(), w.double()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    if case["out"] == "e4m3":
        v, e = _to_8_bits(y.view(-1, case["cols"]), case["group"])
        got["out"] = _from_8_bits(v, e, case["group"]).view(y.shape).to(torch.bfloat16)  # exact
    else:
        got["out"] = y.to(dt)
    return got


def _linear4(s):
    case = s["case"]
    n, k = case["n_out"], case["n_in"]
    q = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(n, -1, case["group"])
    w = (q.float() - 8.0) * s["scales"].float()[..., None]
    del q
    if s["offsets"] is not None:
        w += s["offsets"].float()[..., None]
    x = _from_8_bits(s["x"], s["x_exp"], case["x_group"]) if case["x"] == "e4m3" else s["x"].float()
    return (x @ w.view(n, k).T).to(TYPES[case["dtype"]])


# ---- one pass -------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"step": _step, "recurrence": _recurrence, "norm": _norm, "linear4": _linear4}[op](s)
    from linearized_attention_rope_gb300 import hla
    if op == "step":
        return {"out": hla.recurrence_step(s["params"], s["g"], s["x"], s["h"]), "h": s["h"]}
    if op == "recurrence":
        states = s["states"] if case["gradient"] else None
        out, h_last = hla.recurrence(s["params"], s["g"], s["x"], s["cu_seqlens"], h0=s["h0"], states=states,
                                     ws=s["ws"])
        if not case["gradient"]:
            return {"out": out, "h_last": h_last}
        grads = hla.recurrence_backward(s["params"], s["g"], s["x"], states, s["dout"], s["cu_seqlens"], h0=s["h0"],
                                        dh_last=s["dh_last"], ws=s["ws"])
        got = {"out": out, "h_last": h_last, "g": grads["g"], "x": grads["x"]}
        if case["carried"]:
            got["h0"] = grads["h0"]
        return got
    if op == "norm":
        if case["gradient"]:
            dx, dw = hla.rms_norm_backward(s["params"], s["x"], s["dout"], weight=s["weight"], dsum=s["residual"],
                                           ws=s["ws"])
            return {"x": dx, "weight": dw}
        y = hla.rms_norm(s["params"], s["x"], weight=s["weight"], residual=s["residual"])
        got = {"sum": y.sum} if case["residual"] else {}
        if case["out"] == "e4m3":
            unit = y.exp.view(torch.float8_e8m0fnu).to(torch.bfloat16)  # the values that the bytes stand for
            got["out"] = (y.out.view(torch.float8_e4m3fn).to(torch.bfloat16).view(*unit.shape, -1) *
                          unit.unsqueeze(-1)).view(y.out.shape)
        else:
            got["out"] = y.out
        return got
    return hla.linear4(s["params"], s["x"], s["w"], s["scales"], offsets=s["offsets"], x_exp=s["x_exp"])


# ---- the same from the definitions, in 64 bits ----------------------------------------------------------

def _exact_recurrence(case, s):
    group, cu = case["gate_dim"], s["cu"]
    if cu[-1] > 140000:
        return None
    x = s["x"].double()
    a = s["g"].double().exp()
    a = a[:, torch.arange(case["channels"], device="cuda") // group]
    h, n = torch.empty_like(x), len(cu) - 1
    h_last = torch.zeros(n, case["channels"], dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h_last += s["h0"]
    for i in range(n):  # one row after another
        y = h_last[i]
        for t in range(cu[i], cu[i + 1]):
            y = torch.addcmul(x[t], a[t], y, out=h[t])
        h_last[i] = y.clone()
    if case["op"] == "step":
        return {"out": h, "h": h_last}
    if not case["gradient"]:
        return {"out": h, "h_last": h_last}
    dx, dg = s["dout"].double(), torch.zeros_like(x)
    dh0 = s["dh_last"].double()
    for i in range(n):
        b, e = cu[i], cu[i + 1]
        if e == b:
            continue
        dx[e - 1] += dh0[i]
        for t in range(e - 2, b - 1, -1):
            dx[t].addcmul_(a[t + 1], dx[t + 1])
        dh0[i] = a[b] * dx[b]
        dg[b + 1:e] = dx[b + 1:e] * a[b + 1:e] * h[b:e - 1]
        if s["h0"] is not None:
            dg[b] = dh0[i] * s["h0"][i]
    got = {"out": h, "h_last": h_last, "x": dx, "g": dg.reshape(len(dg), -1, group).sum(2)}
    if case["carried"]:
        got["h0"] = dh0
    return got


def _exact_norm(case, s):
    w = s["weight"].double()
    got = {}
    if case["gradient"]:
        x, dy = s["x"].double(), s["dout"].double()
        length = torch.sqrt((x * x).sum(-1, keepdim=True) / case["cols"] + 1e-6)
        along = (dy * w * x).sum(-1, keepdim=True) / (case["cols"] * length ** 2)
        got["x"] = (dy * w - x * along) / length
        if s["residual"] is not None:
            got["x"] += s["residual"].double()
        got["weight"] = (dy * x / length).reshape(-1, case["cols"]).sum(0)
        return got
    x = s["x"].double()
    if s["residual"] is not None:  # the sum is kept in the layer's type, and what is kept is normalised
        got["sum"] = x + s["residual"].double()
        x = got["sum"].to(s["x"].dtype).double()
    got["out"] = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["cols"] + 1e-6) * w
    if case["out"] == "e4m3":  # next to a border between two 8-bit floats either of them is right
        got["out"] = None
    return got


def _exact_linear4(case, s):
    x = s["x"]
    if case["x"] == "e4m3":
        unit = torch.exp2(s["x_exp"].double() - 127.0)
        at = torch.arange(case["n_in"], device="cuda") // (case["x_group"] or case["n_in"])
        x = x.view(torch.float8_e4m3fn).to(torch.float64) * unit[:, at]
    x = x.double()
    if 2.0 * x.shape[0] * case["n_in"] * case["n_out"] > 1e11:
        return None
    at = torch.arange(case["n_in"], device="cuda") // case["group"]
    out = []
    for n in range(0, case["n_out"], 2048):
        b = s["w"][n:n + 2048]
        w = torch.empty(len(b), case["n_in"], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (b % 16).double(), (b // 16).double()
        w = (w - 8.0) * s["scales"][n:n + 2048].double()[:, at]
        if s["offsets"] is not None:
            w = w + s["offsets"][n:n + 2048].double()[:, at]
        out.append(torch.einsum("mk,nk->mn", x, w))
    return torch.cat(out, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_linear4(case, s) if case["op"] == "linear4" else _exact_recurrence(case, s)
