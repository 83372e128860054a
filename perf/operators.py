"""The operators of a backbone's full softmax layers, as cases that can be timed.

Rotary positions (forward and gradient), causal attention over packed prompts (forward, forward with
gradients, and a chunk of a prompt behind keys that are already there), the write of new keys and values
into a paged cache with their read-back, and the decode step over such a cache.  `run` computes a case in
elementary torch operations, or, where `own` is true, by the calls a user makes of
linearized_attention_rope_gb300.
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
        # one decode step's tokens of 64 sequences, positions anywhere in a 128 K context
        dict(name="rope_tokens", op="rope", tokens=64, q_heads=32, kv_heads=8, dim=128, rot=128, pairs="half",
             scaling="bands", factor=8.0, original=8192, base=500000.0, dtype="bf16", far=131072, gradient=False),
        # the gradient of a packed batch's rotation: fp32, interleaved pairs in half of the head, stretched context
        dict(name="rope_gradient", op="rope", tokens=8193, q_heads=64, kv_heads=8, dim=128, rot=64,
             pairs="interleaved", scaling="yarn", factor=4.0, original=32768, base=1000000.0, dtype="f32",
             far=131072, gradient=True),
        # a batch of short prompts packed together: launch latency and ragged ends
        dict(name="prompt_short", op="attention", lens="5,64,1,130,33,0,200,77", cached="0,0,0,0,0,0,0,0",
             q_heads=4, kv_heads=2, dim=64, dtype="bf16", gradient=False),
        # one long prompt of an 8 B model's layer
        dict(name="prompt_long", op="attention", lens="32768", cached="0", q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", gradient=False),
        # the next chunks of two prompts, behind keys that were computed before
        dict(name="prompt_chunk", op="attention", lens="500,1012", cached="16000,7001", q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", gradient=False),
        # training on one 4096-token sequence of the same layer
        dict(name="train_one", op="attention", lens="4096", cached="0", q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", gradient=True),
        # training on a ragged pack of a 32 B model's layer (eight query heads per key head)
        dict(name="train_packed", op="attention", lens="1024,2999,4096,8190", cached="0,0,0,0", q_heads=64, kv_heads=8,
             dim=128, dtype="bf16", gradient=True),
        # the small fp32 layer that numerics are checked on, with its gradients
        dict(name="train_f32", op="attention", lens="512,301", cached="0,0", q_heads=4, kv_heads=2, dim=64,
             dtype="f32", gradient=True),
        # prompts' keys and values into an 8-bit cache and back out for the next chunk
        dict(name="cache_prompt", op="cache", lens="16384,8191,5000,3000", starts="0,0,0,0", page=64, kv_heads=8,
             dim=128, dtype="bf16", kept="e4m3"),
        # a few rows per sequence at ragged positions, from an fp32 layer
        dict(name="cache_tokens", op="cache", lens="1,4,0,1,7,1,2,1", starts="0,100,17,4095,60,8191,63,1000", page=16,
             kv_heads=4, dim=64, dtype="f32", kept="e4m3"),
        # a decode step of 64 sequences at 8192 tokens each, cache in 8 bits
        dict(name="decode_batch", op="decode", lens=",".join(["8192"] * 64), page=64, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", kept="e4m3"),
        # a decode step of a few sequences of very different lengths, cache in bf16
        dict(name="decode_ragged", op="decode", lens="1,777,131072,20001,4095", page=16, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", kept="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 8]), kv


def _text(values):
    return ",".join(str(int(v)) for v in values)


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "cache", "decode"])
    q_heads, kv_heads = _heads(rng)
    dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        return dict(op=op, tokens=_spread(rng, 1, 8192), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 16]), pairs=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "bands", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    original=rng.choice([4096, 8192, 32768]), base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    dtype=dtype, far=_spread(rng, 1000, 1000000), gradient=rng.random() < 0.5)
    if op == "attention":
        n = _spread(rng, 1, 12)
        gradient = rng.random() < 0.5
        total = _spread(rng, 16, 1500 if dtype == "f32" else 8192)
        lens = [max(0, int(total / n * rng.uniform(0.0, 2.0))) for _ in range(n)]
        lens[rng.randrange(n)] += 1
        before = rng.random() < 0.3
        cached = [_spread(rng, 1, 4000) if before and rng.random() < 0.7 else 0 for _ in range(n)]
        return dict(op=op, lens=_text(lens), cached=_text(cached), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    dtype=dtype, gradient=gradient)
    kept = rng.choice(["e4m3", "e4m3", dtype])
    page = rng.choice([16, 32, 64, 128, 256])
    n = _spread(rng, 1, 64)
    if op == "cache":
        total = _spread(rng, 1, 32768)
        lens = [max(0, int(total / n * rng.uniform(0.0, 2.0))) for _ in range(n)]
        lens[rng.randrange(n)] += 1
        return dict(op=op, lens=_text(lens), starts=_text([_spread(rng, 1, 5000) - 1 for _ in range(n)]), page=page,
                    kv_heads=kv_heads, dim=dim, dtype=dtype, kept=kept)
    most = _spread(rng, 1, min(131072, 524288 // n))
    return dict(op=op, lens=_text([max(0, int(most * rng.uniform(0.0, 1.0)) + 1) for _ in range(n)]), page=page,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype, kept=kept)


def _numbers(text):
    return [int(x) for x in text.split(",")]


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _pairs(case):
    return sum(a * c + a * (a + 1) // 2 for a, c in zip(_numbers(case["lens"]), _numbers(case["cached"])))


def work(case):
    op, b = case["op"], SIZES[case["dtype"]]
    if op == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 2 * n * case["dim"] * b + 8 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "attention":
        rows = sum(_numbers(case["lens"]))
        keys = rows + sum(_numbers(case["cached"]))
        q, kv = rows * case["q_heads"] * case["dim"] * b, keys * case["kv_heads"] * case["dim"] * b
        if case["gradient"]:  # q, k, v, dout in; out, dq, dk, dv out
            return {"bytes": 4 * q + 4 * kv, "flops": 14 * case["dim"] * case["q_heads"] * _pairs(case)}
        return {"bytes": 2 * q + 2 * kv + 4 * rows * case["q_heads"],
                "flops": 4 * case["dim"] * case["q_heads"] * _pairs(case)}
    kept = SIZES[case["kept"]]
    row = case["dim"] * kept + (1 if case["kept"] == "e4m3" else 0)
    if op == "cache":  # rows in, cache rows out, cache rows in, rows out; keys and values
        n = sum(_numbers(case["lens"])) * case["kv_heads"]
        return {"bytes": 2 * n * (2 * case["dim"] * b + 2 * row), "flops": 4 * n * case["dim"]}
    lens = _numbers(case["lens"])
    return {"bytes": 2 * sum(lens) * case["kv_heads"] * row + 2 * len(lens) * case["q_heads"] * case["dim"] * b,
            "flops": 4 * sum(lens) * case["q_heads"] * case["dim"]}


# ---- inputs ---------------------------------------------------------------------------------------------

class _Source:
    """Seeded tensors: standard normal values, and keys gathered around one direction per head."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def keys(self, n, heads, dim):
        mean = self.normal(heads, dim)
        return mean / mean.norm(dim=-1, keepdim=True) + 0.6 * self.normal(n, heads, dim)

    def whole(self, lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=self.g, device="cuda")

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(src, case, lens):
    """A page table [sequences, pages of the longest] over pages in a scattered order; unused entries are -1."""
    need = [-(-n // case["page"]) for n in lens]
    wide, base = max(1, max(need)), _offsets(need)
    order = src.order(max(1, base[-1])).to(torch.int32)
    column = torch.arange(wide, device="cuda")
    need, base = torch.tensor(need, device="cuda"), torch.tensor(base[:-1], device="cuda")
    at = (base[:, None] + column[None]).clamp(max=order.numel() - 1)
    return torch.where(column[None] < need[:, None], order[at], -1).contiguous(), order.numel()


def prepare(case, seed):
    src = _Source(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = {"case": case}
    if op == "rope":
        n = case["tokens"]
        s["q"] = src.normal(n, case["q_heads"], case["dim"]).to(dt)
        s["k"] = src.keys(n, case["kv_heads"], case["dim"]).to(dt)
        s["positions"] = src.whole(0, case["far"], n)
        s["freq"], s["gain"] = _frequencies(case)
        if own:
            from linearized_attention_rope_gb300 import hla
            s["rope"] = hla.RopeParams(
                case["q_heads"], case["kv_heads"], case["dim"], rot_dim=case["rot"],
                layout={"half": hla.ROPE_HALF, "interleaved": hla.ROPE_INTERLEAVED}[case["pairs"]],
                scaling={"none": hla.ROPE_SCALE_NONE, "linear": hla.ROPE_SCALE_LINEAR,
                         "bands": hla.ROPE_SCALE_BANDS, "yarn": hla.ROPE_SCALE_YARN}[case["scaling"]],
                dtype={"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16}[case["dtype"]], base=case["base"],
                factor=case["factor"], original_len=case["original"])
        return s
    lens = _numbers(case["lens"])
    if op == "attention":
        cached = _numbers(case["cached"])
        rows, keys = sum(lens), sum(lens) + sum(cached)
        s["q"] = src.normal(rows, case["q_heads"], case["dim"]).to(dt)
        s["k"] = src.keys(keys, case["kv_heads"], case["dim"]).to(dt)
        s["v"] = src.normal(keys, case["kv_heads"], case["dim"]).to(dt)
        s["cu_q"], s["cu_k"] = _offsets(lens), _offsets([a + c for a, c in zip(lens, cached)])
        s["cu_seqlens_q"], s["cu_seqlens_k"] = _int32(s["cu_q"]), _int32(s["cu_k"])
        if case["gradient"]:
            s["dout"] = src.normal(rows, case["q_heads"], case["dim"]).to(dt)
        # each row's sequence and position, and each key's (the plain form's mask)
        s["row_seq"], s["row_pos"] = _places(lens, cached)
        s["key_seq"], s["key_pos"] = _places([a + c for a, c in zip(lens, cached)], [0] * len(lens))
        if own:
            from linearized_attention_rope_gb300 import hla
            s["params"] = hla.AttnParams(case["q_heads"], case["kv_heads"], case["dim"],
                                         dtype={"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16}[case["dtype"]])
            s["ws"] = hla.alloc_attention_workspace(s["params"], rows, keys, len(lens), backward=case["gradient"])
        return s
    starts = _numbers(case["starts"]) if op == "cache" else [0] * len(lens)
    table, n_pages = _pages(src, case, [a + b if a else 0 for a, b in zip(lens, starts)])
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    s["table"] = table
    if op == "cache":
        n = sum(lens)
        size = torch.exp2(src.normal(n, 1, 1))  # tokens differ in size
        s["k"] = (src.keys(n, case["kv_heads"], case["dim"]) * size).to(dt)
        s["v"] = (src.normal(n, case["kv_heads"], case["dim"]) * size).to(dt)
        s["cu_seqlens"] = _int32(_offsets(lens))
        s["starts"] = torch.tensor(starts, dtype=torch.int64, device="cuda")
        s["row_seq"], s["row_pos"] = _places(lens, starts)
        kind = torch.uint8 if case["kept"] == "e4m3" else TYPES[case["kept"]]
        s["cache"] = {"k": torch.zeros(shape, dtype=kind, device="cuda"),
                      "v": torch.zeros(shape, dtype=kind, device="cuda")}
        if case["kept"] == "e4m3":
            s["cache"]["k_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda")
            s["cache"]["v_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda")
    else:
        s["q"] = src.normal(len(lens), case["q_heads"], case["dim"]).to(dt)
        s["lens"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
        rows = n_pages * case["page"]
        k = src.keys(rows, case["kv_heads"], case["dim"]).view(n_pages, case["page"], case["kv_heads"], -1)
        k = k.transpose(1, 2).contiguous()
        v = src.normal(*shape)
        if case["kept"] == "e4m3":
            (k, ke), (v, ve) = _to_8_bits(k), _to_8_bits(v)
            s["cache"] = {"k": k, "v": v, "k_exp": ke, "v_exp": ve}
        else:
            s["cache"] = {"k": k.to(TYPES[case["kept"]]), "v": v.to(TYPES[case["kept"]])}
    if own:
        from linearized_attention_rope_gb300 import hla
        dtype = {"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16}[case["dtype"]]
        kept = {"f32": hla.DTYPE_F32, "bf16": hla.DTYPE_BF16, "e4m3": hla.DTYPE_E4M3}[case["kept"]]
        s["kv"] = hla.Cache(hla.CacheParams(case["kv_heads"], case["dim"], case["page"], n_pages, table.shape[1],
                                            dtype=dtype, cache_dtype=kept), table, **s["cache"])
        if op == "decode":
            s["params"] = hla.AttnParams(case["q_heads"], case["kv_heads"], case["dim"], dtype=dtype)
            s["ws"] = hla.alloc_decode_workspace(s["params"], s["kv"])
    return s


def _places(lens, first):
    """Per row of a packed batch: its sequence, and its position when sequence i's rows start at first[i]."""
    n = torch.tensor(lens, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n, output_size=sum(lens))
    begin = torch.tensor([f - o for f, o in zip(first, _offsets(lens))], device="cuda")
    return seq, torch.arange(sum(lens), device="cuda") + begin[seq]


# ---- the plain forms ------------------------------------------------------------------------------------

def _frequencies(case):
    """Angle per position of every pair (float64), and the factor on the rotated values."""
    r = case["rot"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    w = case["base"] ** (-2.0 * i / r)
    f, orig = case["factor"], float(case["original"])
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "bands":  # waves longer than the original context stretch, ones below a quarter stay
        turns = orig * w / (2 * math.pi)
        blend = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return w * ((1 - blend) / f + blend), 1.0
    if case["scaling"] == "yarn":
        def index(turns):
            return r * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(case["base"]))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


def _turned(x, cos, sin, case):
    r = case["rot"]
    y = x.float()
    z = y.clone()
    if case["pairs"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        z[..., :r // 2], z[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        z[..., 0:r:2], z[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return z.to(x.dtype)


def _rope(s):
    case = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos = (angle.cos() * s["gain"]).float()[:, None]
    sin = (angle.sin() * (-s["gain"] if case["gradient"] else s["gain"])).float()[:, None]
    return _turned(s["q"], cos, sin, case), _turned(s["k"], cos, sin, case)


def _chunks(s):
    """Row ranges of a packed batch with the keys they can see; the score block of one stays near 2 GB."""
    case, cu_q, cu_k = s["case"], s["cu_q"], s["cu_k"]
    out, r0, seq = [], 0, 0
    while r0 < cu_q[-1]:
        while cu_q[seq + 1] <= r0:
            seq += 1
        k0, r1, last = cu_k[seq], r0, seq
        while r1 < cu_q[-1]:
            while cu_q[last + 1] <= r1:
                last += 1
            step = min(128, cu_q[last + 1] - r1)
            k1 = cu_k[last + 1] - (cu_q[last + 1] - (r1 + step))
            if r1 > r0 and case["q_heads"] * (r1 + step - r0) * (k1 - k0) > 1 << 29:
                break
            r1, kept = r1 + step, k1
        out.append((r0, r1, k0, kept))
        r0 = r1
    return out


def _by_head(x, kv_heads):
    """[rows, heads, d] -> fp32 [kv_heads, group * rows, d]"""
    n, h, d = x.shape
    return x.float().view(n, kv_heads, h // kv_heads, d).permute(1, 2, 0, 3).reshape(kv_heads, -1, d)


def _by_row(x, rows):
    """[kv_heads, group * rows, d] -> [rows, heads, d]"""
    h, n, d = x.shape
    return x.view(h, n // rows, rows, d).permute(2, 0, 1, 3).reshape(rows, -1, d)


def _scores(s, c, q, k):
    case, (r0, r1, k0, k1) = s["case"], c
    group = case["q_heads"] // case["kv_heads"]
    hidden = (s["row_seq"][r0:r1, None] != s["key_seq"][k0:k1]) | (s["row_pos"][r0:r1, None] < s["key_pos"][k0:k1])
    x = torch.bmm(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(case["dim"]))
    x.view(case["kv_heads"], group, r1 - r0, k1 - k0).masked_fill_(hidden, -math.inf)
    return x


def _attention(s):
    case, n = s["case"], s["case"]["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    if case["gradient"]:
        dq = torch.empty_like(out)
        dk, dv = (torch.zeros(n, s["k"].shape[0], case["dim"], device="cuda") for _ in range(2))
    for c in _chunks(s):
        r0, r1, k0, k1 = c
        q, k, v = _by_head(s["q"][r0:r1], n), _by_head(s["k"][k0:k1], n), _by_head(s["v"][k0:k1], n)
        x = _scores(s, c, q, k)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p.div_(total)
        o = torch.bmm(p, v)
        out[r0:r1] = _by_row(o, r1 - r0)
        lse[r0:r1] = _by_row(top + total.log(), r1 - r0)[..., 0]
        if case["gradient"]:
            do = _by_head(s["dout"][r0:r1], n)
            dv[:, k0:k1].baddbmm_(p.transpose(1, 2), do)
            dp = torch.bmm(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True))
            ds = dp.mul_(p).mul_(1.0 / math.sqrt(case["dim"]))
            dq[r0:r1] = _by_row(torch.bmm(ds, k), r1 - r0)
            dk[:, k0:k1].baddbmm_(ds.transpose(1, 2), q)
    dt = s["q"].dtype
    if case["gradient"]:
        return {"out": out.to(dt), "q": dq.to(dt), "k": dk.transpose(0, 1).to(dt), "v": dv.transpose(0, 1).to(dt)}
    return {"out": out.to(dt), "lse": lse}


def _to_8_bits(x):
    """Rows (last axis) as 8-bit floats and a power of two: the smallest one that keeps the row within 448."""
    x = x.float()
    part, power = torch.frexp(x.abs().amax(-1))
    e = torch.where(part == 0, -127, power - 9 + (part > 0.875).int()).clamp(min=-127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _from_8_bits(x, e):
    return torch.ldexp(x.view(torch.float8_e4m3fn).float(), e.int()[..., None] - 127)


def _cache(s):
    case, kv = s["case"], s["cache"]
    page = s["table"].long()[s["row_seq"], s["row_pos"] // case["page"]]
    at = s["row_pos"] % case["page"]
    out = {}
    if case["kept"] == "e4m3":
        (k, ke), (v, ve) = _to_8_bits(s["k"]), _to_8_bits(s["v"])
        kv["k"][page, :, at], kv["k_exp"][page, :, at] = k, ke
        kv["v"][page, :, at], kv["v_exp"][page, :, at] = v, ve
        out["k"] = _from_8_bits(kv["k"][page, :, at], kv["k_exp"][page, :, at]).to(s["k"].dtype)
        out["v"] = _from_8_bits(kv["v"][page, :, at], kv["v_exp"][page, :, at]).to(s["k"].dtype)
    else:
        kv["k"][page, :, at], kv["v"][page, :, at] = s["k"], s["v"]
        out["k"], out["v"] = kv["k"][page, :, at], kv["v"][page, :, at]
    return out


def _decode(s):
    case, kv, n = s["case"], s["cache"], s["case"]["kv_heads"]
    table = s["table"].long().clamp(min=0)

    def rows(name):  # [sequences, kv heads, positions, d]
        x = kv[name][table].transpose(1, 2)
        if case["kept"] == "e4m3":
            x = _from_8_bits(x, kv[name + "_exp"][table].transpose(1, 2))
        return x.reshape(x.shape[0], n, -1, case["dim"]).float()

    k = rows("k")
    q = s["q"].float().view(len(k), n, -1, case["dim"])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(case["dim"]))
    del k
    hidden = torch.arange(x.shape[-1], device="cuda") >= s["lens"][:, None]
    p = x.masked_fill_(hidden[:, None, None], -math.inf).softmax(-1)
    v = rows("v").masked_fill_(hidden[:, None, :, None], 0.0)
    return torch.matmul(p, v).view(s["q"].shape).to(s["q"].dtype)


# ---- one pass -------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rope": _rope, "attention": _attention, "cache": _cache, "decode": _decode}[op](s)
    from linearized_attention_rope_gb300 import hla
    if op == "rope":
        return (hla.rope_backward if case["gradient"] else hla.rope)(s["rope"], s["q"], s["k"], s["positions"])
    if op == "attention":
        out, lse = hla.attention(s["params"], s["q"], s["k"], s["v"], s["cu_seqlens_q"], s["cu_seqlens_k"],
                                 ws=s["ws"])
        if not case["gradient"]:
            return {"out": out, "lse": lse}
        grads = hla.attention_backward(s["params"], s["q"], s["k"], s["v"], out, lse, s["dout"], s["cu_seqlens_q"],
                                       s["cu_seqlens_k"], ws=s["ws"])
        return {"out": out, "q": grads["q"], "k": grads["k"], "v": grads["v"]}
    if op == "cache":
        hla.cache_write(s["kv"], s["k"], s["v"], s["cu_seqlens"], s["starts"])
        k, v = hla.cache_read(s["kv"], s["cu_seqlens"], s["starts"], s["k"].shape[0])
        return {"k": k, "v": v}
    return hla.attention_decode(s["params"], s["kv"], s["q"], s["lens"], ws=s["ws"])


# ---- the same from the definitions, in 64 bits ----------------------------------------------------------

def _exact_rope(case, s):
    r, d = case["rot"], case["dim"]
    f, orig, gain, two_pi = case["factor"], case["original"], 1.0, 2.0 * math.pi
    rates = []
    for i in range(r // 2):
        w = math.exp(-math.log(case["base"]) * 2 * i / r)
        wave = two_pi / w
        if case["scaling"] == "linear":
            w = w / f
        elif case["scaling"] == "bands":
            if wave > orig:
                w = w / f
            elif wave >= orig / 4.0:
                near = (orig / wave - 1.0) / 3.0
                w = w * near + w / f * (1.0 - near)
        elif case["scaling"] == "yarn":
            gain = 1.0 + math.log(f) / 10.0
            edge = [r / 2.0 * math.log(orig / (two_pi * t)) / math.log(case["base"]) for t in (32.0, 1.0)]
            lo, hi = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
            far = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            w = w * (1.0 - far) + w / f * far
        rates.append(w)
    i = torch.arange(r // 2, device="cuda")
    first, second = (i, i + r // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.polar(torch.full((), gain, dtype=torch.float64, device="cuda"), torch.outer(
        s["positions"].double(), torch.tensor(rates, dtype=torch.float64, device="cuda")))[:, None]
    if case["gradient"]:
        turn = turn.conj()
    out = []
    for x in (s["q"], s["k"]):
        x = x.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_attention(case, s):
    lens, cached = _numbers(case["lens"]), _numbers(case["cached"])
    h, d, group = case["q_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    full = sum(a * (a + c) for a, c in zip(lens, cached)) * h * d * (14 if case["gradient"] else 4)
    if full > 1.2e13:
        return None
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), None
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    q0 = k0 = 0
    for a, c in zip(lens, cached):
        q1, k1 = q0 + a, k0 + a + c
        if a:
            unseen = torch.ones(a, a + c, dtype=torch.bool, device="cuda").triu(c + 1)
        for head in range(h if a else 0):
            q = s["q"][q0:q1, head].double()
            k, v = (s[n][k0:k1, head // group].double() for n in "kv")
            logits = (q @ k.T / d ** 0.5).masked_fill(unseen, -math.inf)
            lse[q0:q1, head] = logits.logsumexp(1)
            p = (logits - lse[q0:q1, head, None]).exp()
            out[q0:q1, head] = p @ v
            if case["gradient"]:
                do = s["dout"][q0:q1, head].double()
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / d ** 0.5
                dq[q0:q1, head] = ds @ k
                dk[k0:k1, head // group] += ds.T @ q
                dv[k0:k1, head // group] += p.T @ do
        q0, k0 = q1, k1
    if case["gradient"]:
        return {"out": out, "q": dq, "k": dk, "v": dv}
    return {"out": out, "lse": lse}


def _exact_cache(case, s):
    out = {}
    for name in "kv":
        x = s[name].double()
        if case["kept"] == "e4m3":
            top = x.abs().amax(-1, keepdim=True)
            unit = torch.exp2(torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -127))))
            unit = torch.where(unit * 224.0 >= top, unit / 2, unit)  # log2 may round up to the next whole number
            unit = torch.where(unit * 448.0 < top, unit * 2, unit).clamp(min=2.0 ** -127)
            x = x / unit
            # eighths of the value's own power of two, none finer than 2^-9; halves to even
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step * unit
        out[name] = x
    return out


def _exact_decode(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, page, d = case["q_heads"] // case["kv_heads"], case["page"], case["dim"]
    for n, length in enumerate(_numbers(case["lens"])):
        if not length:
            continue
        ids = s["table"][n, :-(-length // page)].long()
        got = {}
        for name in "kv":
            x = s["cache"][name][ids]
            if case["kept"] == "e4m3":
                x = x.view(torch.float8_e4m3fn).to(torch.float64) * \
                    torch.exp2(s["cache"][name + "_exp"][ids].double() - 127.0)[..., None]
            got[name] = x.double().permute(1, 0, 2, 3).reshape(case["kv_heads"], -1, d)[:, :length]
        q = s["q"][n].double().view(case["kv_heads"], group, d)
        w = torch.softmax(torch.einsum("hgd,hkd->hgk", q, got["k"]) / d ** 0.5, -1)
        out[n] = torch.einsum("hgk,hkd->hgd", w, got["v"]).reshape(-1, d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attention": _exact_attention, "cache": _exact_cache,
            "decode": _exact_decode}[case["op"]](case, s)
