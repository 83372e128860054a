"""GPU packed causal attention and its gradient against a 64-bit form: types, head groups, lengths from none to
several blocks, chunks behind earlier keys, rows that see nothing, padding, strides, streams and graphs.

Tolerances, per element (u = eps / 2 of the stored type, u32 = 2^-24; mag = the sums with every product replaced
by its magnitude):
  scores: d fp32 products and sums, off by at most d u32 sum |q k| scale, which is the relative error of exp;
  a sum over L keys adds at most L u32.  fp32 layers: out and dv (2 d S + L + 32) u32 mag, with S the largest
  sum |q k| scale; dq and dk the same with twice the score error (p and dp) and their own sums.
  bf16 layers add one rounding of p (and of dp's factor ds) to bf16, one of the stored out that D is formed
  from, and the result's own: out, dv: u mag + u |x|; dq, dk: 3 u mag + u |x| (a rounding of ds, and D off by u |do| |o|).
"""
import math

import pytest
import torch

import attention_cases as ac
from linearized_attention_rope_gb300 import hla

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
TYPE = {"f32": (hla.DTYPE_F32, torch.float32), "bf16": (hla.DTYPE_BF16, torch.bfloat16)}


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    build.build()


def make(dtype, d, hq, hkv, q_lens, k_lens, pad_q=0, pad_k=0, seed=0):
    t = TYPE[dtype][1]
    tq, tk = sum(q_lens) + pad_q, sum(k_lens) + pad_k
    x = {"q": ac.randn(seed + 1, tq, hq, d), "k": ac.randn(seed + 2, tk, hkv, d), "v": ac.randn(seed + 3, tk, hkv, d),
         "dout": ac.randn(seed + 4, tq, hq, d)}
    return {n: v.to(t) for n, v in x.items()}


def params(dtype, d, hq, hkv, scale=0.0):
    return hla.AttnParams(hq, hkv, d, dtype=TYPE[dtype][0], scale=scale)


def run(prm, x, q_lens, k_lens, backward=True, same=False):
    g = {n: t.cuda() for n, t in x.items()}
    cq, ck = ac.cu(q_lens), None if same else ac.cu(k_lens)
    ws = hla.alloc_attention_workspace(prm, g["q"].shape[0], g["k"].shape[0], len(q_lens), backward=True)
    out, lse = hla.attention(prm, g["q"], g["k"], g["v"], cq, ck, ws=ws)
    grads = hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], cq, ck, ws=ws) if backward else {}
    torch.cuda.synchronize()
    assert hla.check_workspace_error(ws) == 0
    return out, lse, grads


def check(dtype, d, x, ref, out, lse, grads, q_lens, k_lens, scale=None):
    r_out, r_lse, r_grads, mag = ref
    scale = 1 / math.sqrt(d) if scale is None else scale
    nq, nk = sum(q_lens), sum(k_lens)
    qm = x["q"][:nq].double().abs()
    km = x["k"][:nk].double().abs()
    S = float(scale * qm.norm(dim=-1).max() * km.norm(dim=-1).max()) if nq and nk else 0.0
    L = max([1] + k_lens + [n * (x["q"].shape[1] // x["k"].shape[1]) for n in q_lens])
    fp = (2 * d * S + L + 32) * U32
    u = ac.EPS[TYPE[dtype][1]] / 2
    half = 0.0 if dtype == "f32" else u
    off = (lse.cpu().double()[:nq] - r_lse).abs()
    seen = torch.isfinite(r_lse)
    assert torch.equal(torch.isneginf(lse.cpu()[:nq]), ~seen)
    assert (off[seen] <= fp + 4 * U32 * r_lse[seen].abs()).all()
    got = {"out": out[:nq], **{n: g[: nq if n == "q" else nk] for n, g in grads.items()}}
    want = {"out": r_out, **r_grads}
    for name, g in got.items():
        n = 3 if name in ("q", "k") else 1
        tol = (n * half + 3 * fp) * mag[name] + 1.01 * u * want[name].abs()
        diff = (g.cpu().double() - want[name]).abs()
        assert (diff <= tol).all(), f"{name}: {float((diff - tol).max())} over, of {float(want[name].abs().max())}"
        # on the whole (independent roundings): far below the bound per element.  Not where the exact result
        # cancels: a row with one key has p = 1 and dp = D, so dq = 0 exactly, while dp and D, two sums of d
        # products, each keep up to d u32 of their magnitude (for that the bound per element stands)
        lim = 1e-4 if dtype == "f32" else 4 * u / math.sqrt(3)
        if float(want[name].norm()) > 1e-2 * float(mag[name].norm()):
            assert ac.rel(g, want[name]) <= lim, f"{name}: {ac.rel(g, want[name])}"


def full_check(dtype, d, hq, hkv, q_lens, k_lens=None, scale=None, seed=0):
    same = k_lens is None
    k_lens = q_lens if same else k_lens
    x = make(dtype, d, hq, hkv, q_lens, k_lens, seed=seed)
    out, lse, grads = run(params(dtype, d, hq, hkv, scale or 0.0), x, q_lens, k_lens, same=same)
    ref = ac.attention(x["q"], x["k"], x["v"], q_lens, k_lens, scale, dout=x["dout"])
    check(dtype, d, x, ref, out, lse, grads, q_lens, k_lens, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (6, 2), (8, 1), (12, 2)])
def test_packed_prompts(dtype, d, hq, hkv):
    full_check(dtype, d, hq, hkv, [1, 33, 0, 200, 64, 5])


@pytest.mark.parametrize("dtype,d,lens", [("bf16", 128, [1]), ("bf16", 64, [1]), ("bf16", 128, [128]),
                                          ("bf16", 128, [129]), ("bf16", 128, [255, 257]), ("bf16", 64, [700]),
                                          ("bf16", 128, [900, 31]), ("f32", 64, [1]), ("f32", 128, [65, 190])])
def test_lengths_around_the_tiles(dtype, d, lens):
    full_check(dtype, d, 4, 2, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,lens", [(1, 1, [3]), (8, 2, [0, 4, 6, 4]), (4, 4, [40, 128, 17]), (16, 1, [90])])
def test_short_prompts_are_rounded_once(d, hq, hkv, lens):
    # one key tile: probabilities and score gradients in two bf16 parts (2^-16 of them left), so that results are off by
    # their own rounding, u of their size, and by the rest: out, dv 2^-16 mag, dq, dk that and their dS, 2^-15 mag,
    # plus the fp32 sums (as above)
    x = make("bf16", d, hq, hkv, lens, lens)
    out, lse, grads = run(params("bf16", d, hq, hkv), x, lens, lens, same=True)
    r_out, _, r_grads, mag = ac.attention(x["q"], x["k"], x["v"], lens, lens, dout=x["dout"])
    S = float(x["q"].double().norm(dim=-1).max() * x["k"].double().norm(dim=-1).max()) / math.sqrt(d)
    fp, u = 3 * (2 * d * S + 32 + max(lens) * hq // hkv) * U32, ac.EPS[torch.bfloat16] / 2
    for name, got, want in [("out", out, r_out)] + [(n, grads[n], r_grads[n]) for n in "qkv"]:
        part = 2.0 ** -15 if name in ("q", "k") else 2.0 ** -16
        off = (got.cpu().double() - want).abs()
        assert (off <= (part + fp) * mag[name] + 1.01 * u * want.abs()).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_behind_earlier_keys(dtype, d):
    full_check(dtype, d, 4, 2, [1, 40, 130, 3], [300, 41, 390, 3])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 1)])
def test_few_rows_over_many_keys(d, hq, hkv):
    # the keys are cut over blocks and joined: rows whose parts differ in number, an empty sequence, a row that sees
    # its first keys only in the last part
    full_check("bf16", d, hq, hkv, [1, 17, 0, 40], [5000, 2100, 30, 40])
    full_check("bf16", d, hq, hkv, [3], [9001])


@pytest.mark.parametrize("d,hq,hkv,lens", [(64, 1, 1, [2500]), (128, 1, 1, [2200, 2050])])
def test_whole_prompts_of_few_heads(d, hq, hkv, lens):
    # the keys are cut as well; early items have fewer parts than the longest
    full_check("bf16", d, hq, hkv, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 4), (12, 2)])
def test_few_rows_over_many_keys_in_fp32(d, hq, hkv):
    # keys cut over blocks and joined: sequences of more, fewer and no parts, a row that sees a few keys of the first
    full_check("f32", d, hq, hkv, [5, 46, 0, 31, 12], [656, 46, 700, 3537, 6])
    full_check("f32", d, hq, hkv, [3], [9001])
    full_check("f32", d, hq, hkv, [70], [530])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,q_lens,k_lens", [(8, 1, [700, 0, 300], None), (16, 1, [900], None),
                                                  (6, 2, [1500, 7], None), (32, 1, [130, 260], [130, 700]),
                                                  (24, 2, [500], [200])])
def test_few_key_blocks_of_many_rows(d, hq, hkv, q_lens, k_lens):
    # the rows that see a key block are cut over blocks and joined: whole head groups and pieces of them
    full_check("bf16", d, hq, hkv, q_lens, k_lens)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_no_key(dtype, d):
    # fewer keys than queries: the first rows see nothing; a sequence without keys; one without queries
    full_check(dtype, d, 4, 2, [60, 200, 10, 0], [20, 3, 0, 70])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_lens,k_lens", [([5, 3], [0, 0]), ([0, 0], [4, 70])])
def test_no_keys_at_all_or_no_queries(dtype, q_lens, k_lens):
    # nothing is seen: out and every gradient are 0, lse -infinity; padding is left alone
    x = make(dtype, 64, 4, 2, q_lens, k_lens, pad_q=2 if sum(q_lens) else 0, pad_k=2 if sum(k_lens) else 0)
    nq, nk = sum(q_lens), sum(k_lens)
    g = {n: t.cuda() for n, t in x.items()}
    prm, cq, ck = params(dtype, 64, 4, 2), ac.cu(q_lens), ac.cu(k_lens)
    ws = hla.alloc_attention_workspace(prm, g["q"].shape[0], g["k"].shape[0], 2, backward=True)
    out, lse = torch.full_like(g["q"], 7.0), torch.full(g["q"].shape[:2], 7.0, device="cuda")
    grads = {n: torch.full_like(g[n], 7.0) for n in "qkv"}
    hla.attention(prm, g["q"], g["k"], g["v"], cq, ck, out=out, lse=lse, ws=ws)
    hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], cq, ck, grads=grads, ws=ws)
    assert hla.check_workspace_error(ws) == 0
    assert (out[:nq] == 0).all() and torch.isneginf(lse[:nq]).all() and (lse[nq:] == 7.0).all()
    for t, n in ((out, nq), (grads["q"], nq), (grads["k"], nk), (grads["v"], nk)):
        assert (t[:n] == 0).all() and (t[n:] == 7.0).all()
    bad = ac.cu([3, 99])  # past the other side's rows, of which there are none
    if nq:
        hla.attention(prm, g["q"], g["k"], g["v"], cq, bad, out=out, lse=lse, ws=ws)
        assert hla.check_workspace_error(ws) != 0
    hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], *((cq, bad) if nq else (bad, ck)),
                           grads=grads, ws=ws)
    assert hla.check_workspace_error(ws) != 0


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_layers_with_many_heads(d):
    # enough blocks for the wider ones
    full_check("f32", d, 32, 8, [300, 0, 345])
    full_check("f32", d, 32, 32, [200, 150, 90], [300, 150, 20])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,lens", [(1, 1, [300]), (4, 2, [330, 201, 0, 15]), (8, 4, [260, 400]), (12, 4, [700, 160])])
def test_fp32_layers_by_block_size(d, hq, hkv, lens):
    # few, more and enough blocks of the smaller sizes
    full_check("f32", d, hq, hkv, lens)
    full_check("f32", d, hq, hkv, [n // 2 for n in lens], lens)


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_layers_with_many_heads_and_nan_outside(d):
    # the rows of one sequence and the padding hold NaN: the others stay what they are, bit for bit
    lens = [130, 75, 200]
    x = make("f32", d, 32, 8, lens, lens, pad_q=30, pad_k=30)
    want = run(params("f32", d, 32, 8), x, lens, lens)
    for n in x:
        x[n][130:205] = math.nan
        x[n][405:] = math.inf
    got = run(params("f32", d, 32, 8), x, lens, lens)
    keep = torch.cat([torch.arange(130), torch.arange(205, 405)]).cuda()
    for a, b in ((want[0], got[0]), (want[1], got[1]), *((want[2][n], got[2][n]) for n in "qkv")):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_sequences(dtype):
    lens = [(7 * i) % 23 for i in range(75)]
    full_check(dtype, 64, 2, 1, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length,hq,hkv", [(64, 32, 8), (130, 4, 1), (512, 32, 8), (33, 6, 2)])
def test_many_short_items_again_and_again(d, length, hq, hkv):
    # thousands of items of a few tiles each, many calls back to back: every hand-over between the warps of a block
    # in every order that timing allows; all results equal, no wait runs out
    lens = [length] * (16384 // length)
    prm, c, n = hla.AttnParams(hq, hkv, d), ac.cu(lens), sum(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v, do = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv, hq))
    ws = hla.alloc_attention_workspace(prm, n, n, len(lens), backward=True)
    out, lse = hla.attention(prm, q, k, v, c, ws=ws)
    grads = hla.attention_backward(prm, q, k, v, out, lse, do, c, ws=ws)
    o2, l2, g2 = torch.empty_like(out), torch.empty_like(lse), {m: torch.empty_like(t) for m, t in grads.items()}
    for _ in range(100):
        hla.attention(prm, q, k, v, c, out=o2, lse=l2, ws=ws)
        hla.attention_backward(prm, q, k, v, o2, l2, do, c, grads=g2, ws=ws)
    assert hla.check_workspace_error(ws) == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2) and all(torch.equal(grads[m], g2[m]) for m in grads)
    a, b = 2 * length, 3 * length  # one of them against the 64-bit form
    x = {m: t[a:b].cpu() for m, t in (("q", q), ("k", k), ("v", v), ("dout", do))}
    ref = ac.attention(x["q"], x["k"], x["v"], [length], [length], dout=x["dout"])
    check("bf16", d, x, ref, out[a:b], lse[a:b], {m: t[a:b] for m, t in grads.items()}, [length], [length])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scale_and_large_scores(dtype):
    # scores of +-60: one key takes almost everything in many rows
    full_check(dtype, 64, 2, 1, [150], scale=2.0, seed=5)


def dq_bound(d, x, lens, scale):
    """dq in 64 bits, and the 2-norm that its rounding errors add up to over the whole tensor, for D of 32 bits: per row,
    independent roundings of ds to bf16 (u / sqrt(3) of each) in the sum with k, of the result, and a D that may be off by
    four times u times the 2-norm of the row's ds, times sum p k less the mean of 16 keys that the row's whole tile sees."""
    u, want, size = ac.EPS[torch.bfloat16] / 2, [], 0.0
    a = 0
    for n in lens:
        q, k, v, do = (x[m][a:a + n].double() for m in ("q", "k", "v", "dout"))
        g = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            kk, vv = k[:, h // g], v[:, h // g]
            s = (q[:, h] @ kk.T * scale).masked_fill(torch.ones(n, n).triu(1).bool(), -math.inf)
            p = torch.softmax(s, 1)
            dp = do[:, h] @ vv.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
            dq = ds @ kk
            want.append(dq)
            size += float((ds ** 2 @ kk ** 2 + dq ** 2).sum()) * u * u / 3
            tile = 128 // min(16, g & -g)  # positions
            seen = torch.arange(n)[:, None] // tile * tile + 1
            mean = kk[(2 * torch.arange(16) + 1) * seen // 32].mean(1)
            size += float((16 * u * u * (ds ** 2).sum(1, keepdim=True) * (p @ kk - mean) ** 2).sum())
        a += n
    return want, math.sqrt(size)


@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 1), (128, 1, 1), (128, 4, 1)])
@pytest.mark.parametrize("lens", [[700], [200, 333]])
@pytest.mark.parametrize("kind", ["peaked", "shifted", "flat"])
def test_gradient_of_rows_whose_score_gradients_nearly_cancel(d, hq, hkv, lens, kind):
    # rows of several key tiles where one key takes almost all (out is nearly a value, and dp - D nearly 0), and values and
    # keys with a common part (out as large as a value, which cancels in ds): dq must not carry the rounding of out
    x = make("bf16", d, hq, hkv, lens, lens, seed=17)
    n, scale = sum(lens), 1 / math.sqrt(d)
    if kind == "peaked":  # the row's query is its own key, long enough for a share of 1 - 2^-10 or so
        t = 9.0 + math.log(n)
        kk = x["k"].double().repeat_interleave(hq // hkv, 1)
        x["q"] = (kk * (t / scale / (kk ** 2).sum(-1, keepdim=True))).bfloat16()
    if kind == "shifted":
        x["k"], x["v"] = (x[m] + 4 * ac.randn(3, 1, hkv, d, dtype=torch.bfloat16) for m in "kv")
    want, size = dq_bound(d, x, lens, scale)
    _, _, grads = run(params("bf16", d, hq, hkv), x, lens, lens)
    off, a, got = 0.0, 0, grads["q"].cpu().double()
    for i, m in enumerate(lens):
        for h in range(hq):
            off += float(((got[a:a + m, h] - want[i * hq + h]) ** 2).sum())
        a += m
    total = math.sqrt(sum(float((w ** 2).sum()) for w in want))
    assert math.sqrt(off) <= 1.2 * size + 2e-5 * total


@pytest.mark.parametrize("d,hq,hkv", [(64, 7, 1), (128, 5, 1), (64, 3, 3), (64, 14, 2)])
@pytest.mark.parametrize("lq,lk", [(241, 242), (560, 561), (259, 260), (300, 310), (300, 340), (300, 364)])
def test_gradient_of_a_first_tile_that_sees_few_keys_whole(d, hq, hkv, lq, lk):
    # two key tiles, but only one to 64 keys that every row of the query tile sees
    full_check("bf16", d, hq, hkv, [lq], [lk], scale=0.3, seed=lq + d)


def test_two_calls_at_once():
    # two layers' calls on two streams, a workspace each, beside each other: bit for bit what they are alone
    cases = [("bf16", 128, 8, 2, [900, 700]), ("bf16", 64, 4, 4, [1500])]
    alone, at_once, keep = [], [], []
    for dtype, d, hq, hkv, lens in cases:
        x = make(dtype, d, hq, hkv, lens, lens, seed=d)
        alone.append(run(params(dtype, d, hq, hkv), x, lens, lens, same=True))
        keep.append({n: t.cuda() for n, t in x.items()})
    tables = [ac.cu(c[4]) for c in cases]
    ws = [hla.alloc_attention_workspace(params(*c[:4]), sum(c[4]), sum(c[4]), len(c[4]), True) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        at_once = []
        for c, g, cu, w, s in zip(cases, keep, tables, ws, streams):
            out, lse = hla.attention(params(*c[:4]), g["q"], g["k"], g["v"], cu, ws=w, stream=s)
            at_once.append((out, lse, hla.attention_backward(params(*c[:4]), g["q"], g["k"], g["v"], out, lse, g["dout"],
                                                             cu, ws=w, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(alone, at_once):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            assert all(torch.equal(a[2][n], b[2][n]) for n in "qkv")


def test_inputs_of_another_stream_are_kept_until_it_is_done():
    # the caller lets go of its inputs while the call still waits behind other work on its stream
    x = make("bf16", 64, 4, 2, [300], [300])
    want, _, _ = run(params("bf16", 64, 4, 2), x, [300], [300], backward=False, same=True)
    cu, s = ac.cu([300]), torch.cuda.Stream()
    ws = hla.alloc_attention_workspace(params("bf16", 64, 4, 2), 300, 300, 1)
    a = torch.randn(4096, 4096, device="cuda")
    g = {n: x[n].cuda() for n in "qkv"}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(30):  # some milliseconds
            a @ a
    out, _ = hla.attention(params("bf16", 64, 4, 2), g["q"], g["k"], g["v"], cu, ws=ws, stream=s)
    del g
    junk = [torch.full_like(want, math.nan) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(junk) == 8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_padding_is_left_alone_and_kept_out(dtype, d):
    # rows behind the last sequence hold NaN: nothing of them is read into results, none of them is written
    q_lens, k_lens = [50, 77], [50, 140]
    x = make(dtype, d, 4, 2, q_lens, k_lens, pad_q=30, pad_k=41)
    nq, nk = sum(q_lens), sum(k_lens)
    for n in ("q", "dout"):
        x[n][nq:] = math.nan
    for n in ("k", "v"):
        x[n][nk:] = math.nan
    prm = params(dtype, d, 4, 2)
    g = {n: t.cuda() for n, t in x.items()}
    cq, ck = ac.cu(q_lens), ac.cu(k_lens)
    ws = hla.alloc_attention_workspace(prm, nq + 30, nk + 41, 2, backward=True)
    out, lse = torch.full_like(g["q"], 7.0), torch.full(g["q"].shape[:2], 7.0, device="cuda")
    grads = {n: torch.full_like(g[n], 7.0) for n in "qkv"}
    hla.attention(prm, g["q"], g["k"], g["v"], cq, ck, out=out, lse=lse, ws=ws)
    hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], cq, ck, grads=grads, ws=ws)
    assert hla.check_workspace_error(ws) == 0
    for t, n in ((out, nq), (lse, nq), (grads["q"], nq), (grads["k"], nk), (grads["v"], nk)):
        assert (t[n:] == 7.0).all()
    ref = ac.attention(x["q"][:nq], x["k"][:nk], x["v"][:nk], q_lens, k_lens, dout=x["dout"][:nq])
    check(dtype, d, x, ref, out, lse, grads, q_lens, k_lens)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_stay_out(dtype, d):
    # a sequence of NaN and infinities between two others changes nothing of them
    lens = [70, 90, 41]
    x = make(dtype, d, 2, 1, lens, lens)
    x["q"][70:160], x["k"][70:160], x["v"][70:160], x["dout"][70:160] = math.nan, math.inf, -math.inf, math.nan
    out, lse, grads = run(params(dtype, d, 2, 1), x, lens, lens)
    for a, b in ((0, 70), (160, 201)):
        y = {n: t[a:b] for n, t in x.items()}
        ref = ac.attention(y["q"], y["k"], y["v"], [b - a], [b - a], dout=y["dout"])
        check(dtype, d, y, ref, out[a:b], lse[a:b], {n: t[a:b] for n, t in grads.items()}, [b - a], [b - a])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 4, 1), (128, 3, 1), (64, 8, 1)])
@pytest.mark.parametrize("n,real", [(70, 50), (300, 130), (260, 255)])
def test_later_rows_stay_out(dtype, d, hq, hkv, n, real):
    """A padded batch: the rows from `real` on hold NaN and infinities, as keys, values and queries.  Nothing of them
    reaches the rows before them: outputs, lse and dq (dk and dv do get the padded rows' gradients: those that
    dout makes are kept to the rows before)."""
    x = make(dtype, d, hq, hkv, [n], [n], seed=n)
    clean = {m: t.clone() for m, t in x.items()}
    g = ac.gen(n)
    for m in ("q", "k", "v"):
        bad = torch.randint(0, 3, x[m][real:].shape, generator=g)
        x[m][real:] = torch.where(bad == 0, math.nan, torch.where(bad == 1, math.inf, -math.inf)).to(x[m].dtype)
    out, lse, grads = run(params(dtype, d, hq, hkv), x, [n], [n])
    y = {m: t[:real] for m, t in clean.items()}
    ref = ac.attention(y["q"], y["k"], y["v"], [real], [real], dout=y["dout"])
    ref[2].pop("k"), ref[2].pop("v")
    check(dtype, d, y, ref, out[:real], lse[:real], {"q": grads["q"][:real]}, [real], [real])
    assert torch.isnan(out[real:]).all() and torch.isnan(lse[real:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 8, 1)])
def test_infinite_and_nan_values_reach_the_rows_that_see_them(dtype, d, hq, hkv):
    n = 200
    x = make(dtype, d, hq, hkv, [n], [n], seed=7)
    places = {(3, 0): math.inf, (100, 5): math.nan, (130, d - 1): -math.inf, (150, 9): math.inf, (199, 1): math.nan}
    clean = x["v"].clone()
    for (key, col), value in places.items():
        x["v"][key, :, col] = value
        clean[key, :, col] = 0.0
    out, lse, _ = run(params(dtype, d, hq, hkv), x, [n], [n], backward=False)
    ref = ac.attention(x["q"], x["k"], clean, [n], [n])
    rows, want = torch.arange(n), ref[0].clone()
    for (key, col), value in places.items():
        want[rows >= key, :, col] = value
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    fine = want.isfinite()
    u = ac.EPS[TYPE[dtype][1]] / 2
    tol = (0.0 if dtype == "f32" else u) * ref[3]["out"] + 1e-4 * ref[3]["out"] + 1.01 * u * want.abs().nan_to_num(0, 0, 0)
    assert ((got - want).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("d,hq,hkv,n,real", [(64, 1, 1, 2500, 1700), (128, 8, 1, 900, 640), (64, 16, 1, 700, 130)])
def test_later_rows_stay_out_where_the_work_is_cut(d, hq, hkv, n, real):
    # keys cut into parts (long prompts of few heads), rows cut into parts (few key blocks): as above
    x = make("bf16", d, hq, hkv, [n], [n], seed=n)
    clean = {m: t.clone() for m, t in x.items()}
    g = ac.gen(n)
    for m in ("q", "k", "v"):
        bad = torch.randint(0, 3, x[m][real:].shape, generator=g)
        x[m][real:] = torch.where(bad == 0, math.nan, torch.where(bad == 1, math.inf, -math.inf)).to(x[m].dtype)
    out, lse, grads = run(params("bf16", d, hq, hkv), x, [n], [n])
    y = {m: t[:real] for m, t in clean.items()}
    ref = ac.attention(y["q"], y["k"], y["v"], [real], [real], dout=y["dout"])
    ref[2].pop("k"), ref[2].pop("v")
    check("bf16", d, y, ref, out[:real], lse[:real], {"q": grads["q"][:real]}, [real], [real])
    assert torch.isnan(out[real:]).all() and torch.isnan(lse[real:]).all()


def test_infinite_and_nan_values_reach_the_rows_that_see_them_in_parts():
    n, d = 2500, 64
    x = make("bf16", d, 1, 1, [n], [n], seed=7)
    places = {(3, 0): math.inf, (700, 5): math.nan, (1500, d - 1): -math.inf, (2400, 9): math.inf, (2499, 1): math.nan}
    clean = x["v"].clone()
    for (key, col), value in places.items():
        x["v"][key, :, col] = value
        clean[key, :, col] = 0.0
    out, lse, _ = run(params("bf16", d, 1, 1), x, [n], [n], backward=False)
    ref = ac.attention(x["q"], x["k"], clean, [n], [n])
    rows, want = torch.arange(n), ref[0].clone()
    for (key, col), value in places.items():
        want[rows >= key, :, col] = value
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    fine, u = want.isfinite(), ac.EPS[torch.bfloat16] / 2
    tol = (u + 1e-4) * ref[3]["out"] + 1.01 * u * want.abs().nan_to_num(0, 0, 0)
    assert ((got - want).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 1, 1), (128, 3, 1), (64, 4, 1), (128, 16, 1)])
@pytest.mark.parametrize("lq,lk,row", [(256, 257, 0), (300, 301, 130), (200, 391, 77), (200, 391, 7), (500, 430, 127), (300, 300, 40),
                                       (900, 1000, 33)])
def test_non_finite_rows_reach_no_further_than_the_keys_beside_theirs(dtype, d, hq, hkv, lq, lk, row):
    # infinities and NaN in one row's dout and q: dk and dv of the keys from 128 after the last one that it sees (fp32: from
    # the next one) are those of the other rows
    x = make(dtype, d, hq, hkv, [lq], [lk], seed=lq)
    clean = {n: t.clone() for n, t in x.items()}
    clean["q"][row], clean["dout"][row] = 0.0, 0.0  # adds nothing to dk and dv of keys that it does not see
    x["dout"][row], x["q"][row] = math.inf, math.nan
    out, lse, grads = run(params(dtype, d, hq, hkv), x, [lq], [lk])
    ref = ac.attention(clean["q"], clean["k"], clean["v"], [lq], [lk], dout=clean["dout"])
    first = min(lk, max(0, row + lk - lq + 1) + (0 if dtype == "f32" else 127))
    keep, rows = torch.arange(first, lk), torch.cat([torch.arange(row), torch.arange(row + 1, lq)])
    y = {n: clean[n] for n in clean}
    for part in (2, 3):
        for n in "kv":
            ref[part][n] = ref[part][n][keep]
        ref[part]["q"] = ref[part]["q"][rows]
    r_out, r_lse = ref[0][rows], ref[1][rows]
    ref[3]["out"] = ref[3]["out"][rows]
    u, L = ac.EPS[TYPE[dtype][1]] / 2, max(lk, lq * hq // hkv)
    S = float(y["q"].double().norm(dim=-1).max() * y["k"].double().norm(dim=-1).max()) / math.sqrt(d)
    fp, half = (2 * d * S + L + 32) * U32, 0.0 if dtype == "f32" else u  # as in the head of test_gpu_attention.py
    got = {"out": out.cpu()[rows], "q": grads["q"].cpu()[rows], "k": grads["k"].cpu()[keep], "v": grads["v"].cpu()[keep]}
    want = {"out": r_out, **ref[2]}
    for name, g in got.items():
        tol = ((3 if name in "qk" else 1) * half + 3 * fp) * ref[3][name] + 1.01 * u * want[name].abs()
        assert ((g.double() - want[name]).abs() <= tol).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 1), (128, 3, 3)])
def test_a_large_dout_reaches_the_keys_that_its_row_sees(dtype, d, hq, hkv):
    # one row's dout and q are so large that their products overflow: dk and dv of the keys behind it are the other rows'
    n, row = 300, 140
    x = make(dtype, d, hq, hkv, [n], [n], seed=3)
    clean = {m: t.clone() for m, t in x.items()}
    clean["q"][row], clean["dout"][row] = 0.0, 0.0
    big = torch.finfo(TYPE[dtype][1]).max
    for m in ("q", "dout"):
        x[m][row] = torch.where(ac.randn(9, *x[m][row].shape) < 0, -big, big).to(x[m].dtype)
    _, _, grads = run(params(dtype, d, hq, hkv), x, [n], [n])
    ref = ac.attention(clean["q"], clean["k"], clean["v"], [n], [n], dout=clean["dout"])
    u = ac.EPS[TYPE[dtype][1]] / 2
    S = float(clean["q"].double().norm(dim=-1).max() * clean["k"].double().norm(dim=-1).max()) / math.sqrt(d)
    fp, half = (2 * d * S + n * hq // hkv + 32) * U32, 0.0 if dtype == "f32" else u
    for name in "kv":
        want, mag = ref[2][name][row + 1:], ref[3][name][row + 1:]
        tol = ((3 if name == "k" else 1) * half + 3 * fp) * mag + 1.01 * u * want.abs()
        assert ((grads[name].cpu().double()[row + 1:] - want).abs() <= tol).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 1), (128, 3, 3), (64, 8, 1)])
def test_finite_rows_of_any_size_stay_out(dtype, d, hq, hkv):
    # the padding and the sequence in between hold the type's largest values, whose products overflow
    lens = [50, 90, 141]
    x = make(dtype, d, hq, hkv, lens, lens, pad_q=30, pad_k=41)
    big = torch.finfo(TYPE[dtype][1]).max
    for n in x:
        sign = torch.where(ac.randn(9, *x[n].shape) < 0, -big, big).to(x[n].dtype)
        x[n][50:140], x[n][281:] = sign[50:140], sign[281:]
    out, lse, grads = run(params(dtype, d, hq, hkv), x, lens, lens)
    for a, b in ((0, 50), (140, 281)):
        y = {n: t[a:b] for n, t in x.items()}
        ref = ac.attention(y["q"], y["k"], y["v"], [b - a], [b - a], dout=y["dout"])
        check(dtype, d, y, ref, out[a:b], lse[a:b], {n: t[a:b] for n, t in grads.items()}, [b - a], [b - a])


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_slices_of_a_fused_projection(dtype, d):
    hq, hkv, lens = 4, 2, [100, 45]
    x = make(dtype, d, hq, hkv, lens, lens)
    ref = run(params(dtype, d, hq, hkv), x, lens, lens)
    wide = torch.cat([x[n].flatten(1) for n in "qkv"], 1).cuda()
    parts = wide.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = (p.unflatten(1, (-1, d)) for p in parts)
    prm, c = params(dtype, d, hq, hkv), ac.cu(lens)
    out, lse = hla.attention(prm, q, k, v, c)
    grads = hla.attention_backward(prm, q, k, v, out, lse, x["dout"].cuda(), c)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    for n in "qkv":
        assert torch.equal(grads[n], ref[2][n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_32_bits(dtype):
    # tokens 2^27 elements apart, the last ones more than 2^32 from the first: the bits of dense rows
    hq, hkv, d, lens, t = 4, 2, 64, [15, 22], TYPE[dtype][1]
    x = make(dtype, d, hq, hkv, lens, lens)
    ref = run(params(dtype, d, hq, hkv), x, lens, lens, same=True)
    wide = torch.empty(sum(lens) << 27, dtype=t, device="cuda")
    q, k, v = (wide.as_strided((sum(lens), h, d), (1 << 27, d, 1), at)
               for h, at in ((hq, 0), (hkv, 1 << 20), (hkv, 1 << 26)))
    for n, y in zip("qkv", (q, k, v)):
        y.copy_(x[n])
    prm, c = params(dtype, d, hq, hkv), ac.cu(lens)
    out, lse = hla.attention(prm, q, k, v, c)
    grads = hla.attention_backward(prm, q, k, v, out, lse, x["dout"].cuda(), c)
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    assert all(torch.equal(grads[n], ref[2][n]) for n in "qkv")
    rp, pos = hla.RopeParams(hq, hkv, d, dtype=TYPE[dtype][0]), torch.arange(sum(lens), device="cuda")
    want = hla.rope(rp, q.contiguous(), k.contiguous(), pos)
    hla.rope(rp, q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_gradient_against_differences():
    # (f(x + e r) - f(x - e r)) / 2e of sum(dout out), summed in float64 from the fp32 layer's outputs, against
    # the gradient's product with r.  Outputs are off by about 50 u32 of their size each, so the quotient by
    # sqrt(n) 50 u32 / e; the third derivative adds about e^2.
    lens, d, hq, hkv = [40, 25], 64, 2, 1
    x = make("f32", d, hq, hkv, lens, lens, seed=20)
    prm, c = params("f32", d, hq, hkv), ac.cu(lens)
    _, _, grads = run(prm, x, lens, lens)
    e = 2.0 ** -6
    for i, n in enumerate("qkv"):
        r = ac.randn(40 + i, *x[n].shape, dtype=torch.float32)
        f = []
        for sign in (1, -1):
            y = {m: (t + sign * e * r if m == n else t).cuda() for m, t in x.items()}
            out, _ = hla.attention(prm, y["q"], y["k"], y["v"], c)
            f.append(float((out.double() * y["dout"].double()).sum()))
        step = float(((x[n] + e * r).double() - (x[n] - e * r).double()).flatten() @ grads[n].cpu().double().flatten()) / (2 * e)
        size = float(grads[n].double().norm()) * float(r.double().norm()) / math.sqrt(r.numel())
        assert abs((f[0] - f[1]) / (2 * e) - step) <= 20 * e * e * size + 1e-3 * size


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
def test_runs_agree_bit_for_bit_on_any_stream_and_in_a_graph(dtype, d):
    lens = [300, 1, 170]
    x = make(dtype, d, 4, 2, lens, lens)
    prm, c = params(dtype, d, 4, 2), ac.cu(lens)
    g = {n: t.cuda() for n, t in x.items()}
    ref = run(prm, x, lens, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = hla.attention(prm, g["q"], g["k"], g["v"], c, stream=side)
    grads = hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], c, stream=side)
    side.synchronize()
    assert torch.equal(out, ref[0]) and all(torch.equal(grads[n], ref[2][n]) for n in "qkv")
    ws = hla.alloc_attention_workspace(prm, sum(lens), sum(lens), 3, backward=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = hla.attention(prm, g["q"], g["k"], g["v"], c, ws=ws)
        g2 = hla.attention_backward(prm, g["q"], g["k"], g["v"], o2, l2, g["dout"], c, ws=ws)
    for _ in range(2):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, ref[0]) and all(torch.equal(g2[n], ref[2][n]) for n in "qkv")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_lens,k_lens,hq,hkv", [([3], [9001], 4, 2), ([40, 1], [2000, 3100], 8, 4), ([700, 0, 300], [700, 5, 300], 8, 1)])
def test_the_workspace_of_a_large_call_serves_smaller_ones(dtype, q_lens, k_lens, hq, hkv):
    # work cut into parts takes what parts the workspace has room for; with less than one part needs it is refused
    d, n = 64, len(q_lens)
    prm, x = params(dtype, d, hq, hkv), make(dtype, d, hq, hkv, q_lens, k_lens, seed=3)
    g, cq, ck = {m: t.cuda() for m, t in x.items()}, ac.cu(q_lens), ac.cu(k_lens)
    ref = ac.attention(x["q"], x["k"], x["v"], q_lens, k_lens, dout=x["dout"])
    own, least = ([hla.attention_workspace_bytes(prm, sum(q_lens), sum(k_lens), m, b) for b in (False, True)]
                  for m in (n, 1000))  # (of many sequences there are enough blocks: one part)
    large = [hla.attention_workspace_bytes(prm, 20000, 20000, 8, b) for b in (False, True)]
    assert all(a >= b for a, b in zip(large, least)) and (own != least or dtype == "f32")
    for share in (0.0, 0.3, 0.7, 1.0):
        size = [max(256, int(a + share * (b - a)) // 16 * 16) for a, b in zip(least, own)]
        ws = [torch.zeros(s + 64, dtype=torch.uint8, device="cuda") for s in size]
        for w, s in zip(ws, size):
            w[s:] = 123
        out, lse = hla.attention(prm, g["q"], g["k"], g["v"], cq, ck, ws=ws[0][:size[0]])
        grads = hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], cq, ck, ws=ws[1][:size[1]])
        check(dtype, d, x, ref, out, lse, grads, q_lens, k_lens)
        assert all((w[s:] == 123).all() and hla.check_workspace_error(w) == 0 for w, s in zip(ws, size))
    for fn, args in ((hla.attention, ()), (hla.attention_backward, (out, lse, g["dout"]))):
        with pytest.raises(hla.HlaError) as e:
            fn(prm, g["q"], g["k"], g["v"], *args, cq, ck, ws=ws[0][:240])
        assert e.value.status == hla.HLA_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("table", [[0, 50, 40, 100], [5, 50, 60, 100], [0, 50, 60, 300], [0, -7, 1 << 30, 20]])
def test_malformed_tables_are_flagged(dtype, table):
    x = make(dtype, 64, 2, 1, [100], [100])
    prm, g = params(dtype, 64, 2, 1), {n: t.cuda() for n, t in x.items()}
    c = torch.tensor(table, dtype=torch.int32, device="cuda")
    ws = hla.alloc_attention_workspace(prm, 100, 100, 3, backward=True)
    out, lse = hla.attention(prm, g["q"], g["k"], g["v"], c, ws=ws)
    assert hla.check_workspace_error(ws) != 0 and hla.check_workspace_error(ws) == 0
    hla.attention_backward(prm, g["q"], g["k"], g["v"], out, lse, g["dout"], c, ws=ws)
    assert hla.check_workspace_error(ws) != 0


@pytest.mark.parametrize("d,hq,hkv,q_lens,k_lens", [(128, 8, 1, [2300], [2300]), (64, 8, 1, [2300], [2300]),
                                                    (128, 3, 1, [1500, 900], [1500, 1900]), (64, 6, 1, [1011, 700], [1011, 3000])])
def test_longer_prompts_against_64_bit_on_the_gpu(d, hq, hkv, q_lens, k_lens):
    # many rounds of the rings of tiles, with a ragged last tile in every group of heads
    x = make("bf16", d, hq, hkv, q_lens, k_lens, seed=9)
    out, lse, grads = run(params("bf16", d, hq, hkv), x, q_lens, k_lens)
    y = {n: t.cuda() for n, t in x.items()}
    ref = ac.attention(y["q"], y["k"], y["v"], q_lens, k_lens, dout=y["dout"])
    ref = tuple({n: t.cpu() for n, t in r.items()} if isinstance(r, dict) else r.cpu() for r in ref)
    check("bf16", d, x, ref, out, lse, grads, q_lens, k_lens)
