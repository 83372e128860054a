"""The operators together, as a layer runs them: a decode step of a recurrent layer between frozen 4-bit projections, its
training step, and the norm of q's and k's heads in front of rotary positions and attention."""
import pytest
import torch

import layer_cases as lc
from linearized_attention_rope_gb300 import hla

pytestmark = pytest.mark.gpu
E4M3 = hla.DTYPE_E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    build.build()


def rel(got, ref):
    return float((got.cpu().double() - ref).norm() / ref.norm())


def test_decode_step_of_a_recurrent_layer():
    # residual stream -> norm to 8 bits -> gates and inputs -> recurrence -> projection -> next norm with the residual,
    # six steps captured once and replayed, against the same in float64 from the same weights
    n, d, c, steps = 5, 256, 384, 6
    norm = hla.NormParams(d, out_dtype=E4M3, group=32)
    up = hla.Linear4Params(d, 2 * c, group=64, x_dtype=E4M3, x_group=32)
    down = hla.Linear4Params(c, d, group=128)
    rec = hla.RecurrenceParams(c, gate_dtype=hla.DTYPE_BF16)
    bf = lambda *a: lc.randn(*a, dtype=torch.bfloat16).cuda()  # noqa: E731
    q_up = hla.linear4_quantize(up, bf(1, 2 * c, d) / 16, True)
    q_down = hla.linear4_quantize(down, bf(2, d, c) / 20)
    weight, stream = bf(3, d).abs(), bf(4, n, d)
    branch, h = torch.zeros_like(stream), torch.zeros(n, c, device="cuda")
    fresh = bf(5, steps, n, d)
    ws = hla.alloc_linear4_workspace(up, n)

    def step():
        y = hla.rms_norm(norm, branch, weight=weight, residual=stream, sum=stream)
        p = hla.linear4(up, y.out, q_up[0], q_up[1], offsets=q_up[2], x_exp=y.exp, ws=ws)
        p[:, :c].abs_().neg_()
        o = hla.recurrence_step(rec, p[:, :c], p[:, c:], h)
        hla.linear4(down, o, q_down[0], q_down[1], out=branch)

    before = [t.clone() for t in (branch, h, stream)]
    step()
    for t, b in zip((branch, h, stream), before):
        t.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, b in zip((branch, h, stream), before):
        t.copy_(b)
    dq = lambda q, g: lc.unpack4(*[None if t is None else t.cpu() for t in q], g)[0]  # noqa: E731
    w_up, w_down = dq(q_up, 64), dq(q_down, 128)
    bf16 = lambda t: t.to(torch.bfloat16).double()  # noqa: E731

    def to_8_bits(y):
        y = y.reshape(n, -1, 32)
        unit = torch.exp2(torch.ceil(torch.log2(y.abs().amax(-1, keepdim=True) / 448)))
        return ((y / unit).to(torch.float8_e4m3fn).double() * unit).reshape(n, -1)

    s64, b64, h64 = stream.cpu().double(), torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, c, dtype=torch.float64)
    for t in range(steps):
        stream.add_(fresh[t])
        s64 = bf16(s64 + fresh[t].cpu().double())
        graph.replay()
        s64 = bf16(s64 + b64)
        y, _ = lc.norm(s64, weight.cpu().double(), 1e-6, 0.0)
        p = bf16(to_8_bits(y) @ w_up.T)
        h64 = torch.exp(-p[:, :c].abs()) * h64 + p[:, c:]
        b64 = bf16(bf16(h64) @ w_down.T)
    # The form above rounds where the layer does.  What is left are fp32's roundings (about 40 U) that turn one of bf16's:
    # of one value in 40 U / 2^-9, about 1e-3, by 2^-8 of it, so 2^-8 sqrt(1e-3) = 1.3e-4 of a tensor, at four places a
    # step; a value so changed turns an 8-bit rounding in one of 16 cases, by 2^-4: 2^-4 sqrt(1e-3 / 16) = 5e-4.  Six steps
    # of both, added up: 6 (4 x 1.3e-4 + 5e-4) = 6e-3.
    assert rel(stream, s64) < 6e-3 and rel(h, h64) < 6e-3 and rel(branch, b64) < 6e-3


def test_training_step_of_a_recurrent_layer():
    # norm -> projections (plain products) -> recurrence and back, fp32, against autograd in float64
    lens, d, c = [70, 1, 200], 128, 192
    n, cu = sum(lens), lc.cu(lens)
    norm, rec = hla.NormParams(d, dtype=hla.DTYPE_F32), hla.RecurrenceParams(c, dtype=hla.DTYPE_F32)
    f = lambda *a: lc.randn(*a, dtype=torch.float32)  # noqa: E731
    x, w, wg, wx, dout = f(1, n, d), 1 + 0.1 * f(2, d), f(3, d, c) / 16, f(4, d, c) / 16, f(5, n, c)
    leaves = [t.double().requires_grad_() for t in (x, w, wg, wx)]
    x64, w64, wg64, wx64 = leaves
    y64 = x64 * (x64.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w64
    g64, v64, outs = -(y64 @ wg64).square(), y64 @ wx64, []
    at = lc.offsets(lens)
    for s in range(len(lens)):
        h = torch.zeros(c, dtype=torch.float64)
        for t in range(at[s], at[s + 1]):
            h = g64[t].exp() * h + v64[t]
            outs.append(h)
    (torch.stack(outs) * dout.double()).sum().backward()

    xd, wd, wgd, wxd, dod = (t.cuda() for t in (x, w, wg, wx, dout))
    y = hla.rms_norm(norm, xd, weight=wd).out
    z = y @ wgd
    g, v = -z.square(), y @ wxd
    states = hla.alloc_recurrence_states(rec, n)
    out, _ = hla.recurrence(rec, g, v, cu, states=states)
    grads = hla.recurrence_backward(rec, g, v, states, dod, cu)
    dz = -2 * z * grads["g"]
    dy = dz @ wgd.T + grads["x"] @ wxd.T
    dx, dw = hla.rms_norm_backward(norm, xd, dy, weight=wd)
    # fp32 throughout: sums of at most 200 terms, a few hundred roundings of 6e-8
    assert rel(out, torch.stack(outs).detach()) < 1e-5
    for got, leaf in ((dx, x64), (dw, w64), (y.T @ dz, wg64), (y.T @ grads["x"], wx64)):
        assert rel(got, leaf.grad) < 2e-5


def test_heads_normed_before_rotary_attention():
    # q and k of a fused projection: a norm per head, rotary positions in place, attention
    n, hq, hkv, d = 200, 4, 2, 64
    wide = lc.randn(1, n, (hq + 2 * hkv) * d, dtype=torch.float32)
    wq, wk = 1 + 0.2 * lc.randn(2, d, dtype=torch.float32), 1 + 0.2 * lc.randn(3, d, dtype=torch.float32)
    dev = wide.cuda()
    q, k, v = (t.view(n, -1, d) for t in dev.split([hq * d, hkv * d, hkv * d], 1))
    f32 = hla.DTYPE_F32
    q = hla.rms_norm(hla.NormParams(d, n_heads=hq, dtype=f32), q, weight=wq.cuda()).out
    k = hla.rms_norm(hla.NormParams(d, n_heads=hkv, dtype=f32), k, weight=wk.cuda()).out
    rope = hla.RopeParams(hq, hkv, d, dtype=f32)
    hla.rope(rope, q, k, torch.arange(n, device="cuda"), q_out=q, k_out=k)
    out, _ = hla.attention(hla.AttnParams(hq, hkv, d, dtype=f32), q, k, v, lc.cu([n]))
    import attention_cases as ac
    r = wide.double()
    q64, k64, v64 = (t.reshape(n, -1, d) for t in r.split([hq * d, hkv * d, hkv * d], 1))
    freq, gain = hla.rope_frequencies(rope)
    pos = torch.arange(n)
    q64 = ac.rope(lc.norm(q64, wq.double(), 1e-6, 0.0)[0], pos, freq, gain, d, False)
    k64 = ac.rope(lc.norm(k64, wk.double(), 1e-6, 0.0)[0], pos, freq, gain, d, False)
    kk, vv = k64.repeat_interleave(hq // hkv, 1), v64.repeat_interleave(hq // hkv, 1)
    x = torch.einsum("qhd,khd->hqk", q64, kk) / d ** 0.5
    p = x.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf")).softmax(-1)
    # scores up to about 30 off by 30 roundings of fp32 each
    assert rel(out, torch.einsum("hqk,khd->qhd", p, vv)) < 1e-4
