"""GPU products with 4-bit weights against the 64-bit form: groups, offsets, types of rows, one token to several blocks,
odd widths, strides, infinities and NaN, and the quantisation."""
import pytest
import torch

import layer_cases as lc
from linearized_attention_rope_gb300 import hla

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = hla.DTYPE_F32, hla.DTYPE_BF16, hla.DTYPE_E4M3
TYPE = {F32: torch.float32, BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    build.build()


def weights(prm, offsets, seed=1):
    dt = TYPE[prm.dtype]
    w = torch.randint(0, 256, (prm.n_out, prm.n_in // 2), generator=lc.gen(seed), dtype=torch.uint8)
    shape = (prm.n_out, prm.n_in // prm.group)
    return w, torch.exp2(lc.randn(seed + 1, *shape)).to(dt), lc.randn(seed + 2, *shape).to(dt) if offsets else None


def rows(prm, n, seed=5):
    """x for the call (and its exponents), and the values in float64."""
    x = lc.randn(seed, n, prm.n_in)
    if prm.x_dtype != E4M3:
        x = x.to(TYPE[prm.dtype])
        return x, None, x.double()
    q = x.clamp(-300, 300).to(torch.float8_e4m3fn)
    groups = prm.n_in // prm.x_group if prm.x_group else 1
    e = torch.randint(110, 140, (n, groups), generator=lc.gen(seed + 1), dtype=torch.uint8)
    unit = torch.exp2(e.double() - 127).repeat_interleave(prm.n_in // groups, 1)
    return q.view(torch.uint8), e, q.double() * unit


def call(prm, x, e, w, s, o, **kw):
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return hla.linear4(prm, up(x), up(w), up(s), offsets=up(o), x_exp=up(e), **kw)


def check(prm, n, offsets):
    w, s, o = weights(prm, offsets)
    x, e, v = rows(prm, n)
    got = call(prm, x, e, w, s, o)
    y, err = lc.linear4(v, w, s, o, prm.group, 3 if x.dtype == torch.float32 else 1)
    lc.close(got, y, err)
    return got, (x, e, w, s, o)


@pytest.mark.parametrize("dtype,x_dtype,x_group", [(BF16, -1, 0), (F32, -1, 0), (BF16, E4M3, 32), (F32, E4M3, 0),
                                                   (BF16, E4M3, 128)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("n,n_in,n_out", [(1, 128, 16), (1, 4096, 40), (3, 1280, 1), (8, 384, 200), (9, 2048, 33),
                                          (16, 896, 100), (17, 128, 7), (33, 1152, 130), (61, 640, 31), (65, 256, 65),
                                          (130, 512, 50)])
def test_matches_64_bit(dtype, x_dtype, x_group, group, offsets, n, n_in, n_out):
    prm = hla.Linear4Params(n_in, n_out, group, dtype, x_dtype, x_group)
    got, args = check(prm, n, offsets)
    assert torch.equal(call(prm, *args), got)  # fixed order of sums


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_in,group", [(32, 32), (96, 32), (64, 64), (192, 64), (4128, 32)])
@pytest.mark.parametrize("n", [1, 20, 64])
def test_inputs_that_end_inside_a_tile(dtype, n_in, group, n):
    check(hla.Linear4Params(n_in, 24, group, dtype), n, True)


@pytest.mark.parametrize("n", [1, 5, 16, 40])
def test_wide(n):
    check(hla.Linear4Params(8192, 3001, 128, BF16, E4M3, 32), n, True)


def test_strided_and_unaligned_rows():
    prm = hla.Linear4Params(256, 48)
    w, s, o = weights(prm, False)
    wide = lc.randn(3, 11, 600, dtype=torch.bfloat16)
    for lo in (0, 8, 1, 3):
        x = wide[:, lo:lo + 256]
        got = hla.linear4(prm, wide.cuda()[:, lo:lo + 256], w.cuda(), s.cuda())
        lc.close(got, *lc.linear4(x.double(), w, s, None, 128, 1))
    odd = lc.randn(4, 7, 256 + 3, dtype=torch.bfloat16)  # rows that start anywhere
    got = hla.linear4(prm, odd.cuda()[:, :256], w.cuda(), s.cuda())
    lc.close(got, *lc.linear4(odd[:, :256].double(), w, s, None, 128, 1))


@pytest.mark.parametrize("n", [1, 9, 20])
@pytest.mark.parametrize("lo", [0, 1, 4, 8])
@pytest.mark.parametrize("offsets", [False, True])
def test_fp32_rows_of_a_wider_tensor(n, lo, offsets):
    # rows that start on 32, on 4 and on 16 bytes, a multiple of 32 bytes apart: no access may be wider than what they start on
    prm = hla.Linear4Params(384, 48, 64, F32)
    w, s, o = weights(prm, offsets)
    wide = lc.randn(3, n, 400, dtype=torch.float32)
    x, dev = wide[:, lo:lo + 384], wide.cuda()[:, lo:lo + 384]
    assert dev.data_ptr() % 32 == 4 * lo % 32
    got = hla.linear4(prm, dev, w.cuda(), s.cuda(), offsets=None if o is None else o.cuda())
    lc.close(got, *lc.linear4(x.double(), w, s, o, 64, 3))
    assert torch.equal(got, call(prm, x.contiguous(), None, w, s, o))


@pytest.mark.parametrize("n", [11, 24, 61, 65])
@pytest.mark.parametrize("dtype,x_dtype,x_group", [(BF16, -1, 0), (F32, -1, 0), (BF16, E4M3, 32), (F32, E4M3, 0)])
@pytest.mark.parametrize("width", [600, 603])
def test_rows_of_a_wider_tensor(n, dtype, x_dtype, x_group, width):
    # up to sixteen rows and more, on 16 bytes and off them, a multiple of 16 bytes apart and not
    prm = hla.Linear4Params(320, 48, 64, dtype, x_dtype, x_group)
    w, s, o = weights(prm, True)
    x, e, v = rows(prm, n)
    want = call(prm, x, e, w, s, o)
    lc.close(want, *lc.linear4(v, w, s, o, 64, 3))
    for lo in (0, 1, 4, 8, 16):
        wide = torch.zeros(n, width, dtype=x.dtype, device="cuda")
        wide[:, lo:lo + 320] = x.cuda()
        got = hla.linear4(prm, wide[:, lo:lo + 320], w.cuda(), s.cuda(), offsets=o.cuda(), x_exp=None if e is None else e.cuda())
        assert torch.equal(got, want), lo


@pytest.mark.parametrize("n", [24, 61, 65])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offsets", [False, True])
def test_infinities_and_nan_stay_with_their_token_of_many(n, dtype, offsets):
    prm = hla.Linear4Params(256, 140, 64, dtype)
    w, s, o = weights(prm, offsets)
    x, _, v = rows(prm, n)
    bad = x.clone()
    at = [0, 7, n - 8, n - 1]
    bad[0, 100], bad[7, 5], bad[n - 8], bad[n - 1, 255] = float("nan"), float("inf"), torch.finfo(x.dtype).max, float("-inf")
    got = call(prm, bad, None, w, s, o)
    keep = [i for i in range(n) if i not in at]
    y, err = lc.linear4(v, w, s, o, 64, 3)
    lc.close(got[keep], y[keep], err[keep])
    assert got[0].isnan().all() and not got[[7, n - 1]].isfinite().any()


@pytest.mark.parametrize("n", [3, 11, 24, 61])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("offsets", [False, True])
def test_the_largest_rows(n, dtype, group, offsets):
    # values of up to 2^118, all of one sign, through weights of one sign: the largest sums that a group can have
    prm = hla.Linear4Params(384, 40, group, dtype)
    _, s, o = weights(prm, offsets)
    w = torch.zeros(40, 192, dtype=torch.uint8)  # q - 8 = -8
    w[20:] = 0xff                                # 7
    s, o = s * 2.0 ** -20, o if o is None else o * 2.0 ** -20
    big = 2.0 ** 118 * (1 - torch.finfo(TYPE[dtype]).eps)
    x = torch.full((n, 384), big, dtype=torch.float64)
    x[1] *= -1
    x[2] = big * torch.rand(384, generator=lc.gen(3), dtype=torch.float64)
    x = x.to(TYPE[dtype])
    lc.close(call(prm, x, None, w, s, o), *lc.linear4(x.double(), w, s, o, group, 3))


def test_infinities_and_nan_stay_with_their_token():
    for dtype in (BF16, F32):
        prm = hla.Linear4Params(256, 40, dtype=dtype)
        w, s, o = weights(prm, True)
        x, _, v = rows(prm, 12)
        bad = x.clone()
        bad[3, 100], bad[7, 5], bad[9] = float("nan"), float("inf"), torch.finfo(x.dtype).max
        got = call(prm, bad, None, w, s, o)
        keep = [i for i in range(12) if i not in (3, 7, 9)]
        y, err = lc.linear4(v, w, s, o, 128, 3)
        lc.close(got[keep], y[keep], err[keep])
        assert got[3].isnan().all() and not got[7].isfinite().any()


@pytest.mark.parametrize("n,dtype", [(40, BF16), (61, F32), (129, BF16)])
def test_many_rows_in_a_graph_and_on_two_streams(n, dtype):
    prm = hla.Linear4Params(1088, 700, 64, dtype)
    w, s, o = weights(prm, True)
    xs = [rows(prm, n, seed)[0].cuda() for seed in (5, 8)]
    w, s, o = w.cuda(), s.cuda(), o.cuda()
    want = [hla.linear4(prm, x, w, s, offsets=o) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, stream in zip(xs, streams):
        stream.wait_stream(torch.cuda.current_stream())
        got.append(hla.linear4(prm, x, w, s, offsets=o, stream=stream))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, ws = xs[0].clone(), hla.alloc_linear4_workspace(prm, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hla.linear4(prm, x, w, s, offsets=o, ws=ws)
    for i in (0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])


def test_no_tokens():
    prm = hla.Linear4Params(128, 8)
    w, s, _ = weights(prm, False)
    assert hla.linear4(prm, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), w.cuda(), s.cuda()).shape == (0, 8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offsets", [False, True])
def test_quantise(dtype, group, offsets):
    prm = hla.Linear4Params(384, 50, group, dtype)
    weight = lc.randn(1, 50, 384, dtype=TYPE[dtype])
    weight[3, :group] = 0
    weight[4, :group] = 0.5
    w, s, o = hla.linear4_quantize(prm, weight.cuda(), offsets)
    assert (o is not None) == offsets
    y, _ = lc.unpack4(w.cpu(), s.cpu(), None if o is None else o.cpu(), group)
    # half a step, what the scale's rounding takes from the 7 (8) steps, and the offset's own rounding
    g = weight.double().reshape(50, -1, group)
    u = lc.EPS[TYPE[dtype]] / 2
    if offsets:
        step = (g.amax(-1) - g.amin(-1)) / 15
        slack = u * (16 * step + g.abs().amax(-1) + 8 * step)
        assert s.cpu().double().sub(step).abs().max() <= 2 * u * step.max() + 3 * lc.U * g.abs().max()
    else:
        step = g.abs().amax(-1) / 7
        slack = u * 8 * step
        assert (s.cpu().double() - step).abs().max() <= (u + 2 * lc.U) * step.max()
    off = (y.reshape(g.shape) - g).abs()
    assert (off <= (step / 2 + slack + 20 * lc.U * g.abs().amax(-1))[..., None]).all()
    x = lc.randn(2, 4, 384, dtype=TYPE[dtype])
    q = [t if t is None else t.cpu() for t in (w, s, o)]
    lc.close(hla.linear4(prm, x.cuda(), w, s, offsets=o), *lc.linear4(x.double(), *q, group, 3))


def test_graph_and_stream():
    prm = hla.Linear4Params(1024, 512, x_dtype=E4M3, x_group=32)
    w, s, o = weights(prm, True)
    x, e, _ = rows(prm, 9)
    w, s, o, x, e = (t.cuda() for t in (w, s, o, x, e))
    want = hla.linear4(prm, x, w, s, offsets=o, x_exp=e)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hla.linear4(prm, x, w, s, offsets=o, x_exp=e, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    ws = hla.alloc_linear4_workspace(prm, 9)
    with torch.cuda.graph(graph):
        out = hla.linear4(prm, x, w, s, offsets=o, x_exp=e, ws=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
