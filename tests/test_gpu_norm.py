"""GPU root-mean-square norms against the 64-bit form: widths from one value to rows that pass a block's registers, heads,
8-bit rows, strides, in place, infinities and NaN, gradients, graphs and streams."""
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


def shape(prm, n):
    return (n, prm.n_cols) if prm.n_heads == 1 else (n, prm.n_heads, prm.n_cols)


def inputs(prm, n, seed=1):
    dt = TYPE[prm.dtype]
    x = lc.randn(seed, *shape(prm, n)) * torch.exp2(lc.randn(seed + 1, n, *[1] * (len(shape(prm, n)) - 1)))
    return x.to(dt), lc.randn(seed + 2, *shape(prm, n), dtype=dt), (1 + 0.3 * lc.randn(seed + 3, prm.n_cols)).to(dt)


# cols, heads, tokens: a value, odd widths, a warp's, blocks of one, two and four pieces a thread, sixteen single values,
# rows past the registers
SIZES = [(1, 1, 3), (7, 1, 33), (64, 8, 5), (128, 3, 130), (100, 1, 9), (256, 1, 1), (1000, 2, 17), (1024, 1, 40),
         (2056, 1, 3), (4096, 1, 65), (4100, 1, 5), (5120, 1, 700), (8191, 1, 3), (16384, 1, 4), (17000, 1, 2),
         (33001, 1, 2), (65536, 1, 2)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", SIZES)
@pytest.mark.parametrize("residual,weight,offset", [(True, True, 0.0), (False, True, 1.0), (True, False, 0.0)])
def test_norm_matches_64_bit(dtype, cols, heads, n, residual, weight, offset):
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype, eps=1e-5, offset=offset)
    x, r, w = inputs(prm, n)
    got = hla.rms_norm(prm, x.cuda(), weight=w.cuda() if weight else None, residual=r.cuda() if residual else None)
    s = (x + r) if residual else x
    assert got.exp is None and (got.sum is None) == (not residual)
    if residual:  # one rounding of an fp32 sum
        assert torch.equal(got.sum.cpu(), s)
    y, err = lc.norm(s.double(), w.double() if weight else None, 1e-5, offset)
    lc.close(got.out, y, err)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n,group", [(32, 1, 5, 32), (64, 4, 9, 32), (128, 2, 33, 128), (128, 1, 7, 0),
                                                (160, 1, 6, 32), (4096, 1, 64, 32), (4096, 1, 3, 128), (5120, 1, 9, 0),
                                                (16, 1, 2, 0), (16384, 1, 3, 128), (33024, 1, 2, 128), (40000, 1, 2, 32),
                                                (40000, 1, 2, 0)])
def test_norm_to_8_bits(dtype, cols, heads, n, group):
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype, out_dtype=E4M3, group=group)
    x, r, w = inputs(prm, n)
    x[0] = 0
    r[0] = 0  # a row of zeros: exponent byte 0
    got = hla.rms_norm(prm, x.cuda(), weight=w.cuda(), residual=r.cuda())
    s = x + r
    assert torch.equal(got.sum.cpu(), s) and got.out.dtype == torch.uint8
    y, err = lc.norm(s.double(), w.double(), 1e-6, 0.0)
    assert lc.eight(y, err, got.out, got.exp, group) == (True, True, True)
    assert got.exp[0].max() == 0 and (got.out[0] & 127).max() == 0  # a negative weight makes -0


def test_8_bit_rows_with_infinities_and_nan():
    # an infinity makes the mean infinite: the row's finite values become 0 and it NaN; a NaN makes the whole row NaN
    for group in (0, 32):
        prm = hla.NormParams(64, dtype=F32, out_dtype=E4M3, group=group)
        x = torch.ones(3, 64)
        x[0, 5], x[1, 7] = float("inf"), float("nan")
        got = hla.rms_norm(prm, x.cuda())
        v = got.out.view(torch.float8_e4m3fn).float().cpu()
        assert v[0, 5].isnan() and v[0].nan_to_num(0).abs().max() == 0
        assert v[1].isnan().all() and v[2].isfinite().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [128, 1000, 5120, 8191, 33001])
def test_rows_at_the_ends_of_fp32(dtype, cols):
    # rows whose sum of squares is just below 2^128, just above 2^-126 a value without eps, and past 2^128
    prm = hla.NormParams(cols, dtype=dtype, eps=0.0)
    x = lc.randn(1, 3, cols).clamp(-4, 4) / 4 + torch.where(lc.randn(2, 3, cols) > 0, 1.0, -1.0)  # 1 in size, 2 at most
    x[0] *= 0.4 * 2.0 ** 64 / cols ** 0.5
    x[1] *= 2.0 ** -62
    x[2] *= 2.0 ** 66
    x = x.to(TYPE[dtype])
    y, err = lc.norm(x.double(), None, 0.0, 0.0)
    got = hla.rms_norm(prm, x.cuda()).out
    lc.close(got[:2], y[:2], err[:2])
    assert float(got[2].abs().max()) == 0.0


def test_strided_and_unaligned_rows():
    # q, k and v of one fused projection: norm of q's and k's heads in place of their slices, and rows one value in
    wide = lc.randn(1, 50, 14 * 64, dtype=torch.bfloat16).cuda()
    for lo, heads in ((0, 8), (8, 4), (12, 1)):
        prm = hla.NormParams(64, n_heads=heads)
        x = wide[:, lo * 64:(lo + heads) * 64]
        x = x.view(50, heads, 64) if heads > 1 else x
        y, err = lc.norm(x.cpu().double(), None, 1e-6, 0.0)
        lc.close(hla.rms_norm(prm, x).out, y, err)
    for dtype in (F32, BF16):
        flat = lc.randn(2, 20 * 301 + 1, dtype=TYPE[dtype]).cuda()
        x = flat[1:].view(20, 301)[:, :300]
        y, err = lc.norm(x.cpu().double(), None, 1e-6, 0.0)
        lc.close(hla.rms_norm(hla.NormParams(300, dtype=dtype), x).out, y, err)
        got, _ = hla.rms_norm_backward(hla.NormParams(300, dtype=dtype), x, x.contiguous())
        dx, err, _, _ = lc.norm_grad(x.cpu().double(), None, x.cpu().double(), None, 1e-6, 0.0)
        lc.close(got, dx, err)
    with pytest.raises(hla.HlaError):  # 8-bit rows start on 16 bytes
        hla.rms_norm(hla.NormParams(64, out_dtype=E4M3, group=32), wide[:, 1:65])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", [(128, 1, 9), (128, 3, 33), (1024, 1, 4000), (4096, 1, 2000), (5120, 1, 5), (301, 1, 7),
                                          (17000, 1, 2), (33001, 1, 2)])
@pytest.mark.parametrize("lo", [0, 8, 1])
def test_a_residual_of_a_wider_tensor(dtype, cols, heads, n, lo):
    # the residual, and then x as well, as slices; into the layer's type and into 8 bits where the slices lie on 16 bytes
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype)
    x, r, w = inputs(prm, n)
    want = hla.rms_norm(prm, x.cuda(), weight=w.cuda(), residual=r.cuda())
    y, err = lc.norm((x + r).double(), w.double(), 1e-6, 0.0)
    lc.close(want.out, y, err)

    def part(t, pad):
        wide = torch.full((n, heads * cols + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, lo:lo + heads * cols] = t.reshape(n, -1).cuda()
        return wide[:, lo:lo + heads * cols].view(shape(prm, n))

    for a, b in ((x.cuda(), part(r, 16)), (part(x, 32), part(r, 16)), (part(x, 32), r.cuda())):
        got = hla.rms_norm(prm, a, weight=w.cuda(), residual=b)
        assert torch.equal(got.sum, want.sum)
        lc.close(got.out, y, err)
        if lo != 1 and cols % 128 == 0:
            eight = hla.NormParams(cols, n_heads=heads, dtype=dtype, out_dtype=E4M3, group=32)
            got = hla.rms_norm(eight, a, weight=w.cuda(), residual=b)
            assert torch.equal(got.sum, want.sum) and lc.eight(y, err, got.out, got.exp, 32) == (True, True, True)


@pytest.mark.parametrize("cols", [128, 4096, 8191, 33001])
def test_in_place(cols):
    prm = hla.NormParams(cols)
    x, r, w = (t.cuda() for t in inputs(prm, 20))
    ref = hla.rms_norm(prm, x, weight=w, residual=r)
    for target in ("residual", "x"):
        a, b = x.clone(), r.clone()
        got = hla.rms_norm(prm, a, weight=w, residual=b, sum=b if target == "residual" else a)
        assert torch.equal(got.out, ref.out) and torch.equal(b if target == "residual" else a, ref.sum)
    a, b = x.clone(), r.clone()
    got = hla.rms_norm(prm, a, weight=w, residual=b, sum=b, out=a)  # the stream and the branch, both in place
    assert torch.equal(a, ref.out) and torch.equal(b, ref.sum)
    a = x.clone()
    hla.rms_norm(prm, a, weight=w, out=a)
    assert torch.equal(a, hla.rms_norm(prm, x, weight=w).out)
    dx, dw = hla.rms_norm_backward(prm, x, r, weight=w, dsum=ref.out)
    for target in (0, 1):
        a, b = r.clone(), ref.out.clone()
        got, gw = hla.rms_norm_backward(prm, x, a, weight=w, dsum=b, dx=(a, b)[target])
        assert torch.equal(got, dx) and torch.equal(gw, dw)


# more rows than the blocks that stay take at three each: one, two and four pieces a thread
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,n", [(264, 1000), (2056, 1300), (4096, 1001), (8200, 960), (16384, 930)])
@pytest.mark.parametrize("residual,group", [(True, -1), (False, -1), (True, 0), (True, 32)])
def test_many_rows(dtype, cols, n, residual, group):
    if group >= 0:  # 8-bit rows are whole groups, on 16 bytes
        cols -= cols % 32
    prm = hla.NormParams(cols, dtype=dtype, out_dtype=-1 if group < 0 else E4M3, group=max(group, 0))
    x, r, w = inputs(prm, n)
    s = x + r if residual else x
    y, err = lc.norm(s.double(), w.double(), 1e-6, 0.0)
    a, b = x.cuda(), r.cuda()
    got = hla.rms_norm(prm, a, weight=w.cuda(), residual=b if residual else None)
    if residual:
        assert torch.equal(got.sum.cpu(), s)
    if group >= 0:
        assert lc.eight(y, err, got.out, got.exp, group) == (True, True, True)
        return
    lc.close(got.out, y, err)
    wide = torch.zeros(n, cols + 64, dtype=TYPE[dtype], device="cuda")  # rows of a wider tensor, the same values
    wide[:, 64:] = a
    again = hla.rms_norm(prm, wide[:, 64:], weight=w.cuda(), residual=b if residual else None)
    assert torch.equal(again.out, got.out)
    if residual:  # the stream and the branch, both in place
        hla.rms_norm(prm, a, weight=w.cuda(), residual=b, sum=b, out=a)
        assert torch.equal(a, got.out) and torch.equal(b, got.sum)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", [(512, 3, 1100), (1024, 2, 700), (128, 5, 900)])
def test_many_heads_of_a_wider_tensor(dtype, cols, heads, n):
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype)
    x, _, w = inputs(prm, n)
    dout = lc.randn(7, *shape(prm, n), dtype=TYPE[dtype])
    wide = torch.zeros(n, (heads + 2) * cols, dtype=TYPE[dtype], device="cuda")
    wide[:, cols:-cols] = x.reshape(n, -1).cuda()
    part = wide[:, cols:-cols].view(n, heads, cols)
    y, err = lc.norm(x.double(), w.double(), 1e-6, 0.0)
    lc.close(hla.rms_norm(prm, part, weight=w.cuda()).out, y, err)
    dx, dw = hla.rms_norm_backward(prm, part, dout.cuda(), weight=w.cuda())
    ref = lc.norm_grad(x.double(), w.double(), dout.double(), None, 1e-6, 0.0)
    lc.close(dx, ref[0], ref[1])
    lc.close(dw, ref[2], ref[3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", SIZES + [(128, 32, 600), (64, 1, 20011)])
@pytest.mark.parametrize("dsum,weight,offset", [(True, True, 0.0), (False, True, 1.0), (True, False, 0.0)])
def test_norm_gradient_matches_64_bit(dtype, cols, heads, n, dsum, weight, offset):
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype, eps=1e-5, offset=offset)
    x, ds, w = inputs(prm, n)
    dout = lc.randn(7, *shape(prm, n), dtype=TYPE[dtype])
    dx, dw = hla.rms_norm_backward(prm, x.cuda(), dout.cuda(), weight=w.cuda() if weight else None,
                                   dsum=ds.cuda() if dsum else None)
    ref = lc.norm_grad(x.double(), w.double() if weight else None, dout.double(), ds.double() if dsum else None, 1e-5, offset)
    lc.close(dx, ref[0], ref[1])
    assert (dw is None) == (not weight)
    if weight:
        lc.close(dw, ref[2], ref[3])
        again = hla.rms_norm_backward(prm, x.cuda(), dout.cuda(), weight=w.cuda(), dsum=ds.cuda() if dsum else None)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # fixed order of sums


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", [(128, 1, 40), (100, 1, 9), (1000, 1, 33), (1024, 1, 300), (5120, 1, 200), (16384, 1, 3),
                                          (33001, 1, 2)])
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("size,grad", [(2e-18, 1e6), (1e16, 1e-9)])
def test_gradient_of_tiny_and_huge_rows_without_eps(dtype, cols, heads, n, dsum, size, grad):
    # rows of 2e-18 and 1e16 (their squares are normal numbers) and gradients that lie along them: mean(w dy x) / rms^3 leaves
    # fp32's range, the gradient does not.  Every third row is an ordinary one
    prm = hla.NormParams(cols, dtype=dtype, eps=0.0)
    unit, mixed = lc.randn(1, n, cols), (torch.arange(n) % 3 == 2)[:, None]
    size, grad = (torch.where(mixed, 1.0, torch.tensor(y, dtype=torch.float64)) for y in (size, grad))
    x, dout = (size * unit).to(TYPE[dtype]), (grad * (unit + lc.randn(2, n, cols))).to(TYPE[dtype])
    w, ds = (1 + 0.3 * lc.randn(3, cols)).to(TYPE[dtype]), (grad / size * lc.randn(4, n, cols)).to(TYPE[dtype])
    dx, dw = hla.rms_norm_backward(prm, x.cuda(), dout.cuda(), weight=w.cuda(), dsum=ds.cuda() if dsum else None)
    ref = lc.norm_grad(x.double(), w.double(), dout.double(), ds.double() if dsum else None, 0.0, 0.0)
    lc.close(dx, ref[0], ref[1])
    lc.close(dw, ref[2], ref[3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n,pad", [(100, 1, 9, 0), (7, 1, 5, 0), (33, 1, 2, 0), (128, 3, 7, 128), (64, 1, 33, 8), (1000, 1, 3, 1)])
def test_gradient_without_eps(dtype, cols, heads, n, pad):
    # rows that do not fill the last block, dense or slices of a wider tensor: what lies past the last row has no size
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype, eps=0.0)
    x, _, w = inputs(prm, n)
    dout = lc.randn(7, *shape(prm, n), dtype=TYPE[dtype])
    wide = torch.zeros(n, heads * cols + pad, dtype=TYPE[dtype], device="cuda")
    wide[:, pad:] = x.reshape(n, -1).cuda()
    dx, dw = hla.rms_norm_backward(prm, wide[:, pad:].view(shape(prm, n)), dout.cuda(), weight=w.cuda())
    ref = lc.norm_grad(x.double(), w.double(), dout.double(), None, 0.0, 0.0)
    lc.close(dx, ref[0], ref[1])
    lc.close(dw, ref[2], ref[3])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,heads,n", [(7, 1, 33), (128, 3, 130), (1024, 1, 40), (5120, 1, 700), (33001, 1, 2)])
def test_gradient_of_a_frozen_norm(dtype, cols, heads, n):
    # dx alone: the same bits, and nothing written to a workspace
    prm = hla.NormParams(cols, n_heads=heads, dtype=dtype)
    x, ds, w = (t.cuda() for t in inputs(prm, n))
    dout = lc.randn(7, *shape(prm, n), dtype=TYPE[dtype]).cuda()
    want, _ = hla.rms_norm_backward(prm, x, dout, weight=w, dsum=ds)
    ws = torch.full((hla.norm_workspace_bytes(prm),), 7, dtype=torch.uint8, device="cuda")
    dx, dw = hla.rms_norm_backward(prm, x, dout, weight=w, dsum=ds, ws=ws, need_dweight=False)
    assert dw is None and torch.equal(dx, want) and bool((ws == 7).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dx, dw = hla.rms_norm_backward(prm, x, dout, weight=w, dsum=ds, stream=side, need_dweight=False)
    side.synchronize()
    assert dw is None and torch.equal(dx, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,n", [(7, 20000), (130, 8000), (512, 5000), (1025, 1500), (2560, 1500), (2736, 1200), (4100, 900),
                                    (5120, 700), (8191, 500), (16384, 400), (16390, 400), (33001, 320)])
def test_gradient_stays_in_its_workspace(dtype, cols, n):
    # as many rows as keep every block: their sums fit what the size is given as, and nothing behind it is written
    prm = hla.NormParams(cols, dtype=dtype)
    need = hla.norm_workspace_bytes(prm)
    ws = torch.full((need + (1 << 20),), 7, dtype=torch.uint8, device="cuda")
    x, dout = (torch.randn(n, cols, device="cuda").to(TYPE[dtype]) for _ in range(2))
    w = torch.ones(cols, dtype=TYPE[dtype], device="cuda")
    _, dw = hla.rms_norm_backward(prm, x, dout, weight=w, ws=ws[:need])
    assert bool((ws[need:] == 7).all()) and bool(dw.isfinite().all())
    with pytest.raises(hla.HlaError) as e:
        hla.rms_norm_backward(prm, x, dout, weight=w, ws=ws[:need - 16])
    assert e.value.status == hla.HLA_ERR_WORKSPACE


def test_no_rows():
    prm, w = hla.NormParams(128), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert hla.rms_norm(prm, x, weight=w, residual=x).out.shape == (0, 128)
    dx, dw = hla.rms_norm_backward(prm, x, x, weight=w)
    assert dx.shape == (0, 128) and float(dw.abs().max()) == 0.0


def test_rows_past_32_bits():
    # the last rows of a batch whose elements pass 2^32
    n, cols = (1 << 20) + 1, 4096
    x = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    tail = lc.randn(1, 3, cols, dtype=torch.bfloat16)
    x[-3:] = tail.cuda()
    prm = hla.NormParams(cols)
    out = hla.rms_norm(prm, x, out=x).out
    y, err = lc.norm(tail.double(), None, 1e-6, 0.0)
    lc.close(out[-3:], y, err)
    assert float(out[:8].abs().max()) == 0.0


def test_graph_and_stream():
    prm = hla.NormParams(4096, out_dtype=E4M3, group=32)
    x, r, w = (t.cuda() for t in inputs(prm, 30))
    ref = hla.rms_norm(prm, x, weight=w, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hla.rms_norm(prm, x, weight=w, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got.out, ref.out) and torch.equal(got.exp, ref.exp)
    plain = hla.NormParams(4096)
    ws = hla.alloc_norm_workspace(plain)
    want = hla.rms_norm_backward(plain, x, r, weight=w, ws=ws)
    a = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = hla.rms_norm(prm, a, weight=w, residual=r)
        dx, dw = hla.rms_norm_backward(plain, a, r, weight=w, ws=ws)
    for _ in range(2):
        a.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.out, ref.out) and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        a.zero_()
