"""CPU checks of the norms', the recurrence's and the 4-bit products' entry points: struct layouts, sizes, and the
refusals that happen on the host before any launch (no GPU call is made on any of these paths), and the 64-bit forms
that the GPU tests compare with against differences."""
import ctypes
import math

import pytest
import torch

import layer_cases as lc
from linearized_attention_rope_gb300 import hla

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)
INV, UNS, WS = hla.HLA_ERR_INVALID_ARG, hla.HLA_ERR_UNSUPPORTED, hla.HLA_ERR_WORKSPACE
E4M3 = hla.DTYPE_E4M3


@pytest.fixture(scope="module")
def lib():
    from linearized_attention_rope_gb300 import build

    build.build()
    return hla.load()


def test_struct_sizes():
    assert ctypes.sizeof(hla.CNormParams) == 8 * 4 + 2 * 8
    assert ctypes.sizeof(hla.CRecurrenceParams) == 4 * 4 + 2 * 8
    assert ctypes.sizeof(hla.CLinear4Params) == 6 * 4 + 8


@pytest.mark.parametrize("kw,code", [
    (dict(n_cols=0), INV), (dict(n_heads=0), INV), (dict(n_cols=(1 << 20) + 1), UNS), (dict(dtype=2), UNS),
    (dict(dtype=hla.DTYPE_F32, out_dtype=hla.DTYPE_BF16), UNS), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(offset=math.inf), INV), (dict(group=32), INV), (dict(out_dtype=E4M3, group=64), UNS),
    (dict(out_dtype=E4M3, group=32, n_cols=100), INV), (dict(out_dtype=E4M3, n_cols=100), INV),
])
def test_norm_refusals(lib, kw, code):
    prm = hla.NormParams(**{**dict(n_cols=128), **kw})
    with pytest.raises(hla.HlaError) as e:
        hla.norm_workspace_bytes(prm)
    assert e.value.status == code
    assert lib.hla_rms_norm(ctypes.byref(prm.c()), FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, None) == code


def test_norm_pointer_refusals(lib):
    def fwd(p=hla.NormParams(128).c(), x=FAKE, r=FAKE, w=FAKE, n=4, out=FAKE, exp=None, s=FAKE):
        return lib.hla_rms_norm(ctypes.byref(p), x, r, w, n, out, exp, s, None)

    assert fwd(x=None) == INV and fwd(out=None) == INV and fwd(x=ODD) == INV and fwd(w=ODD) == INV
    assert fwd(s=None) == INV  # a residual without its sum
    assert fwd(exp=FAKE) == INV  # exponents of rows that have none
    assert fwd(n=-1) == INV and fwd(n=1 << 31) == INV
    assert fwd(p=hla.NormParams(128).c(127)) == INV and fwd(p=hla.NormParams(128, n_heads=2).c(0, 200)) == INV
    bad = hla.NormParams(128).c()
    bad.reserved = 1
    assert fwd(p=bad) == INV
    eight = hla.NormParams(128, out_dtype=E4M3, group=32)
    assert fwd(p=eight.c(), exp=None) == INV
    half = ctypes.c_void_p(0x1002)
    assert fwd(p=eight.c(), exp=FAKE, x=half) == INV and fwd(p=eight.c(132), exp=FAKE) == INV  # 16-byte rows
    assert fwd(n=0, x=None, r=None, w=None, out=None, s=None) == hla.HLA_OK

    def bwd(s=FAKE, w=FAKE, do=FAKE, ds=FAKE, n=4, dx=FAKE, dw=FAKE, ws=FAKE, nb=1 << 20):
        return lib.hla_rms_norm_backward(ctypes.byref(hla.NormParams(128).c()), s, w, do, ds, n, dx, dw, ws, nb, None)

    for name in ("s", "do", "dx"):
        assert bwd(**{name: None}) == INV and bwd(**{name: ODD}) == INV
    assert bwd(w=None) == INV  # dweight without the weight
    assert bwd(ws=None) == INV and bwd(nb=100) == WS and bwd(ds=ODD) == INV and bwd(dw=ODD) == INV
    assert bwd(n=0, dw=None, ws=None) == hla.HLA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(n_channels=0), INV), (dict(gate_dim=0), INV), (dict(gate_dim=64, n_channels=96), INV),
    (dict(gate_dim=32), UNS), (dict(dtype=2), UNS), (dict(gate_dtype=2), UNS), (dict(n_channels=1 << 21), UNS),
])
def test_recurrence_refusals(lib, kw, code):
    prm = hla.RecurrenceParams(**{**dict(n_channels=128), **kw})
    with pytest.raises(hla.HlaError) as e:
        hla.recurrence_workspace_bytes(prm, 10)
    assert e.value.status == code
    p = ctypes.byref(prm.c())
    assert lib.hla_recurrence(p, *[FAKE] * 4, 1, 16, *[FAKE] * 4, 1 << 30, None) == code
    assert lib.hla_recurrence_step(p, FAKE, FAKE, FAKE, 2, FAKE, None) == code


def test_recurrence_pointer_refusals(lib):
    c = hla.RecurrenceParams(128)

    def fwd(g=FAKE, x=FAKE, h0=FAKE, cu=FAKE, n=1, total=16, out=FAKE, hl=FAKE, st=FAKE, ws=FAKE, nb=1 << 30, p=c.c()):
        return lib.hla_recurrence(ctypes.byref(p), g, x, h0, cu, n, total, out, hl, st, ws, nb, None)

    for name in ("g", "x", "cu", "out", "ws"):
        assert fwd(**{name: None}) == INV and fwd(**{name: ODD}) == INV
    for name in ("h0", "hl", "st"):
        assert fwd(**{name: ODD}) == INV
    assert fwd(n=0) == INV and fwd(total=-1) == INV and fwd(total=1 << 31) == INV
    assert fwd(nb=255) == WS
    assert fwd(p=c.c(127)) == INV and fwd(p=c.c(0, 127)) == INV

    def bwd(g=FAKE, x=FAKE, h0=FAKE, st=FAKE, cu=FAKE, do=FAKE, dl=FAKE, dg=FAKE, dx=FAKE, d0=FAKE, ws=FAKE, nb=1 << 30):
        return lib.hla_recurrence_backward(ctypes.byref(c.c()), g, x, h0, st, cu, 1, 16, do, dl, dg, dx, d0, ws, nb, None)

    for name in ("g", "x", "st", "cu", "do", "dg", "dx", "ws"):
        assert bwd(**{name: None}) == INV and bwd(**{name: ODD}) == INV
    assert bwd(nb=16) == WS

    def step(g=FAKE, x=FAKE, h=FAKE, n=2, out=FAKE):
        return lib.hla_recurrence_step(ctypes.byref(c.c()), g, x, h, n, out, None)

    for name in ("g", "x", "h", "out"):
        assert step(**{name: None}) == INV and step(**{name: ODD}) == INV
    assert step(n=-1) == INV and step(n=0, g=None) == hla.HLA_OK


def test_recurrence_strides_past_32_bits(lib):
    def call(xs, gs):
        p = hla.RecurrenceParams(64).c(xs, gs)
        return lib.hla_recurrence(ctypes.byref(p), FAKE, FAKE, None, FAKE, 0, 4, FAKE, None, None, FAKE, 1 << 30, None)

    assert call(1 << 32, 0) == UNS and call(0, 1 << 33) == UNS
    assert call((1 << 32) - 1, 0) == INV  # (no sequences)


def test_recurrence_workspace_grows(lib):
    # the workspace of the largest call serves every smaller one
    for prm in (hla.RecurrenceParams(64), hla.RecurrenceParams(4096), hla.RecurrenceParams(8192, gate_dim=128),
                hla.RecurrenceParams(70, dtype=hla.DTYPE_F32)):
        sizes = [hla.recurrence_workspace_bytes(prm, n) for n in
                 (0, 1, 64, 65, 127, 128, 129, 500, 2000, 4097, 10000, 20000, 39000, 80000, 90000, 1000000)]
        assert sizes == sorted(sizes) and sizes[0] >= 256


@pytest.mark.parametrize("kw,code", [
    (dict(n_in=0), INV), (dict(n_out=0), INV), (dict(group=16), UNS), (dict(n_in=192), INV), (dict(dtype=2), UNS),
    (dict(x_dtype=hla.DTYPE_F32), UNS), (dict(x_group=32), INV), (dict(x_dtype=E4M3, x_group=64), UNS),
    (dict(x_dtype=E4M3, x_group=128, group=32, n_in=96), INV),
])
def test_linear4_refusals(lib, kw, code):
    prm = hla.Linear4Params(**{**dict(n_in=256, n_out=64), **kw})
    with pytest.raises(hla.HlaError) as e:
        hla.linear4_workspace_bytes(prm, 3)
    assert e.value.status == code
    p = ctypes.byref(prm.c())
    assert lib.hla_linear4(p, FAKE, None, *[FAKE] * 3, 4, FAKE, FAKE, 1 << 30, None) == code
    assert lib.hla_linear4_quantize(p, *[FAKE] * 4, None) == code


def test_linear4_pointer_refusals(lib):
    def call(p=hla.Linear4Params(256, 64).c(), x=FAKE, xe=None, w=FAKE, sc=FAKE, of=FAKE, n=3, out=FAKE, ws=FAKE, nb=1 << 20):
        return lib.hla_linear4(ctypes.byref(p), x, xe, w, sc, of, n, out, ws, nb, None)

    for name in ("x", "w", "sc", "out"):
        assert call(**{name: None}) == INV and call(**{name: ODD}) == INV
    assert call(of=ODD) == INV and call(xe=FAKE) == INV and call(n=-1) == INV and call(n=1 << 30) == INV
    assert call(p=hla.Linear4Params(256, 64).c(255)) == INV
    eight = hla.Linear4Params(256, 64, x_dtype=E4M3, x_group=32).c()
    assert call(p=eight) == INV and call(p=eight, xe=FAKE, ws=None) == INV and call(p=eight, xe=FAKE, nb=100) == WS
    assert call(n=0, x=None, w=None, sc=None, out=None, ws=None, nb=0) == hla.HLA_OK
    q = ctypes.byref(hla.Linear4Params(256, 64).c())
    for args in ([None] + [FAKE] * 3, [FAKE, ODD, FAKE, FAKE], [FAKE, FAKE, None, FAKE], [FAKE, FAKE, FAKE, ODD]):
        assert lib.hla_linear4_quantize(q, *args, None) == INV


def test_tensor_refusals(lib):
    f, b = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    rec, nrm, lin = hla.RecurrenceParams(128), hla.NormParams(128), hla.Linear4Params(128, 8)
    w, sc = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.bfloat16)
    calls = [
        lambda: hla.rms_norm(nrm, f), lambda: hla.rms_norm(nrm, b[:, :64]), lambda: hla.rms_norm(nrm, b, weight=f[0]),
        lambda: hla.rms_norm(nrm, b, sum=b), lambda: hla.rms_norm(nrm, b, exp=w), lambda: hla.rms_norm(nrm, b.t()),
        lambda: hla.rms_norm(nrm, b[0]), lambda: hla.rms_norm(nrm, b),  # not on a GPU
        lambda: hla.rms_norm_backward(nrm, b, f), lambda: hla.rms_norm_backward(nrm, b, b, dweight=f[0]),
        lambda: hla.recurrence(rec, f, f, cu), lambda: hla.recurrence(rec, b, b, cu),
        lambda: hla.recurrence(rec, f, b, cu.long()), lambda: hla.recurrence(rec, f, b, cu, h0=f),
        lambda: hla.recurrence(rec, f, b, cu, states=f), lambda: hla.recurrence(rec, f, b, cu),
        lambda: hla.recurrence_backward(rec, f, b, None, b, cu), lambda: hla.recurrence_step(rec, f, b, b),
        lambda: hla.recurrence_backward(rec, f, b, f[:1], b, cu, grads={"g": f, "x": b, "h0": f[:1]}),
        lambda: hla.linear4(lin, f, w, sc), lambda: hla.linear4(lin, b, w[:4], sc), lambda: hla.linear4(lin, b, w, sc.float()),
        lambda: hla.linear4(lin, b, w, sc, x_exp=w), lambda: hla.linear4(lin, b, w, sc),
        lambda: hla.linear4_quantize(lin, f), lambda: hla.linear4_quantize(lin, b),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(hla.HlaError) as e:
            call()
        assert e.value.status == INV, i


@pytest.mark.parametrize("cols,rows", [(1, 1824), (1024, 1824), (1025, 912), (2730, 912), (2731, 760), (4096, 608), (5120, 456),
                                       (8192, 304), (16384, 152), (16385, 304), (1 << 20, 304)])
def test_norm_workspace_holds_what_blocks_write(lib, cols, rows):
    assert hla.norm_workspace_bytes(hla.NormParams(cols)) == 4 * cols * rows


def test_a_gradient_that_is_not_wanted_has_no_place(lib):
    b = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(hla.HlaError, match="not wanted") as e:
        hla.rms_norm_backward(hla.NormParams(128), b, b, weight=b[0], dweight=torch.zeros(128), need_dweight=False)
    assert e.value.status == INV


def test_reference_gradients_against_differences():
    # the 64-bit forms' gradients against central differences of the forms: the difference is off by step^2 of the third
    # derivative (about 1e-10 here) and by 1e-16 / step of the values
    step = 1e-5
    lens, c, group = [3, 0, 5], 4, 2
    g, x, h0 = -lc.randn(1, 8, c // group).abs(), lc.randn(2, 8, c), lc.randn(3, 3, c)
    dout, dl = lc.randn(4, 8, c), lc.randn(5, 3, c)
    ref = lc.recurrence(g, x, lens, group, h0, dout, dl)

    def loss(g, x, h0):
        r = lc.recurrence(g, x, lens, group, h0)
        return float((r["out"][0] * dout).sum() + (r["h_last"][0] * dl).sum())

    for name, at in (("g", 0), ("x", 1), ("h0", 2)):
        args = [g, x, h0]
        d = lc.randn(9, *args[at].shape)
        lo, hi = ([a + s * step * d if i == at else a for i, a in enumerate(args)] for s in (-1, 1))
        assert abs((loss(*hi) - loss(*lo)) / (2 * step) - float((ref[name][0] * d).sum())) < 1e-7
    x, w, ds = lc.randn(6, 5, 7), lc.randn(7, 7), lc.randn(8, 5, 7)
    dout = lc.randn(10, 5, 7)
    dx, _, dw, _ = lc.norm_grad(x, w, dout, ds, 1e-3, 0.5)
    f = lambda x, w: float((lc.norm(x, w, 1e-3, 0.5)[0] * dout).sum() + (x * ds).sum())  # noqa: E731
    d, e = lc.randn(11, 5, 7), lc.randn(12, 7)
    assert abs((f(x + step * d, w) - f(x - step * d, w)) / (2 * step) - float((dx * d).sum())) < 1e-7
    assert abs((f(x, w + step * e) - f(x, w - step * e)) / (2 * step) - float((dw * e).sum())) < 1e-7
