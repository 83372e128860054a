"""GPU gated recurrence against the rows one after another in 64 bits: ragged packs, one tile and many, gates per channel
and per head, odd widths, strides, states carried over and in place, gradients, infinities, graphs and streams."""
import pytest
import torch

import layer_cases as lc
from linearized_attention_rope_gb300 import hla

pytestmark = pytest.mark.gpu
F32, BF16 = hla.DTYPE_F32, hla.DTYPE_BF16
TYPE = {F32: torch.float32, BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    build.build()


def gates(seed, n, width, dt, slow=6.0):
    rate = torch.exp(torch.rand(width, generator=lc.gen(seed), dtype=torch.float64) * slow - 7.0)
    return (-rate * torch.nn.functional.softplus(lc.randn(seed + 1, n, width))).to(dt)


def inputs(prm, lens, seed=1):
    n, c, dt = sum(lens), prm.n_channels, TYPE[prm.dtype]
    return dict(g=gates(seed, n, c // prm.gate_dim, TYPE[prm.gate_dtype]), x=lc.randn(seed + 2, n, c, dtype=dt),
                h0=lc.randn(seed + 3, len(lens), c, dtype=torch.float32), dout=lc.randn(seed + 4, n, c, dtype=dt),
                dh_last=lc.randn(seed + 5, len(lens), c, dtype=torch.float32))


def d64(x):
    return None if x is None else x.double()


def check(prm, lens, carried=True, gradient=True, **kw):
    v = inputs(prm, lens, **kw)
    dev = {k: t.cuda() for k, t in v.items()}
    n, cu = sum(lens), lc.cu(lens)
    h0 = dev["h0"] if carried else None
    ws = hla.alloc_recurrence_workspace(prm, n)
    states = hla.alloc_recurrence_states(prm, n)
    out, h_last = hla.recurrence(prm, dev["g"], dev["x"], cu, h0=h0, states=states, ws=ws)
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, prm.gate_dim, d64(v["h0"]) if carried else None,
                        v["dout"].double() if gradient else None, d64(v["dh_last"]))
    lc.close(out, *ref["out"])
    lc.close(h_last, *ref["h_last"])
    plain = hla.recurrence(prm, dev["g"], dev["x"], cu, h0=h0)
    assert torch.equal(plain[0], out) and torch.equal(plain[1], h_last)
    if gradient:
        grads = hla.recurrence_backward(prm, dev["g"], dev["x"], states, dev["dout"], cu, h0=h0, dh_last=dev["dh_last"],
                                        ws=ws)
        assert set(grads) == ({"g", "x", "h0"} if carried else {"g", "x"})
        for name, t in grads.items():
            lc.close(t, *ref[name])
    assert hla.check_workspace_error(ws) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate_dtype", [F32, BF16])
@pytest.mark.parametrize("c,gate_dim", [(64, 1), (130, 1), (33, 1), (1, 1), (128, 64), (192, 64), (256, 128)])
@pytest.mark.parametrize("lens", [[1], [3, 0, 5], [64], [65, 1, 1, 62], [0, 130, 0, 0, 7, 0], [1] * 70, [513]])
def test_matches_64_bit(dtype, gate_dtype, c, gate_dim, lens):
    check(hla.RecurrenceParams(c, gate_dim, dtype, gate_dtype), lens, carried=len(lens) != 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,gate_dim,lens", [(64, 1, [7000]), (64, 1, [2000, 1, 0, 3000, 100]), (128, 128, [3001, 2000]),
                                             (64, 64, [1, 4090, 5])])
def test_many_tiles(dtype, c, gate_dim, lens):
    check(hla.RecurrenceParams(c, gate_dim, dtype, F32), lens)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,gate_dim", [(8192, 1), (8192, 64), (8192, 128), (8191, 1)])
def test_large_runs(dtype, c, gate_dim):
    # enough channels that the tiles' runs are the long ones, in several tiles of time
    check(hla.RecurrenceParams(c, gate_dim, dtype, F32 if c == 8191 else BF16), [100, 500, 1, 333])


def test_long_sequence_against_double_on_the_gpu():
    # 150000 rows of slow gates: in pieces of 64-bit scans by doubling (off by 1e-16 per step)
    n, c = 150001, 64
    prm = hla.RecurrenceParams(c, dtype=F32)
    g, x = gates(1, n, c, torch.float32).cuda(), lc.randn(3, n, c, dtype=torch.float32).cuda()
    out, h_last = hla.recurrence(prm, g, x, lc.cu([n]))
    a, b, k = g.double().exp(), x.double(), 1
    m, steady = x.double().abs(), None
    while k < n:
        b[k:] += a[k:] * b[:-k]
        m[k:] += a[k:] * m[:-k]
        a[k:] *= a[:-k].clone()
        k *= 2
    # every row adds at most 8 U of the magnitudes, and the errors pass on through the gates as the values do
    e, a, k = 8 * lc.U * m, g.double().exp(), 1
    while k < n:
        e[k:] += a[k:] * e[:-k]
        a[k:] *= a[:-k].clone()
        k *= 2
    assert ((out.double() - b).abs() <= e + lc.U * b.abs()).all()
    # and far less than that on the whole: a row's rounding is as often up as down
    assert float((out.double() - b).norm() / b.norm()) < 2e-6
    assert torch.equal(h_last[0], out[-1])


def test_chunks_carry_the_state():
    # a prompt in one piece and in three, the states in place
    prm = hla.RecurrenceParams(192, dtype=F32)
    lens, cut = [300, 1000], [[100, 1], [0, 700], [200, 299]]
    v = inputs(prm, lens)
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, 1, v["h0"].double())
    h, at = v["h0"].cuda(), [0, 300]
    for part in cut:
        rows = torch.cat([torch.arange(a, a + p) for a, p in zip(at, part)])
        out, last = hla.recurrence(prm, v["g"][rows].cuda(), v["x"][rows].cuda(), lc.cu(part), h0=h, h_last=h)
        assert last is h
        lc.close(out, ref["out"][0][rows], ref["out"][1][rows])
        at = [a + p for a, p in zip(at, part)]
    lc.close(h, *ref["h_last"])


@pytest.mark.parametrize("lens", [[5000, 1, 2, 3000], [4, 4, 4, 1, 50]])
def test_states_and_their_gradients_in_place(lens):
    # h_last over h0 and dh0 over dh_last, with sequences that end in other tiles and runs than they start in
    prm = hla.RecurrenceParams(256, dtype=F32)
    v = {k: t.cuda() for k, t in inputs(prm, lens).items()}
    cu, states = lc.cu(lens), hla.alloc_recurrence_states(prm, sum(lens))
    out, last = hla.recurrence(prm, v["g"], v["x"], cu, h0=v["h0"], states=states)
    grads = hla.recurrence_backward(prm, v["g"], v["x"], states, v["dout"], cu, h0=v["h0"], dh_last=v["dh_last"])
    for _ in range(5):
        h, d = v["h0"].clone(), v["dh_last"].clone()
        again, _ = hla.recurrence(prm, v["g"], v["x"], cu, h0=h, h_last=h)
        assert torch.equal(again, out) and torch.equal(h, last)
        got = hla.recurrence_backward(prm, v["g"], v["x"], states, v["dout"], cu, h0=v["h0"], dh_last=d,
                                      grads={"g": torch.empty_like(v["g"]), "x": torch.empty_like(v["x"]), "h0": d})
        assert all(torch.equal(got[k], grads[k]) for k in grads)


def test_strides_and_offsets():
    # gates and inputs as slices of one projection, aligned and one value in
    prm = hla.RecurrenceParams(128, dtype=BF16, gate_dtype=BF16)
    lens = [100, 33]
    for lo in (0, 1, 2):
        wide = lc.randn(5, 133, 300, dtype=torch.bfloat16)
        wide[:, :130] = -wide[:, :130].abs()
        g, x = wide[:, lo:lo + 128], wide[:, 130 + lo:258 + lo]
        ref = lc.recurrence(g.double(), x.double(), lens, 1)
        w = wide.cuda()
        out, last = hla.recurrence(prm, w[:, lo:lo + 128], w[:, 130 + lo:258 + lo], lc.cu(lens))
        lc.close(out, *ref["out"])
        lc.close(last, *ref["h_last"])
        h = torch.zeros(133, 128, device="cuda")
        y = hla.recurrence_step(prm, w[:, lo:lo + 128], w[:, 130 + lo:258 + lo], h)
        lc.close(y, x.double(), torch.zeros(133, 128, dtype=torch.float64))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate_dtype", [F32, BF16])
@pytest.mark.parametrize("c,gate_dim,lens", [(128, 1, [100, 33]), (70, 1, [100, 33]), (128, 64, [100, 33]), (256, 128, [100, 33]),
                                             (64, 1, [2000]), (128, 64, [3000, 1]), (128, 128, [2500])])
def test_slices_of_a_projection(dtype, gate_dtype, c, gate_dim, lens):
    # gates and inputs as slices that start on and off their boundaries: forward pass, gradient, and the step from states
    prm = hla.RecurrenceParams(c, gate_dim, dtype, gate_dtype)
    v, n, cu = inputs(prm, lens), sum(lens), lc.cu(lens)
    dev = {k: t.cuda() for k, t in v.items()}
    states = hla.alloc_recurrence_states(prm, n)
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, gate_dim, v["h0"].double(), v["dout"].double(),
                        v["dh_last"].double())
    one = lc.recurrence(v["g"].double(), v["x"].double(), [1] * n, gate_dim, lc.randn(9, n, c, dtype=torch.float32).double())
    for glo, xlo in ((0, 0), (4, 4), (1, 0), (0, 1), (3, 2)):
        wide_g = torch.full((n, c // gate_dim + 8), float("nan"), dtype=TYPE[gate_dtype], device="cuda")
        wide_x = torch.full((n, c + 8), float("nan"), dtype=TYPE[dtype], device="cuda")
        g, x = wide_g[:, glo:glo + c // gate_dim], wide_x[:, xlo:xlo + c]
        g.copy_(dev["g"])
        x.copy_(dev["x"])
        out, last = hla.recurrence(prm, g, x, cu, h0=dev["h0"], states=states)
        lc.close(out, *ref["out"])
        lc.close(last, *ref["h_last"])
        grads = hla.recurrence_backward(prm, g, x, states, dev["dout"], cu, h0=dev["h0"], dh_last=dev["dh_last"])
        for name, t in grads.items():
            assert t.is_contiguous()
            lc.close(t, *ref[name])
        h = lc.randn(9, n, c, dtype=torch.float32).cuda()
        lc.close(hla.recurrence_step(prm, g, x, h), *one["out"])
        lc.close(h, *one["h_last"])


def test_many_short_sequences():
    # more sequences than a block has threads, most of one row, some of none
    prm = hla.RecurrenceParams(64, dtype=F32)
    lens = [1, 0, 2, 1] * 3000
    v = inputs(prm, lens)
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, 1, v["h0"].double(), v["dout"].double(), v["dh_last"].double())
    dev, ws = {k: t.cuda() for k, t in v.items()}, hla.alloc_recurrence_workspace(prm, sum(lens))
    states, cu = hla.alloc_recurrence_states(prm, sum(lens)), lc.cu(lens)
    out, last = hla.recurrence(prm, dev["g"], dev["x"], cu, h0=dev["h0"], states=states, ws=ws)
    grads = hla.recurrence_backward(prm, dev["g"], dev["x"], states, dev["dout"], cu, h0=dev["h0"], dh_last=dev["dh_last"], ws=ws)
    for t, name in ((out, "out"), (last, "h_last"), (grads["g"], "g"), (grads["x"], "x"), (grads["h0"], "h0")):
        lc.close(t, *ref[name])
    assert hla.check_workspace_error(ws) == 0


def test_infinities_nan_and_closed_gates():
    # a sequence's infinities and NaN stay in it and in their channels; a gate of -infinity starts anew; a gate of 0 keeps all
    prm = hla.RecurrenceParams(64, dtype=F32)
    lens = [700, 700, 700]
    v = inputs(prm, lens)
    v["g"][300], v["g"][301] = float("-inf"), 0.0
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, 1, v["h0"].double(), v["dout"].double(), v["dh_last"].double())
    bad = {k: t.clone() for k, t in v.items()}
    bad["x"][750, 3], bad["h0"][1, 9], bad["dout"][1300, 11] = float("inf"), float("nan"), float("nan")
    dev = {k: t.cuda() for k, t in bad.items()}
    states = hla.alloc_recurrence_states(prm, 2100)
    out, last = hla.recurrence(prm, dev["g"], dev["x"], lc.cu(lens), h0=dev["h0"], states=states)
    grads = hla.recurrence_backward(prm, dev["g"], dev["x"], states, dev["dout"], lc.cu(lens), h0=dev["h0"],
                                    dh_last=dev["dh_last"])
    keep = [i for i in range(64) if i not in (3, 9, 11)]
    for rows in (slice(0, 700), slice(1400, 2100)):
        lc.close(out[rows], ref["out"][0][rows], ref["out"][1][rows])
        for name in "gx":
            lc.close(grads[name][rows], ref[name][0][rows], ref[name][1][rows])
    lc.close(out[700:1400, keep], ref["out"][0][700:1400, keep], ref["out"][1][700:1400, keep])
    lc.close(grads["x"][700:1400, keep], ref["x"][0][700:1400, keep], ref["x"][1][700:1400, keep])
    # (an infinite state is NaN behind a gate near 1, which enters as exp(g) - 1)
    assert not out[750:1400, 3].isfinite().any() and out[700:1400, 9].isnan().all() and grads["x"][700:1301, 11].isnan().all()
    assert last[1, [3, 9]].isfinite().sum() == 0 and last[[0, 2]].isfinite().all()


def test_a_closed_gate_leaves_nothing():
    # states of 1e8 in front of closed gates, and of gates that nearly are
    prm = hla.RecurrenceParams(64, dtype=F32)
    g, x = torch.full((200, 64), -0.01), lc.randn(1, 200, 64, dtype=torch.float32)
    x[0] = 1e8
    g[50], g[150] = float("-inf"), -30.0
    x[100] = 1e8
    ref = lc.recurrence(g.double(), x.double(), [200], 1)
    out, _ = hla.recurrence(prm, g.cuda(), x.cuda(), lc.cu([200]))
    assert torch.equal(out[50].cpu(), x[50])
    lc.close(out, *ref["out"])


def compare(prm, v, lens, names=("out", "h_last", "g", "x", "h0")):
    """v: g, x, dout and, or None, h0 and dh_last, on the CPU; forward pass and gradient against the rows in 64 bits."""
    ref = lc.recurrence(v["g"].double(), v["x"].double(), lens, prm.gate_dim, d64(v["h0"]), v["dout"].double(),
                        d64(v["dh_last"]))
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    states, cu = hla.alloc_recurrence_states(prm, sum(lens)), lc.cu(lens)
    got = dict(zip(("out", "h_last"), hla.recurrence(prm, dev["g"], dev["x"], cu, h0=dev["h0"], states=states)))
    got.update(hla.recurrence_backward(prm, dev["g"], dev["x"], states, dev["dout"], cu, h0=dev["h0"],
                                       dh_last=dev["dh_last"]))
    for name in names:
        if name in got:
            lc.close(got[name], *ref[name])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c,gate_dim", [(64, 1), (70, 1), (128, 64), (128, 128)])
@pytest.mark.parametrize("gate", [0.5, 3.0, 6.0, 80.0])
def test_growing_gates_leave_states_of_zero_alone(dtype, c, gate_dim, gate):
    # hundreds of rows with gates above 1 and nothing in them: what a run multiplies its state by passes fp32's range, the
    # states do not.  In between, seven rows with inputs, over the border of a tile and between closed gates
    prm = hla.RecurrenceParams(c, gate_dim, dtype, F32)
    lens, n = [100, 600], 700
    g = torch.full((n, c // gate_dim), gate) * (1 - 0.25 * torch.rand(n, c // gate_dim, generator=lc.gen(1)))
    x, dout = torch.zeros(n, c), torch.zeros(n, c)
    if gate < 10:
        x[381:388], dout[381:388] = lc.randn(2, 7, c).float(), lc.randn(3, 7, c).float()
        g[380], g[388] = float("-inf"), float("-inf")
    dt = TYPE[dtype]
    compare(prm, dict(g=g, x=x.to(dt), dout=dout.to(dt), h0=None, dh_last=None), lens)


@pytest.mark.parametrize("c,gate_dim", [(64, 1), (70, 1), (128, 64), (128, 128)])
def test_states_that_grow_and_shrink_by_more_than_fp32_holds(c, gate_dim):
    # tiles of 64 rows up and down by exp(90) and more, from 1e-30, and one down by exp(105), from 1e38: every state is a
    # normal number, the factors of those tiles are not
    prm = hla.RecurrenceParams(c, gate_dim, F32, F32)
    rate = 0.97 + 0.03 * torch.rand(c // gate_dim, generator=lc.gen(4))
    up = torch.where(torch.arange(500) % 128 < 64, 1.47, -1.47)[:, None] * rate
    down = torch.where(torch.arange(200) // 64 == 1, -1.65, 0.0)[:, None] * rate
    size = 1 + torch.rand(1, c, generator=lc.gen(5))
    for g, first, last in ((up, 1e-30, 1e10), (down, 1e38, 1e30)):
        zero = torch.zeros(len(g), c)
        compare(prm, dict(g=g, x=zero, dout=zero, h0=first * size, dh_last=last * size.flip(1)), [len(g)])


def test_gates_of_every_size():
    # one row behind a state of 1: exp(g), to the last bit's neighbour
    g = torch.cat([-torch.logspace(-12, 2.2, 5000, dtype=torch.float64), torch.logspace(-8, 1.9, 500, dtype=torch.float64),
                   torch.tensor([0.0, -87.0, -103.0, -1e30, 88.5, 89.5], dtype=torch.float64)]).float()
    prm = hla.RecurrenceParams(len(g), dtype=F32)
    h = torch.ones(1, len(g), device="cuda")
    out = hla.recurrence_step(prm, g[None].cuda(), torch.zeros(1, len(g), device="cuda"), h)
    want = g.double().exp()
    fine = want < 3.4e38
    # exp(g) - 1 or exp(g): 4 roundings of itself; then the state's, rounded.  (gates below exp(-87) count as 0)
    off = (out[0].cpu().double() - want).abs()[fine]
    assert (off <= (4 * torch.minimum((want - 1).abs(), want) + want)[fine] * lc.U + 2.0 ** -125).all()
    assert out[0, -1].isinf() and torch.equal(out, h)


def test_rows_behind_the_last_sequence_and_bad_tables():
    prm = hla.RecurrenceParams(64, dtype=F32)
    v = {k: t.cuda() for k, t in inputs(prm, [50, 50]).items()}
    states, ws = hla.alloc_recurrence_states(prm, 100), hla.alloc_recurrence_workspace(prm, 100)
    out, last = torch.full((100, 64), 7.0, device="cuda"), torch.full((2, 64), 7.0, device="cuda")
    cu = torch.tensor([0, 20, 70], dtype=torch.int32, device="cuda")
    v["x"][70:], v["g"][70:], v["dout"][70:] = float("nan"), float("nan"), float("nan")
    hla.recurrence(prm, v["g"], v["x"], cu, h0=v["h0"], out=out, h_last=last, states=states, ws=ws)
    grads = {"g": torch.full_like(out, 7.0), "x": torch.full_like(out, 7.0), "h0": torch.full_like(last, 7.0)}
    hla.recurrence_backward(prm, v["g"], v["x"], states, v["dout"], cu, h0=v["h0"], grads=grads, ws=ws)
    for t in (out, grads["g"], grads["x"]):
        assert (t[70:] == 7.0).all() and t[:70].isfinite().all()
    assert hla.check_workspace_error(ws) == 0
    for bad in ([0, 60, 40], [5, 20, 100], [0, 50, 200], [-3, 50, 100]):
        hla.recurrence(prm, v["g"], v["x"], torch.tensor(bad, dtype=torch.int32, device="cuda"), states=states, ws=ws)
        assert hla.check_workspace_error(ws) == 1
        hla.recurrence_backward(prm, v["g"], v["x"], states, v["dout"], torch.tensor(bad, dtype=torch.int32, device="cuda"),
                                ws=ws)
        assert hla.check_workspace_error(ws) == 1


def test_no_rows_at_all():
    prm = hla.RecurrenceParams(64, dtype=F32)
    e, h0 = torch.empty(0, 64, device="cuda"), lc.randn(1, 3, 64, dtype=torch.float32).cuda()
    out, last = hla.recurrence(prm, e, e, lc.cu([0, 0, 0]), h0=h0)
    assert out.shape == (0, 64) and torch.equal(last, h0)
    assert float(hla.recurrence(prm, e, e, lc.cu([0, 0, 0]))[1].abs().max()) == 0.0
    grads = hla.recurrence_backward(prm, e, e, hla.alloc_recurrence_states(prm, 0), e, lc.cu([0, 0, 0]), h0=h0, dh_last=h0)
    assert torch.equal(grads["h0"], h0)
    assert hla.recurrence_step(prm, e, e, e).shape == (0, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate_dtype", [F32, BF16])
@pytest.mark.parametrize("n,c,gate_dim", [(1, 64, 1), (7, 130, 1), (64, 4096, 1), (5, 33, 1), (9, 192, 64), (3, 256, 128)])
def test_steps_are_the_recurrence(dtype, gate_dtype, n, c, gate_dim):
    prm = hla.RecurrenceParams(c, gate_dim, dtype, gate_dtype)
    steps = 4
    v = inputs(prm, [steps] * n)
    ref = lc.recurrence(v["g"].double(), v["x"].double(), [steps] * n, gate_dim, v["h0"].double())
    h = v["h0"].cuda()
    for t in range(steps):
        out = hla.recurrence_step(prm, v["g"][t::steps].contiguous().cuda(), v["x"][t::steps].contiguous().cuda(), h)
        lc.close(out, ref["out"][0][t::steps], ref["out"][1][t::steps])
    lc.close(h, *ref["h_last"])


def test_same_bits_whatever_runs_beside():
    # results do not depend on which tiles are found: again, on two streams at once, and in two graphs with a workspace each
    prm = hla.RecurrenceParams(512, dtype=BF16)
    lens = [9000, 4000, 300]
    v = {k: t.cuda() for k, t in inputs(prm, lens).items()}
    cu, n = lc.cu(lens), sum(lens)

    def call(ws, states, stream=None):
        out, last = hla.recurrence(prm, v["g"], v["x"], cu, h0=v["h0"], states=states, ws=ws, stream=stream)
        grads = hla.recurrence_backward(prm, v["g"], v["x"], states, v["dout"], cu, h0=v["h0"], dh_last=v["dh_last"],
                                        ws=ws, stream=stream)
        return out, last, grads["g"], grads["x"], grads["h0"]

    bufs = [(hla.alloc_recurrence_workspace(prm, n + 5000 * i), hla.alloc_recurrence_states(prm, n)) for i in range(2)]
    want = call(*bufs[0])
    torch.cuda.synchronize()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(call(*bufs[0]), want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [call(*b, stream=s) for b, s in zip(bufs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph, b in zip(graphs, bufs):
        with torch.cuda.graph(graph):
            outs.append(call(*b))
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in outs for a, b in zip(g, want))
        for g in outs:
            for t in g:
                t.zero_()
        torch.cuda.synchronize()
    for ws, _ in bufs:
        assert hla.check_workspace_error(ws) == 0
