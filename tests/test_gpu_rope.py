"""GPU rotary positions against a 64-bit form: layouts, scalings, partial heads, strides, far positions,
in place, the gradient, and that the gradient is the transpose of the forward map."""
import math

import pytest
import torch

import attention_cases as ac
from linearized_attention_rope_gb300 import hla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    build.build()


TYPE = {hla.DTYPE_F32: torch.float32, hla.DTYPE_BF16: torch.bfloat16}


def positions(n, far, seed):
    return torch.randint(0, far, (n,), generator=ac.gen(seed), dtype=torch.int64)


def check(got, ref, x, gain, dtype, far):
    # y = a c - b s: the angle as a fraction of a turn is held to 2^-32 and rounded to fp32 (pi 2^-24), the sine
    # and cosine are within 2 ulp, three fp32 roundings, then one of the stored type.  The reference's own angle,
    # far * w in float64, is off by far 2^-53.
    got = got.cpu().double()
    pair = gain * x.abs().max()  # |a| + |b| bounds both sums; use twice the largest value
    tol = 2 * pair * (math.pi * 2 ** -24 + 8 * 2 ** -24 + far * 2.0 ** -53) + ref.abs() * ac.EPS[dtype] / 2
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() - tol).max())


@pytest.mark.parametrize("dtype", [hla.DTYPE_F32, hla.DTYPE_BF16])
@pytest.mark.parametrize("layout", [hla.ROPE_HALF, hla.ROPE_INTERLEAVED])
@pytest.mark.parametrize("d,rot,hq,hkv,n", [(128, 128, 32, 8, 5), (64, 64, 4, 2, 700), (128, 64, 3, 1, 33),
                                            (128, 16, 8, 8, 1), (96, 20, 2, 1, 7), (6, 2, 1, 1, 3),
                                            (256, 256, 2, 2, 9), (80, 40, 5, 5, 401)])
@pytest.mark.parametrize("scaling", [hla.ROPE_SCALE_NONE, hla.ROPE_SCALE_YARN])
def test_rope_matches_64_bit(dtype, layout, d, rot, hq, hkv, n, scaling):
    t = TYPE[dtype]
    prm = hla.RopeParams(hq, hkv, d, rot_dim=rot, layout=layout, scaling=scaling, dtype=dtype, base=10000.0,
                         factor=4.0, original_len=4096)
    q, k = ac.randn(1, n, hq, d, dtype=t), ac.randn(2, n, hkv, d, dtype=t)
    pos = positions(n, 100000, 3)
    w, gain = hla.rope_frequencies(prm)
    for fn, back in ((hla.rope, False), (hla.rope_backward, True)):
        got = fn(prm, q.cuda(), k.cuda(), pos.cuda())
        for g, x in zip(got, (q, k)):
            ref = ac.rope(x.double(), pos, w, gain, rot, layout == hla.ROPE_INTERLEAVED, back)
            check(g, ref, x.double(), gain, t, 100000)


def test_far_positions_and_every_scaling():
    # a million positions away and further; also negative positions (rotate the other way)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 31) + 5, (1 << 40) + 3, -7, -(1 << 33)], dtype=torch.int64)
    q = ac.randn(5, len(pos), 2, 64, dtype=torch.float32)
    for scaling in (hla.ROPE_SCALE_NONE, hla.ROPE_SCALE_LINEAR, hla.ROPE_SCALE_BANDS, hla.ROPE_SCALE_YARN):
        prm = hla.RopeParams(2, 0, 64, scaling=scaling, dtype=hla.DTYPE_F32, factor=8.0, original_len=8192)
        w, gain = hla.rope_frequencies(prm)
        got, none = hla.rope(prm, q.cuda(), None, pos.cuda())
        assert none is None
        # the frequencies themselves are float64 (2^-53 relative); reduce p w mod 2 pi in integers, exactly
        from fractions import Fraction
        tau = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
        ang = torch.tensor([[float((int(p) * Fraction(x)) % tau) for x in w] for p in pos], dtype=torch.float64)
        ref = q.double().clone()
        a, b = q.double()[..., :32], q.double()[..., 32:]
        c, s = gain * ang.cos()[:, None], gain * ang.sin()[:, None]
        ref[..., :32], ref[..., 32:] = a * c - b * s, b * c + a * s
        near = slice(0, 4)  # freq 2^-64 turns and w / 2 pi in float64: p 2^-53 turns of angle error
        check(got[near], ref[near], q.double(), gain, torch.float32, 2 ** 32)
        assert (got.cpu().double() - ref).abs().max() <= 2 * gain * q.abs().max() * (2.0 ** 40 * 2 ** -52 * 7 + 1e-6)


def test_sines_near_half_a_turn_keep_their_bits():
    # the pair (1, 0) of angular frequency 1 becomes (cos p, sin p).  Positions whose angle lies near a half or a whole
    # turn: the sine is small, and off by a rounding of the angle's distance from there (2^-24 of it), 2 ulp of the
    # function's (2^-22 of it), and the frequency's double (p 2^-53, and as much for the product); likewise cosines near a quarter
    p = torch.arange(100000, dtype=torch.int64)
    prm = hla.RopeParams(1, 0, 2, dtype=hla.DTYPE_F32, base=10000.0)
    q = torch.zeros(len(p), 1, 2)
    q[..., 0] = 1.0
    got = hla.rope(prm, q.cuda(), None, p.cuda())[0].cpu().double()[:, 0]
    for i, want in ((0, p.double().cos()), (1, p.double().sin())):
        near = want.abs() < 2.0 ** -6
        assert near.sum() > 500
        tol = want.abs() * 5 * 2.0 ** -24 + p * 2.0 ** -52
        over = ((got[:, i] - want).abs() - tol)[near]
        assert (over <= 0).all(), float(over.max())


def test_frequencies_against_their_definitions():
    r, base, f, orig = 64, 500000.0, 8.0, 8192
    plain = [base ** (-2 * i / r) for i in range(r // 2)]
    get = lambda s: hla.rope_frequencies(hla.RopeParams(1, 1, 64, scaling=s, base=base, factor=f, original_len=orig))  # noqa: E731
    assert get(hla.ROPE_SCALE_NONE) == (pytest.approx(plain, rel=1e-14), 1.0)
    assert get(hla.ROPE_SCALE_LINEAR)[0] == pytest.approx([x / f for x in plain], rel=1e-14)
    for x, y in zip(plain, get(hla.ROPE_SCALE_BANDS)[0]):
        turns = orig * x / (2 * math.pi)
        share = min(1, max(0, (turns - 1) / 3))
        assert y == pytest.approx(x * share + x / f * (1 - share), rel=1e-12)
    w, gain = get(hla.ROPE_SCALE_YARN)
    assert gain == pytest.approx(0.1 * math.log(f) + 1)
    at = [r * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32, 1)]
    lo, hi = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
    for i, (x, y) in enumerate(zip(plain, w)):
        ramp = min(1, max(0, (i - lo) / (hi - lo)))
        assert y == pytest.approx(x / f * ramp + x * (1 - ramp), rel=1e-12)


@pytest.mark.parametrize("dtype", [hla.DTYPE_F32, hla.DTYPE_BF16])
@pytest.mark.parametrize("extra", [0, 8, 1])  # elements behind each token's heads: aligned, and not
def test_slices_of_a_fused_projection_and_in_place(dtype, extra):
    t, n, hq, hkv, d = TYPE[dtype], 37, 6, 2, 64
    prm = hla.RopeParams(hq, hkv, d, dtype=dtype)
    wide = ac.randn(7, n, (hq + 2 * hkv) * d + extra, dtype=t).cuda()
    q, k = wide[:, :hq * d].view(n, hq, d) if not extra else wide[:, :hq * d].unflatten(1, (hq, d)), \
        wide[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    pos = positions(n, 5000, 8).cuda()
    ref = hla.rope(prm, q.contiguous(), k.contiguous(), pos)
    got = hla.rope(prm, q, k, pos)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    before = wide.clone()
    out = hla.rope(prm, q, k, pos, q_out=q, k_out=k)
    assert out[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(wide[:, (hq + hkv) * d:], before[:, (hq + hkv) * d:])  # the rest is left alone


def test_gradient_is_the_transpose():
    # <rope(x), y> = <x, rope_backward(y)> in exact arithmetic; both sides summed in float64 from fp32 results
    prm = hla.RopeParams(3, 1, 128, rot_dim=96, layout=hla.ROPE_INTERLEAVED, scaling=hla.ROPE_SCALE_YARN,
                         dtype=hla.DTYPE_F32, factor=2.0)
    x, y = (ac.randn(s, 50, 3, 128, dtype=torch.float32).cuda() for s in (11, 12))
    pos = positions(50, 1 << 17, 13).cuda()
    fx, _ = hla.rope(prm, x, None, pos)
    gy, _ = hla.rope_backward(prm, y, None, pos)
    lhs, rhs = (fx.double() * y.double()).sum(), (x.double() * gy.double()).sum()
    # each of the 19200 products is off by at most about 12 fp32 roundings of its size
    assert abs(lhs - rhs) <= 12 * 2 ** -24 * float((fx.double() * y.double()).abs().sum())


def test_no_tokens_and_many():
    prm = hla.RopeParams(1, 1, 64)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = hla.rope(prm, e, e, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert out[0].shape == (0, 1, 64)
    n = 70001
    q = torch.randn(n, 1, 64, device="cuda").bfloat16()
    pos = torch.arange(n, device="cuda")
    got, _ = hla.rope(prm, q, None, pos)
    w, gain = hla.rope_frequencies(prm)
    i = torch.tensor([0, 1, 65535, 65536, n - 1])
    ref = ac.rope(q.cpu().double()[i], i, w, gain, 64, False)
    check(got[i.cuda()], ref, q.cpu().double(), gain, torch.bfloat16, n)
