"""CPU checks of the full softmax layers' entry points: struct layouts, sizes, and the refusals that happen on the
host before any launch (no GPU call is made on any of these paths)."""
import ctypes
import math

import pytest
import torch

from linearized_attention_rope_gb300 import hla

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)
INV, UNS = hla.HLA_ERR_INVALID_ARG, hla.HLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from linearized_attention_rope_gb300 import build

    build.build()
    return hla.load()


def test_struct_sizes():
    assert ctypes.sizeof(hla.CRopeParams) == 8 * 4 + 4 * 8 + 2 * 8
    assert ctypes.sizeof(hla.CAttnParams) == 6 * 4 + 3 * 8
    assert ctypes.sizeof(hla.CCacheParams) == 8 * 4
    assert ctypes.sizeof(hla.CCache) == 6 * 8


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=63), INV), (dict(rot_dim=65), INV), (dict(rot_dim=130), INV), (dict(head_dim=258), UNS),
    (dict(layout=2), INV), (dict(scaling=4), INV), (dict(dtype=2), UNS), (dict(base=1.0), INV),
    (dict(base=math.inf), INV), (dict(scaling=1, factor=0.5), INV), (dict(scaling=2, factor=math.nan), INV),
    (dict(scaling=2, original_len=0), INV), (dict(scaling=3, low=4.0, high=1.0), INV), (dict(n_q_heads=-1), INV),
])
def test_rope_refusals(lib, kw, code):
    base = dict(n_q_heads=4, n_kv_heads=2, head_dim=128, factor=2.0)
    base.update(kw)
    with pytest.raises(hla.HlaError) as e:
        hla.rope_frequencies(hla.RopeParams(**base))
    assert e.value.status == code


def test_rope_pointer_refusals(lib):
    c = hla.RopeParams(4, 2, 128).c()
    call = lambda q, k, pos, n, qo, ko, p=c: lib.hla_rope(ctypes.byref(p), q, k, pos, n, qo, ko, None)  # noqa: E731
    assert call(FAKE, FAKE, FAKE, -1, FAKE, FAKE) == INV
    assert call(FAKE, FAKE, FAKE, 1 << 40, FAKE, FAKE) == INV
    assert call(FAKE, FAKE, None, 4, FAKE, FAKE) == INV
    assert call(FAKE, FAKE, FAKE, 4, None, FAKE) == INV  # q without its output
    assert call(None, FAKE, FAKE, 4, FAKE, FAKE) == INV
    assert call(ODD, FAKE, FAKE, 4, FAKE, FAKE) == INV
    assert call(FAKE, FAKE, ODD, 4, FAKE, FAKE) == INV
    assert call(FAKE, FAKE, FAKE, 4, FAKE, FAKE, hla.RopeParams(4, 2, 128).c(q_stride=100)) == INV
    assert call(FAKE, FAKE, FAKE, 0, FAKE, FAKE) == hla.HLA_OK  # nothing to do
    assert call(None, None, None, 9, None, None) == hla.HLA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=3), INV), (dict(head_dim=96), UNS), (dict(dtype=2), UNS), (dict(scale=-1.0), INV),
    (dict(scale=math.nan), INV), (dict(n_kv_heads=0), INV), (dict(n_q_heads=70000, n_kv_heads=1), INV),
])
def test_attention_refusals(lib, kw, code):
    base = dict(n_q_heads=4, n_kv_heads=2, head_dim=128)
    base.update(kw)
    prm = hla.AttnParams(**base)
    with pytest.raises(hla.HlaError) as e:
        hla.attention_workspace_bytes(prm, 16, 16, 1)
    assert e.value.status == code
    assert lib.hla_attention(ctypes.byref(prm.c()), FAKE, FAKE, FAKE, FAKE, FAKE, 1, 16, 16, FAKE, FAKE, FAKE,
                             1 << 20, None) == code


def test_attention_pointer_refusals(lib):
    ok = [FAKE] * 5
    c = hla.AttnParams(4, 2, 128).c()

    def fwd(args=ok, n=1, tq=16, tk=16, out=FAKE, lse=FAKE, ws=FAKE, nb=1 << 30, p=c):
        return lib.hla_attention(ctypes.byref(p), *args, n, tq, tk, out, lse, ws, nb, None)

    assert fwd(n=0) == INV and fwd(tq=-1) == INV and fwd(tk=1 << 31) == INV
    for i in range(4):
        for bad in (None, ODD):
            assert fwd(args=ok[:i] + [bad] + ok[i + 1:]) == INV
    assert fwd(args=ok[:4] + [ODD]) == INV
    assert fwd(args=ok[:4] + [None], tk=17) == INV  # one table for both, but other lengths
    assert fwd(out=None) == INV and fwd(lse=ODD) == INV and fwd(ws=None) == INV
    assert fwd(nb=16) == hla.HLA_ERR_WORKSPACE
    assert fwd(p=hla.AttnParams(4, 2, 128).c(q_stride=511)) == INV  # less than the heads
    assert fwd(p=hla.AttnParams(4, 2, 128).c(k_stride=257)) == INV  # not a multiple of 16 bytes
    bad = hla.AttnParams(4, 2, 128).c()
    bad.reserved = 1
    assert fwd(p=bad) == INV
    assert fwd(tq=0, tk=0, args=[None, None, None, FAKE, FAKE], out=None, lse=None) == hla.HLA_OK

    def bwd(args, n=1, tq=16, tk=16, grads=(FAKE, FAKE, FAKE), ws=FAKE, nb=1 << 30):
        return lib.hla_attention_backward(ctypes.byref(c), *args, n, tq, tk, *grads, ws, nb, None)

    ok = [FAKE] * 8
    for i in range(7):
        for bad in (None, ODD):
            assert bwd(ok[:i] + [bad] + ok[i + 1:]) == INV
    for i in range(3):
        assert bwd(ok, grads=[FAKE] * i + [None] + [FAKE] * (2 - i)) == INV
    assert bwd(ok, nb=256) == hla.HLA_ERR_WORKSPACE
    assert hla.attention_workspace_bytes(hla.AttnParams(4, 2, 128), 1000, 1000, 2, True) >= 1000 * 4 * 4


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=24), UNS), (dict(page_size=0), INV), (dict(head_dim=80), UNS), (dict(n_pages=-1), INV),
    (dict(cache_dtype=hla.DTYPE_F32), UNS), (dict(dtype=hla.DTYPE_E4M3), UNS), (dict(n_kv_heads=0), INV),
])
def test_cache_refusals(lib, kw, code):
    base = dict(n_kv_heads=2, head_dim=128, page_size=16, n_pages=4, max_pages=2)
    base.update(kw)
    c = hla.CacheParams(**base).c()
    n = ctypes.c_size_t()
    assert lib.hla_cache_bytes(ctypes.byref(c), ctypes.byref(n), ctypes.byref(n)) == code
    assert lib.hla_cache_write(ctypes.byref(c), ctypes.byref(hla.CCache(*[0x1000] * 6)), FAKE, FAKE, FAKE, FAKE, 1, 4,
                               None) == code


def test_cache_pointer_refusals(lib):
    c = hla.CacheParams(2, 128, 16, 4, 2).c()
    rows, exps = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.hla_cache_bytes(ctypes.byref(c), ctypes.byref(rows), ctypes.byref(exps)) == 0
    assert (rows.value, exps.value) == (4 * 2 * 16 * 128, 4 * 2 * 16)
    good = [0x1000] * 6
    write = lambda b, k=FAKE, cu=FAKE, st=FAKE, n=1, t=4: lib.hla_cache_write(  # noqa: E731
        ctypes.byref(c), ctypes.byref(hla.CCache(*b)), k, FAKE, cu, st, n, t, None)
    for i in range(6):
        for bad in (0, 0x1008):
            assert write(good[:i] + [bad] + good[i + 1:]) == INV
    assert write(good, k=None) == INV and write(good, cu=ODD) == INV and write(good, st=None) == INV
    assert write(good, n=0) == INV and write(good, t=-1) == INV
    assert write(good, t=0) == hla.HLA_OK
    a = hla.AttnParams(4, 2, 128).c()
    dec = lambda b=good, p=a, cp=c, q=FAKE, ln=FAKE, n=2, out=FAKE, ws=FAKE, nb=1 << 30: lib.hla_attention_decode(  # noqa: E731
        ctypes.byref(p), ctypes.byref(cp), ctypes.byref(hla.CCache(*b)), q, ln, n, out, ws, nb, None)
    assert dec(q=ODD) == INV and dec(ln=None) == INV and dec(out=None) == INV and dec(ws=None) == INV
    assert dec(n=-1) == INV and dec(n=0) == hla.HLA_OK
    assert dec(nb=64) == hla.HLA_ERR_WORKSPACE
    assert dec(p=hla.AttnParams(4, 4, 128).c()) == INV and dec(p=hla.AttnParams(4, 2, 64).c()) == INV
    assert dec(p=hla.AttnParams(4, 2, 128, dtype=hla.DTYPE_F32).c()) == INV
    assert lib.hla_check_cache_error(ctypes.byref(hla.CCache(*[0] * 6)), None, None) == INV


def test_binding_refuses_wrong_tensors(lib):
    """Types, shapes and strides, checked before anything is launched (CPU tensors reach no kernel)."""
    prm = hla.AttnParams(4, 2, 64)
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 8], dtype=torch.int32)

    def refused(fn, *args, **kw):
        with pytest.raises(hla.HlaError) as e:
            fn(*args, **kw)
        assert e.value.status == INV

    refused(hla.attention, prm, q, k, k, cu)  # not on the GPU
    refused(hla.attention, prm, q.float(), k, k, cu)
    refused(hla.attention, prm, q, k, k[:7], cu)
    refused(hla.attention, prm, q, k, k, cu.long())
    refused(hla.attention, prm, q[:, :, ::2], k, k, cu)
    refused(hla.attention, prm, q.transpose(0, 1), k, k, cu)
    refused(hla.attention, prm, q[:1].expand(8, 4, 64), k, k, cu)  # one row for all tokens
    refused(hla.attention, prm, q, k, k, cu[:1])
    refused(hla.attention_backward, prm, q, k, k, q, torch.zeros(8, 3), q, cu)
    rp = hla.RopeParams(4, 2, 64)
    refused(hla.rope, rp, q, k, torch.zeros(8, dtype=torch.int32))
    refused(hla.rope, rp, q, k, torch.zeros(7, dtype=torch.int64))
    refused(hla.rope, rp, None, k, torch.zeros(8, dtype=torch.int64), q_out=q)
    refused(hla.Cache, hla.CacheParams(2, 64, 16, 4, 2), torch.zeros(1, 2, dtype=torch.int32))


def test_rows_of_one_head_at_any_stride():
    # the stride of a dimension of size one says nothing: a fused [T, 1, 3, d] projection's q, k, v
    wide = torch.zeros(5, 1, 3, 64)
    for i in range(3):
        t = wide[:, :, i]
        assert t.stride() == (192, 192, 1)
        assert hla._check_tensor(t, "f", "t", torch.float32, (5, 1, 64), t.device, strided=True) == 192
    with pytest.raises(hla.HlaError):
        hla._check_tensor(wide[:, :, 0], "f", "t", torch.float32, (5, 1, 64), wide.device)  # where dense rows are asked for
    two = torch.zeros(5, 2, 3, 64)[:, :, 0]
    with pytest.raises(hla.HlaError):
        hla._check_tensor(two, "f", "t", torch.float32, (5, 2, 64), two.device, strided=True)
