"""GPU paged cache and decode step against 64-bit forms: the 8-bit rows bit for bit, pages in any order, odd
lengths, pages that end inside a block of keys, bad pages and lengths, and the layer's run as a whole
(rotary positions, prompt attention, cache, decode steps)."""
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


def new_cache(dtype, kept, hkv, d, page, lens, spare=3, seed=0, extra_pages=0):
    """A cache whose sequences own pages in a scattered order; unused entries of the table are -1."""
    need = [-(-n // page) for n in lens]
    n_pages, wide = sum(need) + spare, max(need + [1]) + extra_pages
    order = torch.randperm(n_pages, generator=ac.gen(seed)).tolist()
    table = torch.full((len(lens), wide), -1, dtype=torch.int32)
    for i, m in enumerate(need):
        for j in range(m):
            table[i, j] = order.pop()
    ct = hla.DTYPE_E4M3 if kept == "e4m3" else TYPE[dtype][0]
    prm = hla.CacheParams(hkv, d, page, n_pages, wide, dtype=TYPE[dtype][0], cache_dtype=ct)
    return hla.Cache(prm, table.cuda())


def i64(values):
    return torch.tensor(values, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kept", ["e4m3", "same"])
@pytest.mark.parametrize("d,hkv,page", [(64, 1, 16), (128, 8, 64), (128, 3, 48), (64, 5, 256)])
def test_write_then_read(dtype, kept, d, hkv, page):
    lens, starts = [1, 0, 70, 33, 5], [0, 9, 15, 100, 63]
    t = TYPE[dtype][1]
    cache = new_cache(dtype, kept, hkv, d, page, [a + b for a, b in zip(lens, starts)])
    # rows of very different size, zeros, and values on and beside the 8-bit grid
    k, v = (ac.randn(s, sum(lens), hkv, d) * torch.exp2(6 * ac.randn(s + 1, sum(lens), hkv, 1)) for s in (1, 3))
    k[3], v[4] = 0.0, 0.0
    k[5] = torch.linspace(-448, 448, d, dtype=torch.float64)
    v[5] = (torch.arange(d) - d // 2).double() / 16
    k, v = k.to(t), v.to(t)
    hla.cache_write(cache, k.cuda(), v.cuda(), ac.cu(lens), i64(starts))
    rk, rv = hla.cache_read(cache, ac.cu(lens), i64(starts), sum(lens))
    assert cache.check_error() == 0
    for got, x, buf, exps in ((rk, k, cache.k, cache.k_exp), (rv, v, cache.v, cache.v_exp)):
        if kept == "same":
            assert torch.equal(got.cpu(), x)
            continue
        want, byte = ac.quantise(x.double())
        assert torch.equal(got.cpu(), want.to(t))
        # where the rows lie: page, then head, then position
        row = 0
        for n, (m, s0) in enumerate(zip(lens, starts)):
            for i in range(m):
                pg, at = int(cache.page_table[n, (s0 + i) // page]), (s0 + i) % page
                assert torch.equal(exps[pg, :, at].cpu(), byte[row])
                raw = buf[pg, :, at].cpu().view(torch.float8_e4m3fn).double()
                assert torch.equal(raw * torch.exp2(byte[row].double() - 127)[:, None], want[row])
                row += 1


def test_every_8_bit_value_and_the_halves_between():
    # a row with 448 as its largest is kept at 2^0: grid values come back unchanged, halves go to the even code
    vals = ac.e4m3_values()
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, -vals, mid, -mid])
    x = torch.cat([x, x.new_zeros((-len(x)) % 63)]).view(-1, 63)
    x = torch.cat([x, x.new_full((len(x), 1), 448.0)], 1)[:, None].contiguous()
    cache = new_cache("f32", "e4m3", 1, 64, 16, [len(x)])
    hla.cache_write(cache, x.float().cuda(), (x * 2 ** -100).float().cuda(), ac.cu([len(x)]), i64([0]))
    k, v = hla.cache_read(cache, ac.cu([len(x)]), i64([0]), len(x))
    want, byte = ac.quantise(x)
    assert (byte == 127).all()
    assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), want * 2 ** -100)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extremes_of_the_row_size(dtype):
    t = TYPE[dtype][1]
    big = torch.finfo(t).max
    rows = torch.zeros(6, 1, 64, dtype=t)
    rows[0, 0, 3] = big
    rows[1, 0, 5] = torch.finfo(t).tiny
    rows[2, 0, 7] = 2.0 ** -133  # below the smallest normal
    rows[3, 0, :2] = torch.tensor([math.inf, 1.0])
    rows[4, 0, :2] = torch.tensor([math.nan, 3.0])
    rows[5, 0, :2] = torch.tensor([-math.inf, 0.0])
    cache = new_cache(dtype, "e4m3", 1, 64, 16, [6])
    hla.cache_write(cache, rows.cuda(), rows.cuda(), ac.cu([6]), i64([0]))
    k, _ = hla.cache_read(cache, ac.cu([6]), i64([0]), 6)
    k = k.cpu().double()
    want, _ = ac.quantise(rows[:3].double())
    assert torch.equal(k[:3], want.to(t).double())
    assert k[3, 0, 0] == 448 * 2.0 ** -8 and k[3, 0, 1] == 1.0  # the row's scale comes from its finite values
    assert torch.isnan(k[4, 0, 0]) and k[4, 0, 1] == 3.0
    assert k[5, 0, 0] == -448 * 2.0 ** -127 or dtype == "bf16"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_row_whose_finite_values_are_all_zero(dtype, bad):
    # kept at 2^-127: an infinity becomes the largest 8-bit float there (a normal number of either type), NaN stays
    x = torch.zeros(1, 1, 64, dtype=TYPE[dtype][1])
    x[0, 0, 5] = bad
    cache = new_cache(dtype, "e4m3", 1, 64, 16, [1])
    hla.cache_write(cache, x.cuda(), -x.cuda(), ac.cu([1]), i64([0]))
    for got, sign in zip(hla.cache_read(cache, ac.cu([1]), i64([0]), 1), (1, -1)):
        got = got.cpu().double()[0, 0]
        assert (got[:5] == 0).all() and (got[6:] == 0).all()
        assert torch.isnan(got[5]) if math.isnan(bad) else got[5] == math.copysign(448 * 2.0 ** -127, sign * bad)


def test_rows_out_of_range_are_skipped_and_flagged():
    cache = new_cache("bf16", "e4m3", 2, 64, 16, [20, 20], extra_pages=1)
    cache.page_table[1, 1] = 1000  # a page that is not there
    k = ac.randn(1, 40, 2, 64, dtype=torch.bfloat16).cuda()
    before = cache.k.clone()
    hla.cache_write(cache, k, k, ac.cu([20, 20]), i64([0, 0]))
    assert cache.check_error() != 0 and cache.check_error() == 0
    rk, rv = hla.cache_read(cache, ac.cu([20, 20]), i64([0, 0]), 40)
    assert cache.check_error() != 0
    want, _ = ac.quantise(k.cpu().double())
    assert torch.equal(rk[:36].cpu().double(), want[:36]) and (rk[36:] == 0).all() and (rv[36:] == 0).all()
    used = set(cache.page_table[0, :2].tolist() + cache.page_table[1, :1].tolist())
    for p in range(cache.params.n_pages):
        if p not in used:
            assert torch.equal(cache.k[p], before[p])
    for start in ([-1, 0], [0, 1 << 40], [(1 << 63) - 1, 0]):
        hla.cache_write(cache, k[:2], k[:2], ac.cu([1, 1]), i64(start))
        assert cache.check_error() != 0
    # rows behind the last sequence are left alone
    out = torch.full((5, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    hla.cache_read(cache, ac.cu([1, 1]), i64([0, 0]), 5, k=out, v=out.clone())
    assert (out[2:] == 3).all() and cache.check_error() == 0


def fill(cache, lens, seed=0, size=0.0):
    """Random rows at positions 0 .. len - 1; returns them as the cache holds them (float64, per sequence)."""
    p, n = cache.params, sum(lens)
    t = torch.float32 if p.dtype == hla.DTYPE_F32 else torch.bfloat16
    k, v = (ac.randn(seed + i, n, p.n_kv_heads, p.head_dim) for i in (1, 2))
    v = (v * torch.exp2(size * ac.randn(seed + 3, n, 1, 1))).to(t)
    k = k.to(t)
    hla.cache_write(cache, k.cuda(), v.cuda(), ac.cu(lens), i64([0] * len(lens)))
    assert cache.check_error() == 0
    if p.cache_dtype == hla.DTYPE_E4M3:
        k, v = ac.quantise(k.double())[0], ac.quantise(v.double())[0]
    return k.double().split(lens), v.double().split(lens)


def decode_close(dtype, got, q, ks, vs, scale=None):
    """Per element: scores off by d u32 sum |q k| scale (the relative error of a weight), sums over L keys, one
    rounding of the weight to bf16 (u) in bf16 layers, the result's own rounding."""
    u = ac.EPS[TYPE[dtype][1]] / 2
    half = 0.0 if dtype == "f32" else u
    for n, (k, v) in enumerate(zip(ks, vs)):
        x, d = q[n].double(), q.shape[-1]
        want, mag = ac.decode(x, k, v, scale), ac.decode(x, k, v.abs(), scale)
        sc = scale or 1 / math.sqrt(d)
        # |v| weighted by the true weights bounds the sum's products; heads read their own kv head
        S = float(sc * x.norm(dim=-1).max() * k.norm(dim=-1).max()) if len(k) else 0.0
        tol = (half + (2 * d * S + len(k) + 64) * U32) * mag + 1.01 * u * want.abs()
        diff = (got[n].cpu().double() - want).abs()
        assert (diff <= tol).all(), f"sequence {n} of {len(k)} keys: {float((diff - tol).max())} over"


@pytest.mark.parametrize("dtype,kept", [("f32", "e4m3"), ("f32", "same"), ("bf16", "e4m3"), ("bf16", "same")])
@pytest.mark.parametrize("d,hq,hkv,page", [(128, 8, 2, 64), (64, 3, 3, 16), (128, 6, 1, 48), (64, 8, 1, 256),
                                           (128, 24, 2, 32)])
def test_decode(dtype, kept, d, hq, hkv, page):
    lens = [1, 0, 63, 64, 65, 17, 300, 1023]
    cache = new_cache(dtype, kept, hkv, d, page, lens)
    ks, vs = fill(cache, lens, size=2.0)
    q = ac.randn(9, len(lens), hq, d, dtype=TYPE[dtype][1])
    prm = hla.AttnParams(hq, hkv, d, dtype=TYPE[dtype][0])
    got = hla.attention_decode(prm, cache, q.cuda(), i64(lens))
    assert cache.check_error() == 0
    decode_close(dtype, got, q, ks, vs)


@pytest.mark.parametrize("kept", ["e4m3", "same"])
@pytest.mark.parametrize("n", [1, 70])
def test_decode_one_and_many_sequences(kept, n):
    lens = [20000] if n == 1 else [(37 * i) % 400 for i in range(n)]
    cache = new_cache("bf16", kept, 2, 128, 64, lens)
    ks, vs = fill(cache, lens)
    q = ac.randn(9, n, 8, 128, dtype=torch.bfloat16)
    got = hla.attention_decode(hla.AttnParams(8, 2, 128), cache, q.cuda(), i64(lens))
    decode_close("bf16", got, q, ks, vs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kept", ["e4m3", "same"])
def test_decode_large_scores_and_sizes(dtype, kept):
    # scores of +-100 and value rows whose sizes span 2^-60 .. 2^60
    lens = [500, 90]
    cache = new_cache(dtype, kept, 1, 64, 16, lens)
    ks, vs = fill(cache, lens, seed=4, size=20.0)
    q = ac.randn(9, 2, 4, 64, dtype=TYPE[dtype][1])
    prm = hla.AttnParams(4, 1, 64, dtype=TYPE[dtype][0], scale=3.0)
    decode_close(dtype, hla.attention_decode(prm, cache, q.cuda(), i64(lens)), q, ks, vs, scale=3.0)


@pytest.mark.parametrize("dtype,kept", [("bf16", "e4m3"), ("bf16", "same"), ("f32", "e4m3")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,length", [(1, 5000), (64, 700), (3, 16)])
@pytest.mark.parametrize("gap,ratio", [(0, 40), (10, 7), (13, 12), (14, 30), (20, 12), (30, 0), (0, 90)])
def test_decode_small_weights_beside_a_large_value(dtype, kept, d, n, length, gap, ratio):
    # in every sequence one key scores `gap` (base 2) above the others, and its value row is 2^ratio times theirs, in one
    # column only: the other columns are the other keys', however small their share of the weights
    lens = [length] * n
    cache = new_cache(dtype, kept, 1, d, 64, lens)
    t, total = TYPE[dtype][1], sum(lens)
    k, v = torch.zeros(total, 1, d), ac.randn(5, total, 1, d).float()
    v[..., 0] = 0.0
    for i in range(n):
        at = i * length + (37 * i + 3) % length
        k[at, 0, 0] = 8.0
        v[at] = 0.0
        v[at, 0, 0] = 1.5 * 2.0 ** ratio
    k, v = k.to(t), v.to(t)
    hla.cache_write(cache, k.cuda(), v.cuda(), ac.cu(lens), i64([0] * n))
    if kept == "e4m3":
        k, v = (ac.quantise(x.double())[0] for x in (k, v))
    q = torch.zeros(n, 4, d, dtype=t)
    q[..., 0] = 1.0
    scale = max(gap, 2.0 ** -10) * math.log(2) / 8
    prm = hla.AttnParams(4, 1, d, dtype=TYPE[dtype][0], scale=scale)
    got = hla.attention_decode(prm, cache, q.cuda(), i64(lens))
    assert cache.check_error() == 0
    decode_close(dtype, got, q, k.double().split(lens), v.double().split(lens), scale=prm.c().scale)


@pytest.mark.parametrize("dtype,kept", [("bf16", "e4m3"), ("bf16", "same"), ("f32", "e4m3"), ("f32", "same")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up,down", [(125, -110), (-120, 105), (100, -100)])
def test_decode_of_keys_and_queries_of_any_size(dtype, kept, d, up, down):
    # keys near one end of the range and queries near the other: scores of ordinary size
    lens = [300, 20]
    cache = new_cache(dtype, kept, 2, d, 16, lens)
    t, n = TYPE[dtype][1], sum(lens)
    k = (ac.randn(1, n, 2, d).clamp(-3.5, 3.5) * 2.0 ** up).to(t)
    v = ac.randn(2, n, 2, d).to(t)
    hla.cache_write(cache, k.cuda(), v.cuda(), ac.cu(lens), i64([0, 0]))
    if kept == "e4m3":
        k, v = (ac.quantise(x.double())[0] for x in (k, v))
    q = (ac.randn(9, 2, 8, d) * 2.0 ** down).to(t)
    scale = 2.0 ** -(up + down) / math.sqrt(d)
    got = hla.attention_decode(hla.AttnParams(8, 2, d, dtype=TYPE[dtype][0], scale=scale), cache, q.cuda(), i64(lens))
    decode_close(dtype, got, q, k.double().split(lens), v.double().split(lens), scale=scale)


@pytest.mark.parametrize("dtype,kept", [("f32", "e4m3"), ("bf16", "e4m3"), ("bf16", "same")])
def test_what_lies_behind_the_last_key_stays_out(dtype, kept):
    # the rest of the last page holds NaN codes (E4M3) or NaN
    lens = [70, 5]
    cache = new_cache(dtype, kept, 1, 128, 64, lens)
    for b in (cache.k, cache.v):
        b.fill_(0x7F if kept == "e4m3" else math.nan)
    if kept == "e4m3":
        cache.k_exp.fill_(255)
        cache.v_exp.fill_(255)
    ks, vs = fill(cache, lens)
    q = ac.randn(9, 2, 4, 128, dtype=TYPE[dtype][1])
    got = hla.attention_decode(hla.AttnParams(4, 1, 128, dtype=TYPE[dtype][0]), cache, q.cuda(), i64(lens))
    decode_close(dtype, got, q, ks, vs)


@pytest.mark.parametrize("dtype,kept", [("f32", "e4m3"), ("bf16", "e4m3"), ("bf16", "same")])
def test_bad_lengths_and_pages_are_flagged(dtype, kept):
    lens = [200, 150]
    cache = new_cache(dtype, kept, 1, 128, 64, lens)
    ks, vs = fill(cache, lens)
    q = ac.randn(9, 2, 4, 128, dtype=TYPE[dtype][1])
    prm = hla.AttnParams(4, 1, 128, dtype=TYPE[dtype][0])
    got = hla.attention_decode(prm, cache, q.cuda(), i64([-3, 150]))
    assert cache.check_error() != 0
    decode_close(dtype, got, q, [ks[0][:0], ks[1]], [vs[0][:0], vs[1]])
    hla.attention_decode(prm, cache, q.cuda(), i64([200, 1 << 50]))  # past the table: cut and flagged
    assert cache.check_error() != 0
    cache.page_table[0, 1] = 1 << 30
    got = hla.attention_decode(prm, cache, q.cuda(), i64(lens))
    assert cache.check_error() != 0 and cache.check_error() == 0
    keep = [i for i in range(200) if i // 64 != 1]  # the keys of that page are left out
    decode_close(dtype, got, q, [ks[0][keep], ks[1]], [vs[0][keep], vs[1]])


@pytest.mark.parametrize("dtype,kept", [("f32", "same"), ("f32", "e4m3"), ("bf16", "same"), ("bf16", "e4m3")])
def test_pages_past_32_bits(dtype, kept):
    # the same rows in a small pool and at the end of one of more than 2^32 values: the same bits
    lens, hkv, d, page, n_pages = [200, 77], 8, 128, 64, (1 << 32) // (8 * 64 * 128) + 40
    small = new_cache(dtype, kept, hkv, d, page, lens)
    fill(small, lens)
    pool = lambda t: None if t is None else torch.empty(n_pages, *t.shape[1:], dtype=t.dtype, device="cuda")  # noqa: E731
    first = n_pages - small.params.n_pages
    table = torch.where(small.page_table >= 0, small.page_table + first, -1)
    prm = hla.CacheParams(hkv, d, page, n_pages, table.shape[1], dtype=small.params.dtype,
                          cache_dtype=small.params.cache_dtype)
    big = hla.Cache(prm, table, *(pool(t) for t in (small.k, small.v, small.k_exp, small.v_exp)))
    fill(big, lens)
    cu, start = ac.cu(lens), i64([0, 0])
    for a, b in zip(hla.cache_read(small, cu, start, sum(lens)), hla.cache_read(big, cu, start, sum(lens))):
        assert torch.equal(a, b)
    q = ac.randn(9, 2, 16, d, dtype=TYPE[dtype][1]).cuda()
    ap = hla.AttnParams(16, hkv, d, dtype=TYPE[dtype][0])
    assert torch.equal(hla.attention_decode(ap, small, q, i64(lens)), hla.attention_decode(ap, big, q, i64(lens)))
    assert small.check_error() == 0 and big.check_error() == 0


@pytest.mark.parametrize("dtype,kept", [("f32", "e4m3"), ("bf16", "e4m3"), ("bf16", "same")])
def test_decode_repeats_on_a_stream_and_in_a_graph_with_growing_lengths(dtype, kept):
    lens = [700, 90]
    cache = new_cache(dtype, kept, 2, 64, 16, [720, 110])
    ks, vs = fill(cache, [720, 110])
    q = ac.randn(9, 2, 8, 64, dtype=TYPE[dtype][1])
    prm = hla.AttnParams(8, 2, 64, dtype=TYPE[dtype][0])
    qc, n = q.cuda(), i64(lens)
    ref = hla.attention_decode(prm, cache, qc, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hla.attention_decode(prm, cache, qc, n, stream=side)
    side.synchronize()
    assert torch.equal(other, ref)
    ws = hla.alloc_decode_workspace(prm, cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hla.attention_decode(prm, cache, qc, n, ws=ws)
    for step in range(3):
        graph.replay()
        now = [a + step for a in lens]
        decode_close(dtype, out, q, [k[:a] for k, a in zip(ks, now)], [v[:a] for v, a in zip(vs, now)])
        n.add_(1)


def test_rows_of_a_wider_query_tensor():
    lens = [33, 80, 4]
    cache = new_cache("bf16", "e4m3", 2, 128, 16, lens)
    fill(cache, lens)
    prm = hla.AttnParams(8, 2, 128)
    wide = ac.randn(3, 3, 8 * 128 + 64, dtype=torch.bfloat16).cuda()
    q = wide[:, :1024].unflatten(1, (8, 128))
    assert torch.equal(hla.attention_decode(prm, cache, q, i64(lens)),
                       hla.attention_decode(prm, cache, q.contiguous(), i64(lens)))


@pytest.mark.parametrize("dtype,kept", [("f32", "same"), ("bf16", "same"), ("bf16", "e4m3")])
def test_a_softmax_layer_from_prompt_to_decode(dtype, kept):
    """Prompts in two chunks, then decode steps, as a user runs a full softmax layer: rotate, write to the cache,
    attend (the second chunk over the keys read back).  Against the 64-bit form over the whole sequences."""
    t, d, hq, hkv = TYPE[dtype][1], 64, 4, 2
    first, second, steps = [40, 1, 90], [23, 60, 0], 4
    total = [a + b + steps for a, b in zip(first, second)]
    rp = hla.RopeParams(hq, hkv, d, scaling=hla.ROPE_SCALE_BANDS, factor=8.0, dtype=TYPE[dtype][0])
    ap = hla.AttnParams(hq, hkv, d, dtype=TYPE[dtype][0])
    cache = new_cache(dtype, kept, hkv, d, 16, total)
    x = [{"q": ac.randn(50 + n, m, hq, d, dtype=t), "k": ac.randn(60 + n, m, hkv, d, dtype=t),
          "v": ac.randn(70 + n, m, hkv, d, dtype=t)} for n, m in enumerate(total)]

    def part(lo, hi):  # rows lo[n] .. hi[n] of every sequence, packed and rotated
        rows = {m: torch.cat([s[m][a:b] for s, a, b in zip(x, lo, hi)]).cuda() for m in "qkv"}
        pos = torch.cat([torch.arange(a, b) for a, b in zip(lo, hi)]).cuda()
        q, k = hla.rope(rp, rows["q"], rows["k"], pos)
        return q, k, rows["v"]

    outs = [[] for _ in total]

    def keep(out, lens):
        for n, o in enumerate(out.cpu().split(lens)):
            outs[n].append(o)

    zero, both = [0, 0, 0], [a + b for a, b in zip(first, second)]
    q, k, v = part(zero, first)
    hla.cache_write(cache, k, v, ac.cu(first), i64(zero))
    keep(hla.attention(ap, q, k, v, ac.cu(first))[0], first)
    q, k, v = part(first, both)
    hla.cache_write(cache, k, v, ac.cu(second), i64(first))
    rk, rv = hla.cache_read(cache, ac.cu(both), i64(zero), sum(both))
    keep(hla.attention(ap, q, rk, rv, ac.cu(second), ac.cu(both))[0], second)
    for i in range(steps):
        at = [a + i for a in both]
        q, k, v = part(at, [a + 1 for a in at])
        hla.cache_write(cache, k, v, ac.cu([1, 1, 1]), i64(at))
        keep(hla.attention_decode(ap, cache, q, i64([a + 1 for a in at])), [1, 1, 1])
    assert cache.check_error() == 0
    w, gain = hla.rope_frequencies(rp)
    for n, m in enumerate(total):
        pos = torch.arange(m)
        rq, rk = (ac.rope(x[n][s].double(), pos, w, gain, d, False) for s in "qk")
        got = torch.cat(outs[n]).double()
        want = ac.attention(rq, rk, x[n]["v"], [m], [m])[0]
        # rotated q and k are rounded once each to the layer's type (scores off by 2 u |q| |k| scale, relative in
        # the weights), weights and results once; e4m3 rows add 2^-4 per key and value from the second chunk on.
        # Independent roundings: their 2-norm is about 1 / sqrt(3) of the bound; scores have a size of about 1.
        u = ac.EPS[t] / 2
        lim = 1e-5 if dtype == "f32" else 6 * u
        if kept == "e4m3":
            assert ac.rel(got[:first[n]], want[:first[n]]) <= lim
            lim += 2 * 2.0 ** -4
        assert ac.rel(got, want) <= lim
