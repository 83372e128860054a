// Gradient of packed causal attention for bf16 layers on the tcgen05 tensor
// cores.  With P = 2^(c S - lse) recomputed from the scores, dP = dO V^T,
// D = dO . O per row and dS = P (dP - D):
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, each summing in TMEM in a fixed order:
//   dkdv  a block per 128 keys of a kv head walks the query tiles (packed
//         heads, see attention_tc.cuh) that see them, over all query heads of
//         the group: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   dq    a block per query tile walks the keys it sees: S = Q K^T,
//         dP = dO V^T, dQ += dS K
// That is 7 products in place of the 5 that one pass would take with dQ added
// to memory from many blocks: fp32 atomics would make results depend on the
// order of arrival.  (Adding them in turn, a fixed order, was not tried; the
// traffic is 4 bytes d per row and key tile either way.)  Shared kv heads are summed in the block;
// only where key blocks are few are the rows of one cut over blocks, whose sums
// a third kernel adds in order.
//
// P and dS are rounded to bf16 (the inputs' own precision) and are read by the
// products from TMEM, over the columns of the scores they came from.  The
// roundings of many keys average out in a sum over them; those of few do not:
// query tiles that see one key tile (dQ) and sequences of one key tile (dK, dV)
// take what the rounding leaves as a second bf16 value and a second product
// (errors of sequences up to 128 keys 1.25 to 1.46 -> 1.00 times the rounding of
// the result; 19 x 64 tokens 29 -> 31.6 us).
//
// D of the stored output carries that output's rounding, which moves all of a row's dS the same way.  Where those nearly
// cancel it is all that is left: one key that takes almost all of a row (O is then that key's value), values with a common
// part (O as large as they are, while dP - D is not).  The dq kernel, which runs first, therefore sums D = sum_j P_ij dP_ij
// as well, and leaves it for dk and dv.  Rows that see one key tile take it for dQ at once.  For query tiles of more keys:
//   - the difference of the two, which is the sum of a row's dS, is taken out of dQ as if all keys were the mean of 64 that
//     every row sees (as much of it as stands out from its standard error), so that what keys have in common cancels as it
//     does with dS that add up to 0; not for rows of a few keys (sum P^2 of 1/16 and more), whose own may be far from it;
//   - what is left in dQ is the difference times how far that is from the row's weighted mean of the keys, about their
//     spread times sqrt(1 / 64 + sum P^2).  Tiles in which it adds up, over the 32 rows of a warp, to more than 4 u (u = 2^-8,
//     bf16's) of their dQ, in 2-norms, are listed and done again with the better D.
// (With the stored output alone, dq of rows with P = 1 - 2^-10 was off by 1.2 times its size, that of keys and values
// shifted by 4 by 0.1 to 0.2; now 0.003 to 0.005 and 0.006 to 0.009.  4096 tokens, 32/8 heads of 128: 340 -> 360 us, 361 to 367
// with queries 8 times as long or values and keys shifted by 0.3, 404 where one long tile is done again, 530 where all
// are; 32768 tokens shifted by 1, where 8 of 10 are, 18.5 -> 27.1 ms; 4 x 4096, heads of 64: 930 -> 1073.)
//
// Products and elementwise work alternate: while dV and the next S are formed,
// dS is computed from dP; while dK and the next dP are formed, the next P.
//
// 14 d flops per visible score.  Long sequences are bound by the tensor cores: bf16, 32/8 heads of 128, 32768 tokens in 18.7 to
// 19.0 ms (1620 to 1650 TFLOP/s of the 14 d, 1160 to 1180 of the 10 d that the formulas need).  4096 in 360 us: rows'
// statistics 16, dq 174 (tensor pipe active 52 %), dk and dv 177 (68 %); 4 x 4096 tokens, 32/8 heads of 64, 1073 us (29
// and 42 %, 1.6 and 1.3 instructions of 4 a cycle), where neither is the limit; what is has not been measured.
#include "attention_tc.cuh"

namespace hla {

namespace {

using namespace attn_tc;

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    unsigned long long ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}

// ---- per row: -lse in base-2 logs and -D ------------------------------------

// One warp per 32 / (D / 8) rows: 16 bytes of out and of dout per lane.  A row
// that sees no key has lse = -inf: -inf makes its probabilities 0.
template <int D>
__global__ void __launch_bounds__(256)
attn_stats_kernel(int64_t rows, const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ dout,
                  const float* __restrict__ lse, float2* __restrict__ stats, int* __restrict__ again) {
    constexpr int L = D / 8;  // lanes per row
    if (blockIdx.x == 0 && threadIdx.x == 0) *again = 0;  // the list of query tiles to be done again
    const int64_t r = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
    float s = 0.f;
    if (r < rows) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(out + r * D) + threadIdx.x % L);
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(dout + r * D) + threadIdx.x % L);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
            s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
        }
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (r < rows && threadIdx.x % L == 0) {
        const float l = __ldg(lse + r);
        stats[r] = l == -INFINITY ? make_float2(-INFINITY, 0.f) : make_float2(-l * kLog2e, -s);
    }
}

// Hardware barriers between the elementwise warps (256 threads) and the warp that issues or passes on (32):
// scores, probabilities, score gradients dP and dS ready; in the dq kernel dP and dS by even and odd tiles
// (kBarDq, kBarDs, one more each).
constexpr int kBarS = 1, kBarP = 2, kBarDp = 3, kBarDq = 2, kBarDs = 4;
constexpr int kBarRow = 6;  // the elementwise warps among themselves

template <int D> struct Cfg {
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 8;
    // two fixed tiles (K, V or Q, dO), the ring, two stages of row stats (-lse, then -D; 128 fp32 each), barriers
    static constexpr uint32_t kFix = 0, kRing = 2 * kTile, kStat = kRing + kSlots * kTile, kBar = kStat + 2048;
    static constexpr uint32_t kItem = kBar + 352, kMean = kItem + 80, kSmem = kMean + D * 4 + 64;  // kMean: a key and 16 sums, fp32
    static_assert(sizeof(ItemRing) <= 80 && kSmem <= 227 * 1024, "shared memory layout");
    static constexpr uint32_t kCols = 512;
};

// Probability and score-gradient columns in TMEM: two halves of 64 scores, each
// overlaid by its own 32 columns of bf16 pairs, so that the two warpgroups
// never write what the other still reads.
__device__ __forceinline__ uint32_t half_step(uint32_t cols, int s) { return cols + (s >> 2) * 64 + (s & 3) * 8; }

// 64 fp32 columns at taddr
__device__ __forceinline__ void load64(uint32_t taddr, float2 (&x)[32]) {
    uint32_t r0[32], r1[32];
    umma::tmem_ld32_async(taddr, r0);
    umma::tmem_ld32_async(taddr + 32, r1);
    umma::tmem_wait_ld();
    umma::reg_fence32(r0);
    umma::reg_fence32(r1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = make_float2(__uint_as_float(r0[2 * i]), __uint_as_float(r0[2 * i + 1]));
        x[16 + i] = make_float2(__uint_as_float(r1[2 * i]), __uint_as_float(r1[2 * i + 1]));
    }
}

// Products of 128 x 128 x d and 128 x d x 128 elements, issued by the lane with `lead`.
template <int D>
__device__ __forceinline__ void outer_product(uint32_t d, uint64_t a, uint64_t b, uint32_t lead) {  // d = a b^T over d
    const uint32_t idesc = umma::idesc_bf16(kRows, kRows, false, false);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const uint64_t ks = (uint64_t)((s >> 2) * (kRows * 128 / 16) + (s & 3) * 2);
        umma::mma_lead(d, a + ks, b + ks, idesc, s > 0, lead);
    }
}
template <int D>
__device__ __forceinline__ void inner_product(uint32_t d, uint32_t a_cols, uint64_t b, bool add, bool fine,
                                              uint32_t lead) {
    const uint32_t idesc = umma::idesc_bf16(kRows, D, false, true);  // d += a b over the 128 rows of b
#pragma unroll
    for (int s = 0; s < kRows / 16; ++s)
        umma::mma_ts_lead(d, half_step(a_cols, s), b + (uint64_t)(s * 128), idesc, add || s > 0, lead);
    if (fine)  // the second parts of a
#pragma unroll
        for (int s = 0; s < kRows / 16; ++s)
            umma::mma_ts_lead(d, half_step(a_cols + 32, s), b + (uint64_t)(s * 128), idesc, true, lead);
}

// A warpgroup's 64 values a lane to its 32 columns for the product, as bf16 (with `fine`: and what that leaves, to the
// 32 columns behind them).
__device__ __forceinline__ void store64(uint32_t taddr, const float2 (&x)[32], bool fine) {
    uint32_t w[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = pack_bf2(x[e].x, x[e].y);
    umma::tmem_st32_async(taddr, w);
    if (fine) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            w[e] = pack_bf2(x[e].x - __uint_as_float(w[e] << 16), x[e].y - __uint_as_float(w[e] & 0xffff0000u));
        umma::tmem_st32_async(taddr + 32, w);
    }
    umma::tmem_wait_st();
    umma::fence_before_sync();
}

// ---- dk, dv -----------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attn_dkdv_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const int32_t* __restrict__ cu_q,
                    const int32_t* __restrict__ cu_k, int lpack, int parts, const float2* __restrict__ stats,
                    __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, float* __restrict__ part_dk,
                    float* __restrict__ part_dv, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    using Ring = RingPos<C::kSlots>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int lqb = 7 - lpack, qb = 1 << lqb, groups = A.G >> lpack;  // positions of a query tile; packed head groups
    if (blockIdx.x == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_kv = bars, bar_kve = bar_kv + 8, bar_full = bar_kve + 8, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_dp = bar_s + 8, bar_fix = bar_dp + 8, bar_done = bar_fix + 32;
    const uint32_t bar_oe = bar_done + 8, bar_it = bar_oe + 8, bar_ie = bar_it + 8 * kItems, bar_ask = bar_ie + 8 * kItems;
    const uint32_t bar_want = bar_ask + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 344);
    ItemRing* items = reinterpret_cast<ItemRing*>(sm + C::kItem);
    if (tid == 0) {
        umma::mbar_init(bar_kv, 1);
        umma::mbar_init(bar_kve, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        umma::mbar_init(bar_s, 1);
        umma::mbar_init(bar_dp, 1);
        for (int i = 0; i < 4; ++i) umma::mbar_init(bar_fix + 8 * i, 1);
        umma::mbar_init(bar_done, 1);
        umma::mbar_init(bar_oe, 8);
        for (int i = 0; i < kItems; ++i) {
            umma::mbar_init(bar_it + 8 * i, 1);
            umma::mbar_init(bar_ie + 8 * i, kItemWarps);
        }
        umma::mbar_init(bar_ask, 1);
        umma::mbar_init(bar_want, 1);
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t cS = tmem, cP = tmem + 128, cV = tmem + 256, cK = cV + D;  // S / P, dP / dS, dV, dK

    // an item's query tiles: of each packed head group, `per` tiles from tile i0, the first that sees the block's
    // first key, from its row `lead` on; the last has `tail` rows.  Of these n, from tile r of head h's group on (parts:
    // the item's share)
    struct Span {
        int i0, per, n, lead, tail, r, h;
        __device__ bool edge(int r) const { return (r == 0 && lead > 0) || (r == per - 1 && tail < kRows); }
    };
    auto span = [&](const Item& it) {
        const int off = it.lk - it.lq, p0 = max(0, it.first - off), i0 = p0 >> lqb;
        const int per = __shfl_sync(0xffffffffu, max(0, ((it.lq + qb - 1) >> lqb) - i0), 0);
        const int lead = __shfl_sync(0xffffffffu, (p0 & (qb - 1)) << lpack, 0);
        const int rest = it.lq & (qb - 1), tail = __shfl_sync(0xffffffffu, rest ? rest << lpack : kRows, 0);
        if (parts == 1 || per == 0) return Span{i0, per, per * groups, lead, tail, 0, it.head * A.G};
        const int part = __shfl_sync(0xffffffffu, it.part, 0);
        const int a = (int)((int64_t)per * groups * part / parts), b = (int)((int64_t)per * groups * (part + 1) / parts);
        return Span{i0, per, b - a, lead, tail, a % per, it.head * A.G + (a / per << lpack)};
    };

    if (warp >= 8) {
        give_registers();
        bool ok = true;
        if (warp == 8) {
            // ---- loads: the ring takes Q 0, dO 0, Q 1, dO 1, ... of every item.  Of rows behind the sequence, and of
            //      those that see no key of the block, infinities and NaN are cleared: their probability is 0 (the ring
            //      holds at most four tiles, so four barriers keep a tile's signal until the products have seen it)
            static_assert(C::kSlots <= 8, "tiles in the ring");
            Ring ring;
            int used = 0, fixed = 0, kv_loads = 0;
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                const int ask_at = max(0, sp.n - 2);
                if (sp.n == 0 && lane == 0) umma::mbar_arrive(bar_want);
                int r = sp.r, h = sp.h;
                for (int i = 0; i < sp.n; ++i) {
                    if (i == ask_at && lane == 0) umma::mbar_arrive(bar_want);  // time to look for the next item
                    const int row = it.q0 + ((sp.i0 + r) << lqb);
                    Ring use[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        use[y] = ring.next();
                        if (used++ >= C::kSlots) ok = ok && wait_or_flag(bar_empty + 8 * use[y].slot, use[y].par ^ 1u, err);
                        if (ok && lane == 0) {
                            tma::expect_tx(bar_full + 8 * use[y].slot, C::kTile);
                            for (int b = 0; b < D / 64; ++b)
                                tma::tensor_load_3d(base + C::kRing + use[y].slot * C::kTile + b * (kRows * 128),
                                                    y ? &map_do : &map_q, 64 * b, h, row, bar_full + 8 * use[y].slot);
                        }
                        if (i == 0 && y == 0) {  // the key block, once the last item's scores and dP are formed
                            if (kv_loads++ > 0) ok = ok && wait_or_flag(bar_kve, kv_loads & 1, err);
                            if (ok && lane == 0) {
                                tma::expect_tx(bar_kv, 2 * C::kTile);
                                for (int b = 0; b < D / 64; ++b) {
                                    tma::tensor_load_3d(base + C::kFix + b * (kRows * 128), &map_k, 64 * b, it.head,
                                                        it.k0 + it.first, bar_kv);
                                    tma::tensor_load_3d(base + C::kFix + C::kTile + b * (kRows * 128), &map_v, 64 * b,
                                                        it.head, it.k0 + it.first, bar_kv);
                                }
                            }
                        }
                    }
                    if (sp.edge(r)) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            unsigned char* tile = sm + C::kRing + use[y].slot * C::kTile;
                            ok = ok && wait_or_flag(bar_full + 8 * use[y].slot, use[y].par, err);
                            if (ok && r == 0) clear_nonfinite<D>(tile, 0, sp.lead, [](int) {});
                            if (ok && r == sp.per - 1) clear_nonfinite<D>(tile, sp.tail, kRows, [](int) {});
                        }
                        umma::fence_async_smem();
                        __syncwarp();
                        if (ok && lane == 0) umma::mbar_arrive(bar_fix + 8 * (fixed & 3));
                        ++fixed;
                    }
                    if (++r == sp.per) {
                        r = 0;
                        h += 1 << lpack;
                    }
                }
            }
        } else if (warp == 9) {
            // ---- products: one lane issues, the warp stays together
            const uint32_t lead = umma::elect_one();
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar, parity, err));
            };
            auto done = [&](uint32_t bar) {
                if (ok && lead) umma::commit(bar);
            };
            const uint64_t k_tile = umma::kmajor(base + C::kFix, kRows, 0);
            const uint64_t v_tile = umma::kmajor(base + C::kFix + C::kTile, kRows, 0);
            const uint64_t ring_k = umma::kmajor(base + C::kRing, kRows, 0);
            const uint64_t ring_mn = umma::mnmajor(base + C::kRing, kRows * 128, 0);
            auto at = [&](uint64_t ring0, const Ring& u) { return ring0 + (uint64_t)(u.slot * (C::kTile / 16)); };
            Ring ring;
            int fixed = 0, count = 0;
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (__shfl_sync(0xffffffffu, it.head, 0) < 0) break;
                const Span sp = span(it);
                const int n = sp.n;
                const bool fine = __shfl_sync(0xffffffffu, it.lk, 0) <= kRows;
                if (n == 0) continue;
                int r = sp.r;
                auto ready_q = [&](const Ring& q) {  // a tile's Q (of a first or last tile both, cleared)
                    wait(bar_full + 8 * q.slot, q.par);
                    if (sp.edge(r)) {
                        wait(bar_fix + 8 * (fixed & 3), (fixed >> 2) & 1);
                        ++fixed;
                    }
                    if (++r == sp.per) r = 0;
                    umma::fence_after_sync();
                };
                auto ready_o = [&](const Ring& o) {
                    wait(bar_full + 8 * o.slot, o.par);
                    umma::fence_after_sync();
                };
                Ring q = ring.next(), o = ring.next();
                wait(bar_kv, count & 1);
                ready_q(q);
                if (ok) outer_product<D>(cS, k_tile, at(ring_k, q), lead);
                done(bar_s);
                ready_o(o);
                if (ok) outer_product<D>(cP, v_tile, at(ring_k, o), lead);
                done(bar_dp);
                if (n == 1) done(bar_kve);
                if (count > 0) wait(bar_oe, (count - 1) & 1);  // dV and dK have been read
                for (int i = 0; i < n; ++i) {
                    const bool more = i + 1 < n;
                    const Ring q1 = more ? ring.next() : q, o1 = more ? ring.next() : o;
                    named_sync(kBarP, 288);
                    umma::fence_after_sync();
                    if (ok) inner_product<D>(cV, cS, at(ring_mn, o), i > 0, fine, lead);
                    done(bar_empty + 8 * o.slot);
                    if (more) {
                        ready_q(q1);
                        if (ok) outer_product<D>(cS, k_tile, at(ring_k, q1), lead);
                        done(bar_s);
                    }
                    named_sync(kBarDs, 288);
                    umma::fence_after_sync();
                    if (ok) inner_product<D>(cK, cP, at(ring_mn, q), i > 0, fine, lead);
                    done(bar_empty + 8 * q.slot);
                    if (more) {
                        ready_o(o1);
                        if (ok) outer_product<D>(cP, v_tile, at(ring_k, o1), lead);
                        done(bar_dp);
                        if (i + 2 == n) done(bar_kve);  // K and V have been read for the last time
                    } else {
                        done(bar_done);
                    }
                    q = q1;
                    o = o1;
                }
                ++count;
            }
        } else if (warp == 10) {
            // ---- row stats of each tile (rows behind the sequence: probability 0) in two stages, and "scores ready",
            //      "score gradients ready" passed on to the elementwise warps.  dP of a tile is formed after dS of the
            //      one before it is complete, so by then that one's stage has been read.
            uint32_t t = 0;  // tiles so far
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                int r = sp.r, h = sp.h;
                float2 v[4];
                auto load = [&]() {
                    const int r0 = (sp.i0 + r) << lqb;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int row = lane + 32 * y, p = r0 + (row >> lpack);
                        v[y] = p < it.lq ? __ldg(stats + ((int64_t)it.q0 + p) * A.Hq + h + (row & ((1 << lpack) - 1)))
                                         : make_float2(-INFINITY, 0.f);
                    }
                    if (++r == sp.per) {
                        r = 0;
                        h += 1 << lpack;
                    }
                };
                if (sp.n > 0) load();
                for (int i = 0; i < sp.n; ++i, ++t) {
                    float* st = reinterpret_cast<float*>(sm + C::kStat + (t & 1) * 1024);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        st[lane + 32 * y] = v[y].x;
                        st[128 + lane + 32 * y] = v[y].y;
                    }
                    if (i + 1 < sp.n) load();
                    ok = ok && wait_or_flag(bar_s, t & 1, err);
                    umma::fence_after_sync();
                    umma::fence_before_sync();
                    named_arrive(kBarS, 288);
                    ok = ok && wait_or_flag(bar_dp, t & 1, err);
                    umma::fence_after_sync();
                    umma::fence_before_sync();
                    named_arrive(kBarDp, 288);
                }
            }
        } else {
            schedule_items(A, cu_q, cu_k, kRows, A.Hkv, true, items, bar_it, bar_ie, bar_ask, bar_want, err,
                           [](int kv) { return kv; }, parts);
        }
    } else {
        take_registers();
        // ---- elementwise: lane = key, this warpgroup's 64 of the tile's 128 rows
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const uint32_t tS = cS + lanes + half * 64, tP = cP + lanes + half * 64;
        const float2 c2 = make_float2(A.scale * kLog2e, A.scale * kLog2e);
        uint32_t t = 0;  // tiles so far
        int count = 0;
        bool ok = true;
        for (int x = 0;; ++x) {
            int n, per, r;  // tiles; tiles per head group; the first one's place in it
            int ahead;      // first row that sees the key, from the group's first tile's start
            int tail;       // rows of the last tile
            int64_t at;     // the key's place in the results, or among the parts' (-1: none)
            bool fine;
            {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                const int key = it.first + (tid & 127);
                n = sp.n;
                fine = it.lk <= kRows;
                per = sp.per;
                tail = sp.tail;
                r = sp.r;
                ahead = key - (it.lk - it.lq) - (sp.i0 << lqb);
                at = key < it.lk ? (it.part * A.total_k + it.k0 + key) * A.Hkv + it.head : -1;
            }
            for (int i = 0; i < n; ++i, ++t) {
                const float* st = reinterpret_cast<const float*>(sm + C::kStat + (t & 1) * 1024) + half * 64;
                // rows from column `from` up to `to` see the key
                const int from = max(-kRows, min(kRows, ahead - (r << lqb))) * (1 << lpack) - half * 64;
                const int to = (r == per - 1 ? tail : kRows) - half * 64;
                const uint32_t seen = max(0, to - from);
                const bool edge = __any_sync(0xffffffffu, from > 0 || to < 64);
                if (++r == per) r = 0;
                named_sync(kBarS, 288);
                umma::fence_after_sync();
                float2 p[32];
                load64(tS, p);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 nl = *reinterpret_cast<const float4*>(st + 2 * e);
                    const float2 a = ffma2(p[e], c2, make_float2(nl.x, nl.y));
                    const float2 b = ffma2(p[e + 1], c2, make_float2(nl.z, nl.w));
                    p[e] = make_float2(ex2(a.x), ex2(a.y));
                    p[e + 1] = make_float2(ex2(b.x), ex2(b.y));
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        p[e].x = (uint32_t)(2 * e - from) < seen ? p[e].x : 0.f;
                        p[e].y = (uint32_t)(2 * e + 1 - from) < seen ? p[e].y : 0.f;
                    }
                }
                store64(tS, p, fine);
                named_arrive(kBarP, 288);
                named_sync(kBarDp, 288);
                umma::fence_after_sync();
                float2 d[32];
                load64(tP, d);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 nd = *reinterpret_cast<const float4*>(st + 128 + 2 * e);
                    d[e] = fmul2(p[e], fadd2(d[e], make_float2(nd.x, nd.y)));
                    d[e + 1] = fmul2(p[e + 1], fadd2(d[e + 1], make_float2(nd.z, nd.w)));
                }
                if (edge) {  // (0 times a dP that overflowed is no 0)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        d[e].x = (uint32_t)(2 * e - from) < seen ? d[e].x : 0.f;
                        d[e].y = (uint32_t)(2 * e + 1 - from) < seen ? d[e].y : 0.f;
                    }
                }
                store64(tP, d, fine);
                named_arrive(kBarDs, 288);
            }
            // ---- results: dv by the first warpgroup, dk by the second
            if (n > 0) ok = ok && wait_or_flag(bar_done, count & 1, err);
            umma::fence_after_sync();
            const float mul = half ? A.scale : 1.f;
            __nv_bfloat16* dst = (half ? dk : dv) + at * D;
            float* part = (half ? part_dk : part_dv) + at * D;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                float o[32];
                if (n > 0) {
                    umma::tmem_ld32((half ? cK : cV) + lanes + 32 * b, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (b == D / 32 - 1 && n > 0) {  // dV and dK may be overwritten
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(bar_oe);
                    ++count;
                }
                if (at >= 0 && parts > 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(part + 32 * b + e) =
                            make_float4(o[e] * mul, o[e + 1] * mul, o[e + 2] * mul, o[e + 3] * mul);
                } else if (at >= 0) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(dst + 32 * b + e) = make_uint4(
                            pack_bf2(o[e] * mul, o[e + 1] * mul), pack_bf2(o[e + 2] * mul, o[e + 3] * mul),
                            pack_bf2(o[e + 4] * mul, o[e + 5] * mul), pack_bf2(o[e + 6] * mul, o[e + 7] * mul));
                }
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

// dk and dv from the parts of their rows, in order; eight values per thread, keys of the sequences only.
template <int D>
__global__ void __launch_bounds__(256)
attn_dkdv_join_kernel(AttnDims A, const int32_t* __restrict__ cu_k, int parts, const float* __restrict__ part_dk,
                      const float* __restrict__ part_dv, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv) {
    const int64_t n = A.total_k * A.Hkv * (D / 8), i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / (D / 8) / A.Hkv;
    int64_t a, len;
    seq_range(cu_k, seq_of_token(cu_k, A.n_seqs, t), A.total_k, &a, &len);
    if (t < a || t >= a + len) return;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const float* src = y ? part_dv : part_dk;
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        for (int p = 0; p < parts; ++p) {
            const float4 u = reinterpret_cast<const float4*>(src)[2 * (p * n + i)];
            const float4 w = reinterpret_cast<const float4*>(src)[2 * (p * n + i) + 1];
            lo = make_float4(lo.x + u.x, lo.y + u.y, lo.z + u.z, lo.w + u.w);
            hi = make_float4(hi.x + w.x, hi.y + w.y, hi.z + w.z, hi.w + w.w);
        }
        reinterpret_cast<uint4*>(y ? dv : dk)[i] =
            make_uint4(pack_bf2(lo.x, lo.y), pack_bf2(lo.z, lo.w), pack_bf2(hi.x, hi.y), pack_bf2(hi.z, hi.w));
    }
}

// ---- dq ---------------------------------------------------------------------

__device__ __forceinline__ float sum4(const float2 (&x)[4]) {
    const float2 y = fadd2(fadd2(x[0], x[1]), fadd2(x[2], x[3]));
    return y.x + y.y;
}
__device__ __forceinline__ float2 pair(uint32_t w) {  // of bf16
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
constexpr float kApart = 0x1p-12f;  // (4 u)^2
constexpr int kSample = 64;        // keys
constexpr float kEven = 0x1p-4f;   // sum of P^2 of rows whose keys are many
// The part of a mean c of kSample values, whose squared differences from it add up to v, that is more than two standard
// errors: c (1 - 4 v / (kSample c)^2), 0 if that is negative.
__device__ __forceinline__ float beyond(float c, float v) {
    const float x = kSample * c, r = 4.f * v;
    return x * x > r ? c - r / x / kSample : 0.f;
}

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attn_dq_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const int32_t* __restrict__ cu_q,
                  const int32_t* __restrict__ cu_k, int lpack, const __nv_bfloat16* __restrict__ k, float2* stats,
                  __nv_bfloat16* __restrict__ dq, int* again, bool second, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    if (second) {  // the listed tiles
        pdl_wait();
        if ((int)blockIdx.x >= again[0]) return;
    }
    // K tiles stay until their dQ product, V tiles only for dP: rings of their own, so that V runs ahead
    constexpr int kKs = C::kSlots - 2, kVs = 2;
    using RingK = RingPos<kKs>;
    using RingV = RingPos<kVs>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int qb = kRows >> lpack, n_hg = A.Hq >> lpack;
    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_q = bars, bar_qe = bar_q + 8, bar_full = bar_qe + 8, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_se = bar_s + 8, bar_dp = bar_se + 8, bar_fix = bar_dp + 16;
    const uint32_t bar_clear = bar_fix + 64, bar_done = bar_clear + 16, bar_oe = bar_done + 8, bar_it = bar_oe + 8;
    const uint32_t bar_ie = bar_it + 8 * kItems;
    const uint32_t bar_ask = bar_ie + 8 * kItems, bar_want = bar_ask + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 344);
    int* noted = reinterpret_cast<int*>(sm + C::kBar + 340);  // the item listed last, and one
    ItemRing* items = reinterpret_cast<ItemRing*>(sm + C::kItem);
    if (tid == 0) {
        *noted = 0;
        umma::mbar_init(bar_q, 1);
        umma::mbar_init(bar_qe, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        umma::mbar_init(bar_s, 1);
        umma::mbar_init(bar_se, 8);
        for (int i = 0; i < 8; ++i) umma::mbar_init(bar_fix + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar_dp + 8 * i, 1);
            umma::mbar_init(bar_clear + 8 * i, 1);
        }
        umma::mbar_init(bar_done, 1);
        umma::mbar_init(bar_oe, 8);
        for (int i = 0; i < kItems; ++i) {
            umma::mbar_init(bar_it + 8 * i, 1);
            umma::mbar_init(bar_ie + 8 * i, kItemWarps);
        }
        umma::mbar_init(bar_ask, 1);
        umma::mbar_init(bar_want, 1);
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t cS = tmem, cP = tmem + 128, cQ = tmem + 384;  // S, dP / dS (two buffers), dQ

    // keys the tile sees: [0, end), in n key tiles; from `some` on only some of its rows, in key tiles from `mixed` on
    struct Span { int end, n, some, mixed; };
    auto span = [&](const Item& it) {
        const int end = max(0, min(it.lk, min(it.first + qb, it.lq) + it.lk - it.lq));
        const int some = max(0, min(end, it.first + it.lk - it.lq + 1));
        return Span{end, __shfl_sync(0xffffffffu, (end + kRows - 1) / kRows, 0), some,
                    __shfl_sync(0xffffffffu, some / kRows, 0)};
    };

    if (warp >= 8) {
        give_registers();
        bool ok = true;
        if (warp == 8) {
            // ---- loads: slots 0 .. of the ring are K tiles, the last two V tiles
            static_assert(C::kSlots <= 8, "items in the ring");
            RingK rk;
            RingV rv;
            int used = 0, fixed = 0, q_loads = 0;
            auto load = [&](const CUtensorMap* map, uint32_t slot, int head, int row) {
                if (!ok || lane) return;
                tma::expect_tx(bar_full + 8 * slot, C::kTile);
                for (int b = 0; b < D / 64; ++b)
                    tma::tensor_load_3d(base + C::kRing + slot * C::kTile + b * (kRows * 128), map, 64 * b, head, row,
                                        bar_full + 8 * slot);
            };
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                const int kv = it.head / A.G, ask_at = max(0, sp.n - 2);
                if (sp.n == 0 && lane == 0) umma::mbar_arrive(bar_want);
                RingK k;
                for (int i = 0; i < sp.n; ++i, ++used) {
                    if (i == ask_at && lane == 0) umma::mbar_arrive(bar_want);  // time to look for the next item
                    k = rk.next();
                    if (used >= kKs) ok = ok && wait_or_flag(bar_empty + 8 * k.slot, k.par ^ 1u, err);
                    load(&map_k, k.slot, kv, it.k0 + i * kRows);
                    if (i == 0) {  // the query tile, once the last item's scores and dP are formed
                        if (q_loads++ > 0) ok = ok && wait_or_flag(bar_qe, q_loads & 1, err);
                        if (ok && lane == 0) {
                            tma::expect_tx(bar_q, 2 * C::kTile);
                            for (int b = 0; b < D / 64; ++b) {
                                tma::tensor_load_3d(base + C::kFix + b * (kRows * 128), &map_q, 64 * b, it.head,
                                                    it.q0 + it.first, bar_q);
                                tma::tensor_load_3d(base + C::kFix + C::kTile + b * (kRows * 128), &map_do, 64 * b,
                                                    it.head, it.q0 + it.first, bar_q);
                            }
                        }
                    }
                    const RingV v = rv.next();
                    if (used >= kVs) ok = ok && wait_or_flag(bar_empty + 8 * (kKs + v.slot), v.par ^ 1u, err);
                    load(&map_v, kKs + v.slot, kv, it.k0 + i * kRows);
                }
                if (sp.n > 0) {
                    // keys behind the last visible one: infinities and NaN cleared (dS is 0 there).  The ring holds the K
                    // tiles of at most six items: eight barriers.
                    static_assert(kKs <= 6, "items in the ring");
                    ok = ok && wait_or_flag(bar_full + 8 * k.slot, k.par, err);
                    if (ok) clear_nonfinite<D>(sm + C::kRing + k.slot * C::kTile, sp.end - (sp.n - 1) * kRows, kRows, [](int) {});
                    umma::fence_async_smem();
                    __syncwarp();
                    if (ok && lane == 0) umma::mbar_arrive(bar_fix + 8 * (fixed & 7));
                    ++fixed;
                }
            }
        } else if (warp == 9) {
            // ---- products: one lane issues, the warp stays together
            const uint32_t lead = umma::elect_one();
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar, parity, err));
            };
            auto done = [&](uint32_t bar) {
                if (ok && lead) umma::commit(bar);
            };
            const uint64_t q_tile = umma::kmajor(base + C::kFix, kRows, 0);
            const uint64_t o_tile = umma::kmajor(base + C::kFix + C::kTile, kRows, 0);
            const uint64_t ring_k = umma::kmajor(base + C::kRing, kRows, 0);
            const uint64_t ring_mn = umma::mnmajor(base + C::kRing, kRows * 128, 0);
            RingK rk;
            RingV rv;
            int fixed = 0, cleared = 0, count = 0;
            uint32_t ts = 0;  // tiles so far
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (__shfl_sync(0xffffffffu, it.head, 0) < 0) break;
                const Span sp = span(it);
                const int n = sp.n;
                if (n == 0) continue;
                // S and dP of the item's tile i, once the scores of the tile before have been read; dP goes to the
                // buffer that the tile before last has been taken from.  Returns the slot of its K tile.
                auto tile = [&](int i) {
                    const RingK k = rk.next();
                    const RingV v = rv.next();
                    wait(bar_full + 8 * k.slot, k.par);
                    if (i == n - 1) {
                        wait(bar_fix + 8 * (fixed & 7), (fixed >> 3) & 1);
                        ++fixed;
                    }
                    if (ts > 0) wait(bar_se, (ts - 1) & 1);
                    umma::fence_after_sync();
                    if (ok) outer_product<D>(cS, q_tile, ring_k + (uint64_t)(k.slot * (C::kTile / 16)), lead);
                    done(bar_s);
                    wait(bar_full + 8 * (kKs + v.slot), v.par);
                    umma::fence_after_sync();
                    if (ok)
                        outer_product<D>(cP + (ts & 1) * 128, o_tile,
                                         ring_k + (uint64_t)((kKs + v.slot) * (C::kTile / 16)), lead);
                    done(bar_dp + 8 * (ts & 1));
                    done(bar_empty + 8 * (kKs + v.slot));
                    if (i == n - 1) done(bar_qe);  // Q and dO have been read for the last time
                    ++ts;
                    return k.slot;
                };
                wait(bar_q, count & 1);
                uint32_t k = tile(0);
                if (count > 0) wait(bar_oe, (count - 1) & 1);  // dQ has been read
                for (int i = 0; i < n; ++i) {
                    const uint32_t b = (ts - 1) & 1;  // this tile's buffer and barrier
                    const uint32_t k1 = i + 1 < n ? tile(i + 1) : k;
                    if (i >= sp.mixed) {
                        wait(bar_clear + 8 * (cleared & 1), (cleared >> 1) & 1);
                        ++cleared;
                    }
                    named_sync(kBarDs + b, 288);
                    umma::fence_after_sync();
                    if (ok)
                        inner_product<D>(cQ, cP + b * 128, ring_mn + (uint64_t)(k * (C::kTile / 16)), i > 0, n == 1, lead);
                    if (i + 1 == n) done(bar_done);
                    done(bar_empty + 8 * k);
                    k = k1;
                }
                ++count;
            }
        } else if (warp == 10) {
            // ---- "scores ready", "score gradients ready" passed on to the elementwise warps.  dP runs one tile ahead:
            //      two barriers of either kind, so that no warp, this one included, ever meets the signal of the tile
            //      after its own (the one after that waits until every warp has read the next tile's scores).  Between
            //      the two, infinities and NaN in keys that only some of the tile's rows see are cleared for the
            //      dQ product: the scores are formed already, and dS is 0 in the rows that must not see them, NaN in the
            //      others.  (At most two tiles wait for their product: two barriers.)
            uint32_t t = 0;  // tiles so far
            int cleared = 0;
            RingK rk;
            for (int x = 0;; ++x) {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                for (int i = 0; i < sp.n; ++i, ++t) {
                    const RingK k = rk.next();
                    ok = ok && wait_or_flag(bar_s, t & 1, err);
                    umma::fence_after_sync();
                    umma::fence_before_sync();
                    named_arrive(kBarS, 288);
                    if (i >= sp.mixed) {
                        const int k0 = i * kRows;
                        if (ok)
                            clear_nonfinite<D>(sm + C::kRing + k.slot * C::kTile, max(0, sp.some - k0),
                                               min(kRows, sp.end - k0), [](int) {});
                        umma::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(bar_clear + 8 * (cleared & 1));
                        ++cleared;
                    }
                    ok = ok && wait_or_flag(bar_dp + 8 * (t & 1), (t >> 1) & 1, err);
                    umma::fence_after_sync();
                    umma::fence_before_sync();
                    named_arrive(kBarDq + (t & 1), 288);
                }
            }
        } else {
            schedule_items(A, cu_q, cu_k, qb, n_hg, false, items, bar_it, bar_ie, bar_ask, bar_want, err,
                           [&](int hg) { return hg << lpack; }, 1, true, second ? again : nullptr);
        }
    } else {
        take_registers();
        // ---- elementwise: lane = row, this warpgroup's 64 of the tile's 128 keys
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const float2 c2 = make_float2(A.scale * kLog2e, A.scale * kLog2e);
        uint32_t t = 0;  // tiles so far
        int count = 0;
        bool ok = true;
        for (int x = 0;; ++x) {
            int n, limit;  // key tiles; keys the row sees: [0, limit)
            int64_t at;    // the row's place in the result (-1: none)
            int number;
            // of kSample keys that every row of the tile sees (spread over those), two columns of this thread's share (read
            // before the tiles, used behind them)
            constexpr int kShares = 512 / D, kShare = kSample / kShares;
            uint32_t common[kShare];
            bool few;  // fewer than that: too few to judge by
            {
                const Item it = next_item(items, x, bar_it, bar_ie, err);
                if (it.head < 0) break;
                n = span(it).n;
                number = it.part;
                const int seen = it.first + it.lk - it.lq + 1;
                few = seen < kSample;
                const int step = max(1, seen / kSample), x0 = tid % kShares * kShare;
                const __nv_bfloat16* col = k + it.k0 * A.sk + it.head / A.G * D + tid / kShares * 2;
#pragma unroll
                for (int y = 0; y < kShare; ++y) {
                    common[y] = 0u;
                    if (n > 1 && !second)
                        common[y] = __ldg(reinterpret_cast<const uint32_t*>(col + min((x0 + y) * step, seen - 1) * A.sk));
                }
                const int pos = it.first + (row >> lpack);
                limit = pos < it.lq ? min(it.lk, pos + it.lk - it.lq + 1) : 0;
                at = pos < it.lq ? ((int64_t)it.q0 + pos) * A.Hq + it.head + (row & ((1 << lpack) - 1)) : -1;
            }
            const float2 st = at >= 0 ? stats[at] : make_float2(-INFINITY, 0.f);
            const float2 nl = make_float2(st.x, st.x);
            float2 nd = make_float2(st.y, st.y);
            float2 sum[4], pp[4];  // of P dP and of P^2, this half's (four each: a chain of 32 FMAs takes longer than the rest)
#pragma unroll
            for (int y = 0; y < 4; ++y) sum[y] = pp[y] = make_float2(0.f, 0.f);
            float *halves = reinterpret_cast<float*>(sm + C::kStat), *mean = reinterpret_cast<float*>(sm + C::kMean);
            for (int i = 0; i < n; ++i, ++t) {
                const int seen = limit - i * kRows - half * 64;
                const bool edge = __any_sync(0xffffffffu, seen < 64);
                const uint32_t tP = cP + (t & 1) * 128 + lanes + half * 64;
                named_sync(kBarS, 288);
                umma::fence_after_sync();
                float2 p[32];
                load64(cS + lanes + half * 64, p);
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(bar_se);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 a = ffma2(p[e], c2, nl);
                    p[e] = make_float2(ex2(a.x), ex2(a.y));
                }
                if (!edge)
#pragma unroll
                    for (int e = 0; e < 32; ++e) pp[e & 3] = ffma2(p[e], p[e], pp[e & 3]);
                named_sync(kBarDq + (t & 1), 288);
                umma::fence_after_sync();
                float2 d[32];
                load64(tP, d);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        sum[e & 3].x += 2 * e < seen ? p[e].x * d[e].x : 0.f;
                        sum[e & 3].y += 2 * e + 1 < seen ? p[e].y * d[e].y : 0.f;
                        pp[e & 3].x += 2 * e < seen ? p[e].x * p[e].x : 0.f;
                        pp[e & 3].y += 2 * e + 1 < seen ? p[e].y * p[e].y : 0.f;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[e & 3] = ffma2(p[e], d[e], sum[e & 3]);
                }
                if (n == 1) {  // D of the row from all of its keys: this half's sum and the other's
                    halves[half * 128 + row] = sum4(sum);
                    named_sync(kBarRow, 256);
                    const float D_row = halves[row] + halves[128 + row];
                    nd = make_float2(-D_row, -D_row);
                    if (half == 0 && at >= 0) stats[at].y = -D_row;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    d[e] = fmul2(p[e], fadd2(d[e], nd));
                    if (edge) {
                        d[e].x = 2 * e < seen ? d[e].x : 0.f;
                        d[e].y = 2 * e + 1 < seen ? d[e].y : 0.f;
                    }
                }
                store64(tP, d, n == 1);
                named_arrive(kBarDs + (t & 1), 288);
            }
            // sum of the row's dS; as much of it as is taken out by the mean key; square of what is left of the keys
            float off = 0.f, even = 0.f, far = 0.f;
            if (n > 1 && !second) {      // D for dk and dv, and what of dQ goes with a wrong one
                halves[half * 128 + row] = sum4(sum);
                halves[256 + half * 128 + row] = sum4(pp);
                float2 c = make_float2(0.f, 0.f);
#pragma unroll
                for (int y = 0; y < kShare; ++y) c = fadd2(c, pair(common[y]));
#pragma unroll
                for (int y = 1; y < kShares; y *= 2) {
                    c.x += __shfl_xor_sync(0xffffffffu, c.x, y);
                    c.y += __shfl_xor_sync(0xffffffffu, c.y, y);
                }
                c = make_float2(c.x / kSample, c.y / kSample);
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int y = 0; y < kShare; ++y) {
                    const float2 x = pair(common[y]);
                    v.x += (x.x - c.x) * (x.x - c.x);
                    v.y += (x.y - c.y) * (x.y - c.y);
                }
                float spread = v.x + v.y;
#pragma unroll
                for (int y = 1; y < kShares; y *= 2) {
                    v.x += __shfl_xor_sync(0xffffffffu, v.x, y);
                    v.y += __shfl_xor_sync(0xffffffffu, v.y, y);
                }
                // of the mean, what stands out from its standard error (one large key does not make a mean)
                const float2 m = make_float2(beyond(c.x, v.x), beyond(c.y, v.y));
                float rest = (c.x - m.x) * (c.x - m.x) + (c.y - m.y) * (c.y - m.y), whole = c.x * c.x + c.y * c.y;
#pragma unroll
                for (int y = 16; y; y >>= 1) {
                    spread += __shfl_xor_sync(0xffffffffu, spread, y);
                    rest += __shfl_xor_sync(0xffffffffu, rest, y);
                    whole += __shfl_xor_sync(0xffffffffu, whole, y);
                }
                if (tid % kShares == 0) *reinterpret_cast<float2*>(mean + tid / kShares * 2) = m;
                if (lane == 0) {
                    mean[D + warp] = spread;
                    mean[D + 8 + warp] = __uint_as_float(pack_bf2(rest, whole));
                }
                named_sync(kBarRow, 256);
                const float D_row = halves[row] + halves[128 + row];
                off = D_row + st.y;
                spread = rest = whole = 0.f;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    spread += mean[D + y];
                    const float2 two = pair(__float_as_uint(mean[D + 8 + y]));
                    rest += two.x;
                    whole += two.y;
                }
                // Rows of a few keys may have nothing of the mean in some column: they keep dQ as it is.  (Of half the columns.)
                const float squares = halves[256 + row] + halves[384 + row];
                even = squares < kEven ? off : 0.f;
                far = 0.5f * (spread / kSample * (1.f / kSample + squares) + (squares < kEven ? rest : whole) / kShares);
                if (half == 0 && at >= 0) stats[at].y = -D_row;
            }
            if (n > 0) ok = ok && wait_or_flag(bar_done, count & 1, err);
            umma::fence_after_sync();
            // ---- results: half of the columns each
            __nv_bfloat16* dst = dq + at * D + half * (D / 2);
            float norm = 0.f;
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
                float o[32];
                if (n > 0) {
                    umma::tmem_ld32(cQ + lanes + half * (D / 2) + 32 * b, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (b == D / 64 - 1 && n > 0) {  // dQ may be overwritten
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(bar_oe);
                    ++count;
                }
                if (at >= 0) {
                    const float m = A.scale;
                    if (n > 1 && !second)
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(mean + half * (D / 2) + 32 * b + e);
                            o[e] = fmaf(-even, c.x, o[e]);
                            o[e + 1] = fmaf(-even, c.y, o[e + 1]);
                            o[e + 2] = fmaf(-even, c.z, o[e + 2]);
                            o[e + 3] = fmaf(-even, c.w, o[e + 3]);
                            norm += (o[e] * o[e] + o[e + 1] * o[e + 1]) + (o[e + 2] * o[e + 2] + o[e + 3] * o[e + 3]);
                        }
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(dst + 32 * b + e) =
                            make_uint4(pack_bf2(o[e] * m, o[e + 1] * m), pack_bf2(o[e + 2] * m, o[e + 3] * m),
                                       pack_bf2(o[e + 4] * m, o[e + 5] * m), pack_bf2(o[e + 6] * m, o[e + 7] * m));
                }
            }
            // the tile again where a warp's rows may be off by more
            if (n > 1 && !second) {
                float wrong = at >= 0 ? off * off * far : 0.f;
                norm = at >= 0 ? norm : 0.f;
                if (few) {  // (any difference will do)
                    wrong = at >= 0 ? off * off : 0.f;
                    norm = 0.f;
                }
#pragma unroll
                for (int y = 16; y; y >>= 1) {
                    wrong += __shfl_xor_sync(0xffffffffu, wrong, y);
                    norm += __shfl_xor_sync(0xffffffffu, norm, y);
                }
                if (wrong > kApart * norm && lane == 0 && atomicExch(noted, number + 1) != number + 1)
                    again[1 + atomicAdd(again, 1)] = number;
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

// Parts that the rows of each key block are cut into, a block each, their sums joined: a causal sequence's first key
// block walks all of its query tiles, the last one a few, so few key blocks per SM leave most SMs waiting for the first.
// In tiles (about a microsecond each), for equal sequences: the longest walk or the SMs' share, whichever is more; three
// for the join's launch, and 0.06 for every part written and read.  Gradients in us, one part and the rule's:
//   900 tokens, 16/1 heads of 128: 166 and 50 (15 parts)    82 + 752 + 5 + 782, 8/1 of 64: 72 and 37 (6)
//   4096, 4/1 of 128: 205 and 88 (8)                        1024, 32/8 of 128: 72 and 64 (3)
//   2048, 32/8 of 128: 147 and 123 (2)                      4096, 32/8 of 128: whole
//   200 + 150, 8/2 of 128: whole, 32.7 (in two parts 33.7)
// (A workspace's size must not depend on the device: 152 SMs.)
int key_parts(const AttnDims& A) {
    const double items = (double)std::max<int64_t>(A.n_seqs, (A.total_k + kRows - 1) / kRows) * A.Hkv;
    const double walk = (double)A.total_q * A.G / kRows / A.n_seqs;
    int best = 1;
    double least = std::max(walk, items * walk / (2 * 152));
    for (int p = 2; p <= 16; ++p) {
        const double cost = std::max(walk / p, items * walk / (2 * 152)) + 3.0 + 0.06 * items * p;
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}
size_t stat_bytes(const AttnDims& A) { return ((size_t)A.total_q * A.Hq * sizeof(float2) + 255) / 256 * 256; }
int64_t query_tiles(const AttnDims& A) {  // at most
    const int pack = pack_of(A.G);
    return (A.total_q / (kRows / pack) + A.n_seqs) * (A.Hq / pack);
}
size_t list_bytes(const AttnDims& A) { return ((size_t)(1 + query_tiles(A)) * sizeof(int) + 255) / 256 * 256; }
size_t bytes_of(const AttnDims& A, int64_t parts) {
    return stat_bytes(A) + list_bytes(A) + (parts > 1 ? (size_t)(2 * parts * A.total_k * A.Hkv * A.d) * sizeof(float) : 0);
}

template <int D>
cudaError_t launch(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                   const __nv_bfloat16* out, const float* lse, const __nv_bfloat16* dout, const int32_t* cu_q,
                   const int32_t* cu_k, __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, void* ws, size_t room,
                   int32_t* err, cudaStream_t st) {
    static DeviceCache c1, c2, c3;
    int n_sm = 0;
    cudaError_t e = device_cached(c3, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
    if (e == cudaSuccess) e = device_cached(c1, nullptr, [](int, int*) { return prepare_kernel(attn_dkdv_tc_kernel<D>, Cfg<D>::kSmem); });
    if (e == cudaSuccess)
        e = device_cached(c2, nullptr, [](int, int*) { return prepare_kernel(attn_dq_tc_kernel<D>, Cfg<D>::kSmem); });
    if (e != cudaSuccess) return e;
    const int pack = pack_of(A.G), qb = kRows / pack;
    int lpack = 0;
    while ((1 << lpack) < pack) ++lpack;
    CUtensorMap mq, mo, mk, mv;
    const uint64_t Hq = A.Hq, Hkv = A.Hkv;
    if (!tma::make_map_3d_strided(&mq, q, true, D, Hq, A.total_q, (uint64_t)A.sq * 2, 64, (uint32_t)pack, (uint32_t)qb) ||
        !tma::make_map_3d(&mo, dout, true, D, Hq, A.total_q, 64, (uint32_t)pack, (uint32_t)qb) ||
        !tma::make_map_3d_strided(&mk, k, true, D, Hkv, A.total_k, (uint64_t)A.sk * 2, 64, 1, kRows) ||
        !tma::make_map_3d_strided(&mv, v, true, D, Hkv, A.total_k, (uint64_t)A.sv * 2, 64, 1, kRows))
        return cudaErrorInvalidValue;
    const int parts = parts_within(key_parts(A), room, [&](int p) { return bytes_of(A, p); });
    float2* stats = static_cast<float2*>(ws);
    int* again = reinterpret_cast<int*>(static_cast<char*>(ws) + stat_bytes(A));
    float *part_dk = reinterpret_cast<float*>(static_cast<char*>(ws) + stat_bytes(A) + list_bytes(A)),
          *part_dv = part_dk + parts * A.total_k * A.Hkv * D;
    const int64_t rows = A.total_q * A.Hq, kb = (A.total_k / kRows + A.n_seqs) * A.Hkv * parts,
                  qblocks = query_tiles(A), sb = (rows * (D / 8) + 255) / 256;
    if (kb > INT32_MAX || qblocks > INT32_MAX || sb > INT32_MAX) return cudaErrorInvalidValue;
    attn_stats_kernel<D><<<(unsigned)sb, 256, 0, st>>>(rows, out, dout, lse, stats, again);
    // dq first: it leaves a better D for dk and dv, and a list of tiles that need it themselves (sequences of one key tile
    // have used it)
    attn_dq_tc_kernel<D><<<(unsigned)qblocks, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mo, mk, mv, cu_q, cu_k, lpack, k, stats,
                                                                          dq, again, false, err);
    if (A.total_k > kRows) {
        LaunchCfg lc(dim3((unsigned)std::min<int64_t>(qblocks, n_sm)), dim3(kBlock), Cfg<D>::kSmem, st, true);
        e = cudaLaunchKernelEx(&lc.cfg, attn_dq_tc_kernel<D>, A, mq, mo, mk, mv, cu_q, cu_k, lpack, k, stats, dq, again, true,
                               err);
        if (e != cudaSuccess) return e;
    }
    attn_dkdv_tc_kernel<D><<<(unsigned)kb, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mo, mk, mv, cu_q, cu_k, lpack, parts, stats,
                                                                       dk, dv, part_dk, part_dv, err);
    if (parts > 1) {
        const int64_t n = A.total_k * A.Hkv * (D / 8);
        attn_dkdv_join_kernel<D><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(A, cu_k, parts, part_dk, part_dv, dk, dv);
    }
    return cudaGetLastError();
}

}  // namespace

size_t attention_backward_tc_bytes(const AttnDims& A, bool parts) { return bytes_of(A, parts ? key_parts(A) : 1); }
cudaError_t launch_attention_backward_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                         const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                         const __nv_bfloat16* dout, const int32_t* cu_q, const int32_t* cu_k,
                                         __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, void* ws, size_t room,
                                         int32_t* err, cudaStream_t st) {
    return A.d == 128 ? launch<128>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, room, err, st)
                      : launch<64>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, room, err, st);
}

}  // namespace hla
