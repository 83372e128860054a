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
// order of arrival, and their traffic (4 bytes d per row and key tile) exceeds
// what the two extra products cost.  No gradient is summed outside a block, so
// shared kv heads need no second pass either.
//
// P and dS are rounded to bf16 (the inputs' own precision) and are read by the
// products from TMEM, over the columns of the scores they came from.  Products
// and elementwise work alternate: while dV and the next S are formed, dS is
// computed from dP; while dK and the next dP are formed, the next P.
//
// Bound by the tensor cores: 14 d flops per visible score.
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
                  const float* __restrict__ lse, float2* __restrict__ stats) {
    constexpr int L = D / 8;  // lanes per row
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
// scores, probabilities (dkdv; dq: scores of odd tiles), score gradients dP and dS ready.
constexpr int kBarS = 1, kBarP = 2, kBarDp = 3, kBarDs = 4;

template <int D> struct Cfg {
    static constexpr uint32_t kTile = kRows * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 8;
    // two fixed tiles (K, V or Q, dO), the ring, two stages of row stats (-lse, then -D; 128 fp32 each), barriers
    static constexpr uint32_t kFix = 0, kRing = 2 * kTile, kStat = kRing + kSlots * kTile, kBar = kStat + 2048;
    static constexpr uint32_t kSmem = kBar + 256;
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

// ---- dk, dv -----------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attn_dkdv_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const int32_t* __restrict__ cu_q,
                    const int32_t* __restrict__ cu_k, int lpack, const float2* __restrict__ stats,
                    __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int qb = kRows >> lpack;
    if (blockIdx.x == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, kRows, blockIdx.x / A.Hkv, true);
    if (!B.found) return;  // the whole block
    const int kv = blockIdx.x % A.Hkv, off = B.lk - B.lq;
    // query tiles: of each packed head group, those from the first that sees the block's first key
    const int i0 = max(0, B.first - off) / qb, per = max(0, (B.lq + qb - 1) / qb - i0);
    const int n = __shfl_sync(0xffffffffu, per * (A.G >> lpack), 0);
    const int tail = B.lq % qb ? (B.lq % qb) << lpack : kRows;  // rows of a group's last tile

    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_kv = bars, bar_full = bars + 8, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_dp = bar_s + 8, bar_fix = bar_dp + 8, bar_done = bar_fix + 32;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 248);
    if (tid == 0) {
        umma::mbar_init(bar_kv, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        umma::mbar_init(bar_s, 1);
        umma::mbar_init(bar_dp, 1);
        for (int i = 0; i < 4; ++i) umma::mbar_init(bar_fix + 8 * i, 1);
        umma::mbar_init(bar_done, 1);
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t cS = tmem, cP = tmem + 128, cV = tmem + 256, cK = cV + D;  // S / P, dP / dS, dV, dK
    auto slot_of = [&](int use) { return use % C::kSlots; };
    auto par_of = [&](int use) { return (uint32_t)(use / C::kSlots) & 1u; };
    const int h0 = kv * A.G;
    auto first_row = [&](int i) { return (i0 + i % per) * qb; };
    auto has_tail = [&](int i) { return tail < kRows && i % per == per - 1; };

    if (warp >= 8) {
        give_registers();
        bool ok = true;
        if (warp == 8 && n > 0) {
            // ---- loads: use 2 i of the ring is tile i of Q, use 2 i + 1 of dO.  Rows behind the sequence are
            //      cleared, whatever they hold (the ring holds at most four tiles, so four barriers keep a tile's
            //      signal until the products have seen it)
            static_assert(C::kSlots <= 8, "tiles in the ring");
            if (lane == 0) {
                tma::expect_tx(bar_kv, 2 * C::kTile);
                for (int b = 0; b < D / 64; ++b) {
                    tma::tensor_load_3d(base + C::kFix + b * (kRows * 128), &map_k, 64 * b, kv, (int)(B.k0 + B.first),
                                        bar_kv);
                    tma::tensor_load_3d(base + C::kFix + C::kTile + b * (kRows * 128), &map_v, 64 * b, kv,
                                        (int)(B.k0 + B.first), bar_kv);
                }
            }
            int u = 0, fixed = 0;
            for (; u < 2 * n; ++u) {
                const int i = u >> 1, slot = slot_of(u);
                if (u >= C::kSlots && !(ok = wait_or_flag(bar_empty + 8 * slot, par_of(u - C::kSlots), err))) break;
                if (lane == 0) {
                    tma::expect_tx(bar_full + 8 * slot, C::kTile);
                    for (int b = 0; b < D / 64; ++b)
                        tma::tensor_load_3d(base + C::kRing + slot * C::kTile + b * (kRows * 128),
                                            u & 1 ? &map_do : &map_q, 64 * b, h0 + ((i / per) << lpack),
                                            (int)B.q0 + first_row(i), bar_full + 8 * slot);
                }
                if ((u & 1) && has_tail(i)) {
                    for (int y = u - 1; y <= u && ok; ++y) {
                        ok = wait_or_flag(bar_full + 8 * slot_of(y), par_of(y), err);
                        if (ok) zero_rows<D>(sm + C::kRing + slot_of(y) * C::kTile, tail);
                    }
                    if (!ok) { ++u; break; }
                    umma::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(bar_fix + 8 * (fixed & 3));
                    ++fixed;
                }
            }
            if (!ok) {  // copies in flight land before the block ends
                wait_or_flag(bar_kv, 0, err);
                for (int i = max(0, u - C::kSlots); i < u; ++i) wait_or_flag(bar_full + 8 * slot_of(i), par_of(i), err);
            }
        } else if (warp == 9 && n > 0) {
            // ---- products: one lane issues, the warp stays together
            const uint32_t lead = umma::elect_one();
            const uint32_t id_s = umma::idesc_bf16(kRows, kRows, false, false);
            const uint32_t id_d = umma::idesc_bf16(kRows, D, false, true);
            int fixed = 0;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar, parity, err));
            };
            auto ring = [&](int u) { return base + C::kRing + slot_of(u) * C::kTile; };
            auto ready = [&](int i) {  // Q and dO of tile i, cleared behind the last row
                wait(bar_full + 8 * slot_of(2 * i), par_of(2 * i));
                wait(bar_full + 8 * slot_of(2 * i + 1), par_of(2 * i + 1));
                if (has_tail(i)) {
                    wait(bar_fix + 8 * (fixed & 3), (fixed >> 2) & 1);
                    ++fixed;
                }
                umma::fence_after_sync();
            };
            auto outer = [&](uint32_t d, uint32_t a_tile, uint32_t b_tile) {  // d = a b^T over d
                if (!ok) return;
                const uint64_t a = umma::kmajor(a_tile, kRows, 0), b = umma::kmajor(b_tile, kRows, 0);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t ks = (uint64_t)((s >> 2) * (kRows * 128 / 16) + (s & 3) * 2);
                    umma::mma_lead(d, a + ks, b + ks, id_s, s > 0, lead);
                }
            };
            auto inner = [&](uint32_t d, uint32_t a_cols, uint32_t b_tile, bool add) {  // d += a b over the rows
                if (!ok) return;
                const uint64_t b = umma::mnmajor(b_tile, kRows * 128, 0);
#pragma unroll
                for (int s = 0; s < kRows / 16; ++s)
                    umma::mma_ts_lead(d, half_step(a_cols, s), b + (uint64_t)(s * 128), id_d, add || s > 0, lead);
            };
            auto done = [&](uint32_t bar) {
                if (ok && lead) umma::commit(bar);
            };
            wait(bar_kv, 0);
            ready(0);
            outer(cS, base + C::kFix, ring(0));
            done(bar_s);
            outer(cP, base + C::kFix + C::kTile, ring(1));
            done(bar_dp);
            for (int i = 0; i < n; ++i) {
                const bool more = i + 1 < n;
                named_sync(kBarP, 288);
                umma::fence_after_sync();
                inner(cV, cS, ring(2 * i + 1), i > 0);
                done(bar_empty + 8 * slot_of(2 * i + 1));
                if (more) {
                    ready(i + 1);
                    outer(cS, base + C::kFix, ring(2 * i + 2));
                    done(bar_s);
                }
                named_sync(kBarDs, 288);
                umma::fence_after_sync();
                inner(cK, cP, ring(2 * i), i > 0);
                done(bar_empty + 8 * slot_of(2 * i));
                if (more) {
                    outer(cP, base + C::kFix + C::kTile, ring(2 * i + 3));
                    done(bar_dp);
                }
            }
            done(bar_done);
        } else if (warp == 10) {
            // ---- row stats of each tile (rows behind the sequence: probability 0) in two stages, and "scores ready",
            //      "score gradients ready" passed on to the elementwise warps.  dP of tile i + 1 is formed after dS of
            //      tile i is complete, so by then the stage of tile i has been read.
            auto load = [&](int i, float2 (&x)[4]) {
                const int r0 = first_row(i), hg = h0 + ((i / per) << lpack);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int r = lane + 32 * y, p = r0 + (r >> lpack);
                    x[y] = p < B.lq ? __ldg(stats + (B.q0 + p) * A.Hq + hg + (r & ((1 << lpack) - 1)))
                                    : make_float2(-INFINITY, 0.f);
                }
            };
            float2 x[4];
            if (n > 0) load(0, x);
            for (int i = 0; i < n; ++i) {
                float* st = reinterpret_cast<float*>(sm + C::kStat + (i & 1) * 1024);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    st[lane + 32 * y] = x[y].x;
                    st[128 + lane + 32 * y] = x[y].y;
                }
                if (i + 1 < n) load(i + 1, x);
                ok = ok && wait_or_flag(bar_s, i & 1, err);
                umma::fence_after_sync();
                umma::fence_before_sync();
                named_arrive(kBarS, 288);
                ok = ok && wait_or_flag(bar_dp, i & 1, err);
                umma::fence_after_sync();
                umma::fence_before_sync();
                named_arrive(kBarDp, 288);
            }
        }
        __syncwarp();
    } else {
        take_registers();
        // ---- elementwise: lane = key, this warpgroup's 64 of the tile's 128 rows
        const int half = warp >> 2, key = B.first + (tid & 127);
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const uint32_t tS = cS + lanes + half * 64, tP = cP + lanes + half * 64;
        const float2 c2 = make_float2(A.scale * kLog2e, A.scale * kLog2e);
        for (int i = 0; i < n; ++i) {
            const float* st = reinterpret_cast<const float*>(sm + C::kStat + (i & 1) * 1024) + half * 64;
            // rows from column `from` on see the key: row position >= key - off
            const int from = max(-kRows, min(kRows, key - off - first_row(i))) * (1 << lpack) - half * 64;
            named_sync(kBarS, 288);
            umma::fence_after_sync();
            float2 p[32];
            load64(tS, p);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                const float4 nl = *reinterpret_cast<const float4*>(st + 2 * x);
                const float2 a = ffma2(p[x], c2, make_float2(nl.x, nl.y)), b = ffma2(p[x + 1], c2, make_float2(nl.z, nl.w));
                p[x] = make_float2(ex2(a.x), ex2(a.y));
                p[x + 1] = make_float2(ex2(b.x), ex2(b.y));
            }
            if (__any_sync(0xffffffffu, from > 0)) {
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    p[x].x = 2 * x >= from ? p[x].x : 0.f;
                    p[x].y = 2 * x + 1 >= from ? p[x].y : 0.f;
                }
            }
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) w[x] = pack_bf2(p[x].x, p[x].y);
            umma::tmem_st32_async(tS, w);
            umma::tmem_wait_st();
            umma::fence_before_sync();
            named_arrive(kBarP, 288);
            named_sync(kBarDp, 288);
            umma::fence_after_sync();
            float2 d[32];
            load64(tP, d);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                const float4 nd = *reinterpret_cast<const float4*>(st + 128 + 2 * x);
                const float2 a = fmul2(p[x], fadd2(d[x], make_float2(nd.x, nd.y)));
                const float2 b = fmul2(p[x + 1], fadd2(d[x + 1], make_float2(nd.z, nd.w)));
                w[x] = pack_bf2(a.x, a.y);
                w[x + 1] = pack_bf2(b.x, b.y);
            }
            umma::tmem_st32_async(tP, w);
            umma::tmem_wait_st();
            umma::fence_before_sync();
            named_arrive(kBarDs, 288);
        }
        // ---- results: dv by the first warpgroup, dk by the second
        if (n > 0) wait_or_flag(bar_done, 0, err);
        umma::fence_after_sync();
        const float mul = half ? A.scale : 1.f;
        __nv_bfloat16* dst = (half ? dk : dv) + ((B.k0 + key) * A.Hkv + kv) * D;
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            float o[32];
            if (n > 0) {
                umma::tmem_ld32((half ? cK : cV) + lanes + 32 * b, o);
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = 0.f;
            }
            if (key < B.lk) {
#pragma unroll
                for (int x = 0; x < 32; x += 8)
                    *reinterpret_cast<uint4*>(dst + 32 * b + x) =
                        make_uint4(pack_bf2(o[x] * mul, o[x + 1] * mul), pack_bf2(o[x + 2] * mul, o[x + 3] * mul),
                                   pack_bf2(o[x + 4] * mul, o[x + 5] * mul), pack_bf2(o[x + 6] * mul, o[x + 7] * mul));
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

// ---- dq ---------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attn_dq_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const int32_t* __restrict__ cu_q,
                  const int32_t* __restrict__ cu_k, int lpack, const float2* __restrict__ stats,
                  __nv_bfloat16* __restrict__ dq, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int qb = kRows >> lpack, n_hg = A.Hq >> lpack;
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, qb, blockIdx.x / n_hg, false);
    if (!B.found) return;  // the whole block
    const int h0 = (int)(blockIdx.x % n_hg) << lpack, kv = h0 / A.G, off = B.lk - B.lq;
    const int end = max(0, min(B.lk, min(B.first + qb, B.lq) + off));
    const int n = __shfl_sync(0xffffffffu, (end + kRows - 1) / kRows, 0);

    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_q = bars, bar_full = bars + 8, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_se = bar_s + 16, bar_dp = bar_se + 16, bar_fix = bar_dp + 8;
    const uint32_t bar_done = bar_fix + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 248);
    if (tid == 0) {
        umma::mbar_init(bar_q, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar_s + 8 * i, 1);
            umma::mbar_init(bar_se + 8 * i, 8);
        }
        umma::mbar_init(bar_dp, 1);
        umma::mbar_init(bar_fix, 1);
        umma::mbar_init(bar_done, 1);
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t cS = tmem, cP = tmem + 256, cQ = tmem + 384;  // S (two buffers), dP / dS, dQ
    auto slot_of = [&](int use) { return use % C::kSlots; };
    auto par_of = [&](int use) { return (uint32_t)(use / C::kSlots) & 1u; };

    if (warp >= 8) {
        give_registers();
        bool ok = true;
        if (warp == 8 && n > 0) {
            // ---- loads: use 2 i of the ring is K tile i, use 2 i + 1 is V tile i
            if (lane == 0) {
                tma::expect_tx(bar_q, 2 * C::kTile);
                for (int b = 0; b < D / 64; ++b) {
                    tma::tensor_load_3d(base + C::kFix + b * (kRows * 128), &map_q, 64 * b, h0, (int)(B.q0 + B.first),
                                        bar_q);
                    tma::tensor_load_3d(base + C::kFix + C::kTile + b * (kRows * 128), &map_do, 64 * b, h0,
                                        (int)(B.q0 + B.first), bar_q);
                }
            }
            int u = 0;
            for (; u < 2 * n; ++u) {
                const int slot = slot_of(u);
                if (u >= C::kSlots && !(ok = wait_or_flag(bar_empty + 8 * slot, par_of(u - C::kSlots), err))) break;
                if (lane == 0) {
                    tma::expect_tx(bar_full + 8 * slot, C::kTile);
                    for (int b = 0; b < D / 64; ++b)
                        tma::tensor_load_3d(base + C::kRing + slot * C::kTile + b * (kRows * 128),
                                            u & 1 ? &map_v : &map_k, 64 * b, kv, (int)B.k0 + (u >> 1) * kRows,
                                            bar_full + 8 * slot);
                }
            }
            if (ok) {  // keys behind the last visible one: cleared, whatever they hold (dS is 0 there)
                const int y = 2 * (n - 1);
                ok = wait_or_flag(bar_full + 8 * slot_of(y), par_of(y), err);
                if (ok) zero_rows<D>(sm + C::kRing + slot_of(y) * C::kTile, end - (n - 1) * kRows);
                umma::fence_async_smem();
                __syncwarp();
                if (ok && lane == 0) umma::mbar_arrive(bar_fix);
            }
            if (!ok) {  // copies in flight land before the block ends
                wait_or_flag(bar_q, 0, err);
                for (int i = max(0, u - C::kSlots); i < u; ++i) wait_or_flag(bar_full + 8 * slot_of(i), par_of(i), err);
            }
        } else if (warp == 9 && n > 0) {
            // ---- products: one lane issues, the warp stays together
            const uint32_t lead = umma::elect_one();
            const uint32_t id_s = umma::idesc_bf16(kRows, kRows, false, false);
            const uint32_t id_d = umma::idesc_bf16(kRows, D, false, true);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar, parity, err));
            };
            auto ring = [&](int u) { return base + C::kRing + slot_of(u) * C::kTile; };
            auto outer = [&](uint32_t d, uint32_t a_tile, uint32_t b_tile) {
                if (!ok) return;
                const uint64_t a = umma::kmajor(a_tile, kRows, 0), b = umma::kmajor(b_tile, kRows, 0);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t ks = (uint64_t)((s >> 2) * (kRows * 128 / 16) + (s & 3) * 2);
                    umma::mma_lead(d, a + ks, b + ks, id_s, s > 0, lead);
                }
            };
            auto done = [&](uint32_t bar) {
                if (ok && lead) umma::commit(bar);
            };
            auto score = [&](int i) {  // S of tile i into its buffer, free once tile i - 2 has been read
                if (i >= 2) wait(bar_se + 8 * (i & 1), ((i >> 1) - 1) & 1);
                wait(bar_full + 8 * slot_of(2 * i), par_of(2 * i));
                if (i == n - 1) wait(bar_fix, 0);
                umma::fence_after_sync();
                outer(cS + (i & 1) * 128, base + C::kFix, ring(2 * i));
                done(bar_s + 8 * (i & 1));
            };
            auto grad = [&](int i) {  // dP of tile i
                wait(bar_full + 8 * slot_of(2 * i + 1), par_of(2 * i + 1));
                umma::fence_after_sync();
                outer(cP, base + C::kFix + C::kTile, ring(2 * i + 1));
                done(bar_dp);
                done(bar_empty + 8 * slot_of(2 * i + 1));
            };
            wait(bar_q, 0);
            score(0);
            grad(0);
            if (n > 1) score(1);
            for (int i = 0; i < n; ++i) {
                named_sync(kBarDs, 288);
                umma::fence_after_sync();
                if (ok) {
                    const uint64_t b = umma::mnmajor(ring(2 * i), kRows * 128, 0);
#pragma unroll
                    for (int s = 0; s < kRows / 16; ++s)
                        umma::mma_ts_lead(cQ, half_step(cP, s), b + (uint64_t)(s * 128), id_d, i > 0 || s > 0, lead);
                }
                done(bar_empty + 8 * slot_of(2 * i));
                if (i + 1 < n) grad(i + 1);
                if (i + 2 < n) score(i + 2);
            }
            done(bar_done);
        } else if (warp == 10) {
            // ---- "scores ready", "score gradients ready" passed on to the elementwise warps.  Scores run one tile
            //      ahead: two barriers, so that a slow warp never meets the signal of the tile after its own (the one
            //      after that waits until every warp has read this tile's scores)
            for (int i = 0; i < n; ++i) {
                ok = ok && wait_or_flag(bar_s + 8 * (i & 1), (i >> 1) & 1, err);
                umma::fence_after_sync();
                umma::fence_before_sync();
                named_arrive(kBarS + (i & 1), 288);
                ok = ok && wait_or_flag(bar_dp, i & 1, err);
                umma::fence_after_sync();
                umma::fence_before_sync();
                named_arrive(kBarDp, 288);
            }
        }
        __syncwarp();
    } else {
        take_registers();
        // ---- elementwise: lane = row, this warpgroup's 64 of the tile's 128 keys
        const int half = warp >> 2, row = tid & 127, pos = B.first + (row >> lpack), h = h0 + (row & ((1 << lpack) - 1));
        const bool on = pos < B.lq;
        const int limit = on ? min(B.lk, pos + off + 1) : 0;
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const uint32_t tP = cP + lanes + half * 64;
        const int64_t at = (B.q0 + pos) * A.Hq + h;
        const float2 st = on ? __ldg(stats + at) : make_float2(-INFINITY, 0.f);
        const float2 c2 = make_float2(A.scale * kLog2e, A.scale * kLog2e);
        const float2 nl = make_float2(st.x, st.x), nd = make_float2(st.y, st.y);
        for (int i = 0; i < n; ++i) {
            const int seen = limit - i * kRows - half * 64;
            const bool edge = __any_sync(0xffffffffu, seen < 64);
            named_sync(kBarS + (i & 1), 288);
            umma::fence_after_sync();
            float2 p[32];
            load64(cS + (i & 1) * 128 + lanes + half * 64, p);
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(bar_se + 8 * (i & 1));
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const float2 a = ffma2(p[x], c2, nl);
                p[x] = make_float2(ex2(a.x), ex2(a.y));
            }
            named_sync(kBarDp, 288);
            umma::fence_after_sync();
            float2 d[32];
            load64(tP, d);
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                float2 a = fmul2(p[x], fadd2(d[x], nd));
                if (edge) {
                    a.x = 2 * x < seen ? a.x : 0.f;
                    a.y = 2 * x + 1 < seen ? a.y : 0.f;
                }
                w[x] = pack_bf2(a.x, a.y);
            }
            umma::tmem_st32_async(tP, w);
            umma::tmem_wait_st();
            umma::fence_before_sync();
            named_arrive(kBarDs, 288);
        }
        if (n > 0) wait_or_flag(bar_done, 0, err);
        umma::fence_after_sync();
        // ---- results: half of the columns each
        __nv_bfloat16* dst = dq + at * D + half * (D / 2);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
            float o[32];
            if (n > 0) {
                umma::tmem_ld32(cQ + lanes + half * (D / 2) + 32 * b, o);
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = 0.f;
            }
            if (on) {
#pragma unroll
                for (int x = 0; x < 32; x += 8)
                    *reinterpret_cast<uint4*>(dst + 32 * b + x) = make_uint4(
                        pack_bf2(o[x] * A.scale, o[x + 1] * A.scale), pack_bf2(o[x + 2] * A.scale, o[x + 3] * A.scale),
                        pack_bf2(o[x + 4] * A.scale, o[x + 5] * A.scale), pack_bf2(o[x + 6] * A.scale, o[x + 7] * A.scale));
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

template <int D>
cudaError_t launch(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                   const __nv_bfloat16* out, const float* lse, const __nv_bfloat16* dout, const int32_t* cu_q,
                   const int32_t* cu_k, __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, float2* stats,
                   int32_t* err, cudaStream_t st) {
    static DeviceCache c1, c2;
    cudaError_t e = device_cached(c1, nullptr, [](int, int*) { return prepare_kernel(attn_dkdv_tc_kernel<D>, Cfg<D>::kSmem); });
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
    const int64_t rows = A.total_q * A.Hq, kb = (A.total_k / kRows + A.n_seqs) * A.Hkv,
                  qblocks = (A.total_q / qb + A.n_seqs) * (A.Hq / pack), sb = (rows * (D / 8) + 255) / 256;
    if (kb > INT32_MAX || qblocks > INT32_MAX || sb > INT32_MAX) return cudaErrorInvalidValue;
    attn_stats_kernel<D><<<(unsigned)sb, 256, 0, st>>>(rows, out, dout, lse, stats);
    attn_dkdv_tc_kernel<D><<<(unsigned)kb, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mo, mk, mv, cu_q, cu_k, lpack, stats, dk,
                                                                       dv, err);
    attn_dq_tc_kernel<D><<<(unsigned)qblocks, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mo, mk, mv, cu_q, cu_k, lpack, stats,
                                                                          dq, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                         const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                         const __nv_bfloat16* dout, const int32_t* cu_q, const int32_t* cu_k,
                                         __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, float2* stats,
                                         int32_t* err, cudaStream_t st) {
    return A.d == 128 ? launch<128>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, stats, err, st)
                      : launch<64>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, stats, err, st);
}

}  // namespace hla
