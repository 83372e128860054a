// Packed causal attention of bf16 layers on the tcgen05 tensor cores:
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  out = O / sum P
// in one pass over the keys with the running reference m and sum.
//
// A block takes two query tiles (128 rows each, see attention_tc.cuh) of one
// kv head and walks the keys they see in tiles of 128:
//   warp 8        TMA: both query tiles, then K and V tiles into a ring of
//                 slots; clears the value rows behind the last visible key
//   warp 9        one thread issues every product; S of both tiles (128
//                 columns each) and O of both (d columns each) in TMEM
//   warps 0 - 3   softmax of tile 0, one row per thread
//   warps 4 - 7   the same of tile 1
// While the tensor cores form P V and the next S of one tile (the probabilities
// overwrite the first half of their scores' columns and are read from TMEM as
// the A operand), the other tile's softmax runs.
//
// The reference m follows the running maximum only when it has grown by more
// than 2^8 (the sum and O use the same m, so the result is the same); a row's
// O is then rescaled in TMEM by its own softmax thread, after the products
// before it have completed (they complete before the scores it waits for).
//
// Bound by the tensor cores (4 d flops per visible score) together with the
// softmax's issue slots (about 4 instructions and one exponential per score).
#include "attention_tc.cuh"

namespace hla {

namespace {

using namespace attn_tc;

constexpr float kLazy = 8.0f;
constexpr int kBarS = 1, kBarP = 3;  // hardware barriers: scores ready, probabilities ready (+ tile)

template <int D> struct Cfg {
    static constexpr uint32_t kTile = kRows * D * 2;  // bytes of a tile
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTile, kBar = kRing + kSlots * kTile;
    static constexpr uint32_t kSmem = kBar + 256 + 1024;
    // TMEM columns
    static constexpr uint32_t kS = 0, kO = 256, kCols = 512;
};

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attention_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int lpack,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int pack = 1 << lpack, qb = kRows >> lpack, n_hg = A.Hq >> lpack;
    if (blockIdx.x == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, 2 * qb, blockIdx.x / n_hg, false);
    if (!B.found) return;  // the whole block
    const int hg = blockIdx.x % n_hg, h0 = hg << lpack, kv = h0 / A.G;
    const int off = B.lk - B.lq;
    // positions of tile t: [first + t qb, ...); keys it sees: [0, end(t))
    auto key_end = [&](int t) {
        const int p0 = B.first + t * qb;
        return p0 < B.lq ? max(0, min(B.lk, min(p0 + qb, B.lq) + off)) : 0;
    };
    const int end0 = key_end(0), end1 = key_end(1), end = max(end0, end1);
    const int n0 = __shfl_sync(0xffffffffu, (end0 + kRows - 1) / kRows, 0);
    const int n1 = __shfl_sync(0xffffffffu, (end1 + kRows - 1) / kRows, 0), n = max(n0, n1);

    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_q = bars, bar_full = bars + 16, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_o = bar_s + 16, bar_fix = bar_o + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 248);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar_q + 8 * i, 1);
            umma::mbar_init(bar_s + 8 * i, 1);
            umma::mbar_init(bar_o + 8 * i, 1);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        umma::mbar_init(bar_fix, 1);
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp >= 8) {
    give_registers();
    if (warp == 8) {
        // ---- loads: use u of the ring is K tile u / 2 (even) or V tile u / 2 (odd)
        bool ok = true;
        int issued = 0;
        const int uses = 2 * n;
        if (lane == 0 && n > 0) {
            for (int t = 0; t < 2; ++t) {
                const int p0 = B.first + t * qb;
                if ((t ? n1 : n0) == 0) continue;
                tma::expect_tx(bar_q + 8 * t, C::kTile);
                for (int b = 0; b < D / 64; ++b)
                    tma::tensor_load_3d(base + C::kQ + t * C::kTile + b * (kRows * 128), &map_q, 64 * b, h0,
                                        (int)(B.q0 + p0), bar_q + 8 * t);
            }
            for (; issued < uses && ok; ++issued) {
                const int slot = issued % C::kSlots, round = issued / C::kSlots;
                if (round > 0 && !(ok = wait_or_flag(bar_empty + 8 * slot, (round - 1) & 1, err))) break;
                tma::expect_tx(bar_full + 8 * slot, C::kTile);
                const int tk = (int)B.k0 + (issued >> 1) * kRows;
                for (int b = 0; b < D / 64; ++b)
                    tma::tensor_load_3d(base + C::kRing + slot * C::kTile + b * (kRows * 128),
                                        issued & 1 ? &map_v : &map_k, 64 * b, kv, tk, bar_full + 8 * slot);
            }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        if (n > 0 && ok) {
            // the last V tile: rows behind the last visible key weigh 0; clear them, whatever they hold
            const int u = uses - 1, slot = u % C::kSlots;
            ok = wait_or_flag(bar_full + 8 * slot, (u / C::kSlots) & 1, err);
            zero_rows<D>(sm + C::kRing + slot * C::kTile, end - (n - 1) * kRows);
            umma::fence_async_smem();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(bar_fix);
        }
        if (!ok && lane == 0)  // copies in flight land before the block ends
            for (int i = max(0, issued - C::kSlots); i < issued; ++i)
                wait_or_flag(bar_full + 8 * (i % C::kSlots), (i / C::kSlots) & 1, err);
    } else if (warp == 9) {
        // ---- products: one lane issues, the warp stays together
        const uint32_t lead = umma::elect_one();
        const uint32_t id_s = umma::idesc_bf16(kRows, kRows, false, false);
        const uint32_t id_o = umma::idesc_bf16(kRows, D, false, true);
        bool ok = true;
        auto full = [&](int u) {
            ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar_full + 8 * (u % C::kSlots), (u / C::kSlots) & 1, err));
        };
        auto scores = [&](int t, int j) {
            if (!ok) return;
            const uint32_t kb = base + C::kRing + ((2 * j) % C::kSlots) * C::kTile;
            const uint64_t a = umma::kmajor(base + C::kQ + t * C::kTile, kRows, 0), b = umma::kmajor(kb, kRows, 0);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint64_t ks = (uint64_t)((s >> 2) * (kRows * 128 / 16) + (s & 3) * 2);
                umma::mma_lead(tmem + C::kS + t * kRows, a + ks, b + ks, id_s, s > 0, lead);
            }
            if (lead) umma::commit(bar_s + 8 * t);
        };
        auto values = [&](int t, int j) {
            if (!ok) return;
            const uint32_t vb = base + C::kRing + ((2 * j + 1) % C::kSlots) * C::kTile;
            const uint64_t b = umma::mnmajor(vb, kRows * 128, 0);
#pragma unroll
            for (int s = 0; s < kRows / 16; ++s)
                umma::mma_ts_lead(tmem + C::kO + t * D, tmem + C::kS + t * kRows + 8 * s, b + (uint64_t)(s * 128),
                                  id_o, j > 0 || s > 0, lead);
        };
        auto done = [&](uint32_t bar) {
            if (ok && lead) umma::commit(bar);
        };
        if (n > 0) full(0);
        for (int t = 0; t < 2; ++t) {
            if ((t ? n1 : n0) == 0) continue;
            ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar_q + 8 * t, 0, err));
            umma::fence_after_sync();
            scores(t, 0);
        }
        if (n > 0) done(bar_empty);
        for (int j = 0; j < n; ++j) {
            const bool more = j + 1 < n;
            full(2 * j + 1);
            if (more) full(2 * j + 2);
            else ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar_fix, 0, err));
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? n1 : n0;
                if (j >= nt) continue;
                named_sync(kBarP + t, 160);
                umma::fence_after_sync();
                values(t, j);
                if (j + 1 < nt) scores(t, j + 1);
                else done(bar_o + 8 * t);
            }
            done(bar_empty + 8 * ((2 * j + 1) % C::kSlots));
            if (more) done(bar_empty + 8 * ((2 * j + 2) % C::kSlots));
        }
    } else {
        // ---- warps 10, 11: pass "scores ready" of tile 0, 1 on to its softmax warps
        const int t = warp - 10, nt = t ? n1 : n0;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            ok = ok && wait_or_flag(bar_s + 8 * t, j & 1, err);
            umma::fence_after_sync();
            umma::fence_before_sync();
            named_arrive(kBarS + t, 160);
        }
    }
    } else {
        take_registers();
        // ---- softmax, one row per thread
        const int t = warp >> 2, row = tid & 127, pos = B.first + t * qb + (row >> lpack), h = h0 + (row & (pack - 1));
        const int nt = t ? n1 : n0;
        const bool on = pos < B.lq;
        const int limit = on ? min(B.lk, pos + off + 1) : 0;  // keys the row sees: [0, limit)
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const uint32_t ts = tmem + lanes + C::kS + t * kRows, to = tmem + lanes + C::kO + t * D;
        const float cs = A.scale * kLog2e;
        float m = -INFINITY;
        float2 l = make_float2(0.f, 0.f);
        for (int j = 0; j < nt; ++j) {
            named_sync(kBarS + t, 160);
            umma::fence_after_sync();
            float x[128];
            {
                uint32_t r[4][32];
#pragma unroll
                for (int b = 0; b < 4; ++b) umma::tmem_ld32_async(ts + 32 * b, r[b]);
                umma::tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    umma::reg_fence32(r[b]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[32 * b + i] = __uint_as_float(r[b][i]);
                }
            }
            const int seen = limit - j * kRows;
            if (__any_sync(0xffffffffu, seen < kRows)) {
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i] = i < seen ? x[i] : -INFINITY;
            }
            float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < 128; i += 8)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (i + b + 4 < 128) top[b] = fmaxf(top[b], fmaxf(x[i + b], x[i + b + 4]));
                    else top[b] = fmaxf(top[b], x[i + b]);
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cs;
            const bool grow = mx > m + kLazy;
            if (__any_sync(0xffffffffu, grow)) {
                const float corr = grow ? (m == -INFINITY ? 0.f : ex2(m - mx)) : 1.f;
                if (grow) m = mx;
                l.x *= corr;
                l.y *= corr;
                if (j > 0) {
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) {
                        float o[32];
                        umma::tmem_ld32(to + 32 * b, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= corr;
                        umma::tmem_st32(to + 32 * b, o);
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const float2 c2 = make_float2(cs, cs), m2 = make_float2(-ref, -ref);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 y = ffma2(make_float2(x[64 * b + 2 * i], x[64 * b + 2 * i + 1]), c2, m2);
                    const float2 e = make_float2(ex2(y.x), ex2(y.y));
                    l = fadd2(l, e);
                    p[i] = pack_bf2(e.x, e.y);
                }
                umma::tmem_st32_async(ts + 32 * b, p);
            }
            umma::tmem_wait_st();
            umma::fence_before_sync();
            named_arrive(kBarP + t, 160);
        }
        // ---- the row's output
        const float sum = l.x + l.y;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = (B.q0 + pos) * A.Hq + h;
        if (on) lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        if (nt > 0) wait_or_flag(bar_o + 8 * t, 0, err);
        umma::fence_after_sync();
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            float o[32];
            if (nt > 0) {
                umma::tmem_ld32(to + 32 * b, o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (on) {
                __nv_bfloat16* dst = out + at * D + 32 * b;
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                    *reinterpret_cast<uint4*>(dst + i) =
                        make_uint4(pack_bf2(o[i] * inv, o[i + 1] * inv), pack_bf2(o[i + 2] * inv, o[i + 3] * inv),
                                   pack_bf2(o[i + 4] * inv, o[i + 5] * inv), pack_bf2(o[i + 6] * inv, o[i + 7] * inv));
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

template <int D>
cudaError_t launch(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                   const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out, float* lse, int32_t* err,
                   cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [](int, int*) {
        return prepare_kernel(attention_tc_kernel<D>, Cfg<D>::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int pack = pack_of(A.G), qb = kRows / pack;
    int lpack = 0;
    while ((1 << lpack) < pack) ++lpack;
    CUtensorMap mq, mk, mv;
    if (!tma::make_map_3d_strided(&mq, q, true, D, (uint64_t)A.Hq, (uint64_t)A.total_q, (uint64_t)A.sq * 2, 64,
                                  (uint32_t)pack, (uint32_t)qb) ||
        !tma::make_map_3d_strided(&mk, k, true, D, (uint64_t)A.Hkv, (uint64_t)A.total_k, (uint64_t)A.sk * 2, 64, 1,
                                  kRows) ||
        !tma::make_map_3d_strided(&mv, v, true, D, (uint64_t)A.Hkv, (uint64_t)A.total_k, (uint64_t)A.sv * 2, 64, 1,
                                  kRows))
        return cudaErrorInvalidValue;
    const int64_t blocks = (A.total_q / (2 * qb) + A.n_seqs) * (A.Hq / pack);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    attention_tc_kernel<D><<<(unsigned)blocks, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mk, mv, cu_q, cu_k, lpack, out,
                                                                             lse, err);
    return cudaGetLastError();
}

}  // namespace

bool attention_tc_supported(const AttnDims& A) { return A.total_q > 0 && A.total_k > 0; }

cudaError_t launch_attention_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out,
                                float* lse, int32_t* err, cudaStream_t st) {
    return A.d == 128 ? launch<128>(A, q, k, v, cu_q, cu_k, out, lse, err, st)
                      : launch<64>(A, q, k, v, cu_q, cu_k, out, lse, err, st);
}

}  // namespace hla
