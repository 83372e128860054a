// Decode step of a full softmax layer: one query token per sequence over the
// paged cache.  See attention_decode.cuh for the cut over blocks.
#include <cuda_fp8.h>

#include <algorithm>

#include "attention_decode.cuh"

namespace hla {

namespace {

constexpr int kThreads = 128;
constexpr int kGroup = 8;  // query heads of a kv head per block

// ---- fp32 layers ------------------------------------------------------------
//
// Scores: eight lanes per key, D / 8 values each, partial dot products joined
// by three shuffles.  Values: a thread per column pair, the weights read from
// shared memory.  All in fp32.
template <bool E4M3, int D>
__global__ void __launch_bounds__(kThreads)
decode_f32_kernel(AttnDims A, CacheDims C, hla_cache c, const float* __restrict__ q, DecodeLine L,
                  float* __restrict__ out, DecodePart part) {
    constexpr int E = D / 8;  // elements of a key per lane
    __shared__ float qs[kGroup][D];
    __shared__ float ps[kGroup][kDecodeUnit];  // scores, then weights
    __shared__ float vs[kDecodeUnit];          // scale of each value row
    __shared__ int64_t rows[kDecodeUnit];      // cache rows (-1: none)
    __shared__ float stats[kGroup][2];         // running max, correction
    __shared__ float osum[kThreads / 32][kGroup][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kv = blockIdx.y, g0 = blockIdx.z * kGroup, ng = min(kGroup, A.G - g0);
    pdl_trigger();
    if (blockIdx.x == 0 && kv == 0 && g0 == 0) {  // lengths out of range
        bool bad = false;
        for (int s = tid; s < L.n_seqs; s += kThreads) bad |= __ldg(L.lens + s) < 0 || __ldg(L.lens + s) > L.cap;
        if (bad) atomicExch(c.err, kErrState);
    }
    const int64_t U = line_units(L, 0, nullptr), nb = min((int64_t)gridDim.x, U);
    if (blockIdx.x >= nb) return;
    int64_t u = blockIdx.x * U / nb;
    const int64_t u1 = (blockIdx.x + 1) * U / nb;
    int64_t useq;
    int s = line_find(L, u, &useq);
    const int64_t u0 = u;
    while (u < u1) {
        const int64_t len = L.len(s), su = (len + kDecodeUnit - 1) / kDecodeUnit;
        if (su == 0) { ++s; continue; }
        const int64_t e = min(u1, useq + su);  // this block's units of the sequence: [u, e)
        __syncthreads();
        for (int i = tid; i < ng * D; i += kThreads)
            qs[i / D][i % D] = __ldg(q + (int64_t)s * A.sq + (int64_t)(kv * A.G + g0 + i / D) * D + i % D) *
                               (A.scale * kLog2e);
        // a warp sums every fourth key of a unit; lane owns D / 32 columns
        float acc[kGroup][D / 32];
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int x = 0; x < D / 32; ++x) acc[g][x] = 0.f;
        float mrun = -INFINITY, lrun = 0.f;  // threads 0..ng-1: head tid
        for (int64_t w = u; w < e; ++w) {
            const int64_t p0 = (w - useq) * kDecodeUnit;
            const int n = (int)min((int64_t)kDecodeUnit, len - p0);
            __syncthreads();
            if (tid < kDecodeUnit) {
                int64_t r = -1;
                if (tid < n) {
                    const int64_t p = p0 + tid;
                    const int page = __ldg(c.page_table + (int64_t)s * C.max_pages + p / C.page);
                    if (page >= 0 && page < C.n_pages) r = ((int64_t)page * C.Hkv + kv) * C.page + p % C.page;
                    else atomicExch(c.err, kErrState);
                }
                rows[tid] = r;
                if constexpr (E4M3) vs[tid] = r >= 0 ? exp2f((float)((int)c.v_exp[r] - 127)) : 0.f;
                else vs[tid] = 1.f;
            }
            __syncthreads();
            for (int j = tid / 8; j < kDecodeUnit; j += kThreads / 8) {
                const int64_t r = rows[j];
                float kx[E];
                float ks = 1.f;
                if (r >= 0) {
                    if constexpr (E4M3) {
                        ks = exp2f((float)((int)c.k_exp[r] - 127));
                        const uint8_t* src = static_cast<const uint8_t*>(c.k) + r * D + (tid & 7) * E;
#pragma unroll
                        for (int x = 0; x < E; x += 2) {
                            const __half2_raw hv = __nv_cvt_fp8x2_to_halfraw2(
                                *reinterpret_cast<const __nv_fp8x2_storage_t*>(src + x), __NV_E4M3);
                            const float2 f = __half22float2(__half2(hv));
                            kx[x] = f.x;
                            kx[x + 1] = f.y;
                        }
                    } else {
                        const float* src = static_cast<const float*>(c.k) + r * D + (tid & 7) * E;
#pragma unroll
                        for (int x = 0; x < E; x += 4) load_vec<4>(src + x, kx + x);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < E; ++x) kx[x] = 0.f;
                }
                for (int g = 0; g < ng; ++g) {
                    float d = 0.f;
#pragma unroll
                    for (int x = 0; x < E; ++x) d = fmaf(qs[g][(tid & 7) * E + x], kx[x], d);
#pragma unroll
                    for (int o = 4; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if ((tid & 7) == 0) ps[g][j] = r >= 0 ? d * ks : -INFINITY;
                }
            }
            __syncthreads();
            if (tid < ng) {
                float m = mrun;
                for (int j = 0; j < n; ++j) m = fmaxf(m, ps[tid][j]);
                const float corr = mrun == -INFINITY ? 0.f : exp2f(mrun - m);
                float sum = 0.f;
                for (int j = 0; j < kDecodeUnit; ++j) {
                    const float p = j < n && ps[tid][j] != -INFINITY ? exp2f(ps[tid][j] - m) : 0.f;
                    sum += p;
                    ps[tid][j] = p;
                }
                lrun = lrun * corr + sum;
                mrun = m;
                stats[tid][1] = corr;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kGroup; ++g)
                if (g < ng)
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) acc[g][x] *= stats[g][1];
            for (int j = warp; j < n; j += kThreads / 32) {
                const int64_t r = rows[j];
                if (r < 0) continue;
                float vx[D / 32];
                if constexpr (E4M3) {
                    const uint8_t* src = static_cast<const uint8_t*>(c.v) + r * D + lane * (D / 32);
#pragma unroll
                    for (int x = 0; x < D / 32; x += 2) {
                        const __half2_raw hv = __nv_cvt_fp8x2_to_halfraw2(
                            *reinterpret_cast<const __nv_fp8x2_storage_t*>(src + x), __NV_E4M3);
                        const float2 f = __half22float2(__half2(hv));
                        vx[x] = f.x * vs[j];
                        vx[x + 1] = f.y * vs[j];
                    }
                } else {
                    load_vec<D / 32>(static_cast<const float*>(c.v) + r * D + lane * (D / 32), vx);
                }
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    if (g < ng) {
                        const float p = ps[g][j];
#pragma unroll
                        for (int x = 0; x < D / 32; ++x) acc[g][x] = fmaf(p, vx[x], acc[g][x]);
                    }
            }
        }
        // join the warps; the block's part of the sequence
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
            if (g < ng)
#pragma unroll
                for (int x = 0; x < D / 32; ++x) osum[warp][g][lane * (D / 32) + x] = acc[g][x];
        if (tid < ng) {
            stats[tid][0] = mrun;
            stats[tid][1] = lrun;
        }
        __syncthreads();
        const bool whole = u == useq && e == useq + su;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (u == u0 ? 0 : 1);
        for (int i = tid; i < ng * D; i += kThreads) {
            const int g = i / D, x = i % D, h = kv * A.G + g0 + g;
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) o += osum[w][g][x];
            if (whole) out[((int64_t)s * A.Hq + h) * D + x] = stats[g][1] == 0.f ? 0.f : o / stats[g][1];
            else part.o[(slot * A.Hq + h) * D + x] = o;
        }
        if (!whole && tid < ng) {
            float* t = part.st + (slot * A.Hq + kv * A.G + g0 + tid) * 4;
            t[0] = mrun;
            t[1] = lrun;
            t[2] = mrun;
        }
        u = e;
        useq += su;
        ++s;
    }
}

// ---- bf16 layers ------------------------------------------------------------
//
// Memory bound, so the tensor-core instruction is the warp-level one (m16n8k16),
// whose operands can be taken from global memory straight into registers: a
// warp takes 16 keys at a time and forms
//   S^T [16 keys x 8 heads] = K q^T,  O^T [d x 8 heads] += V^T P^T.
// The order of d inside a product is free, so each lane loads 16-byte pieces
// of its two key rows and reads the query in the same order; P^T comes from
// S^T by an 8 x 8 transpose in registers.  The next keys are loaded as soon as
// this tile's scores are formed, the next values as soon as these are used:
// no shared memory, no block-wide barrier until a sequence ends.
//
// E4M3 rows become fp16 exactly.  The query is scaled by a power of two per
// head into fp16 (bf16 has 8 bits, fp16 11; elements 2^-14 below the largest
// lose bits of 2^-25 of it).  A key row's power of two goes onto its score, a
// value row's into the exponent of its weight: weights are 2^(s - M) 2^ev /
// 2^(Mt - M), with a reference Mt of their own, so rows of any size meet in
// fp16 (11 bits) with the largest product near 1.  bf16 caches: products and
// weights in bf16 (8 bits, the values' own precision).
//
// References are raised only when a score exceeds them by 2^8 (a vote per
// tile, no reduction); the weights stay at most 2^8.

constexpr float kLazy = 8.0f;

__device__ __forceinline__ uint32_t h2_from_e4m3(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
__device__ __forceinline__ float bf16_at(uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); }
__device__ __forceinline__ float safe_ref(float m) { return m == -INFINITY ? 0.f : m; }

template <bool E4M3, int D>
__global__ void __launch_bounds__(kThreads, E4M3 ? 4 : 3)
decode_mma_kernel(AttnDims A, CacheDims C, hla_cache c, const __nv_bfloat16* __restrict__ q, DecodeLine L,
                  __nv_bfloat16* __restrict__ out, DecodePart part) {
    constexpr int kRow = D * (E4M3 ? 1 : 2);      // bytes of a cache row
    constexpr int kKp = kRow / 64;                // 16-byte pieces of a key row per lane
    constexpr int kVw = kRow / 32;                // 32-bit words of a value row per lane
    constexpr int kSteps = D / 16, kMt = D / 16;  // k steps of the scores; d tiles of the output
    constexpr int kWarps = kThreads / 32;
    __shared__ float osum[kWarps][kGroup][D + 4];
    __shared__ float refs[kWarps][kGroup][3];     // M, sum, Mt
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int kv = blockIdx.y, g0 = blockIdx.z * kGroup, ng = min(kGroup, A.G - g0);
    pdl_trigger();
    if (blockIdx.x == 0 && kv == 0 && g0 == 0) {  // lengths out of range
        bool bad = false;
        for (int s = tid; s < L.n_seqs; s += kThreads) bad |= __ldg(L.lens + s) < 0 || __ldg(L.lens + s) > L.cap;
        if (bad) atomicExch(c.err, kErrState);
    }
    const int64_t U = line_units(L, 0, nullptr), nb = min((int64_t)gridDim.x, U);
    if (blockIdx.x >= nb) return;
    int64_t u = blockIdx.x * U / nb;
    const int64_t u1 = (blockIdx.x + 1) * U / nb, u0 = u;
    int64_t useq;
    int s = line_find(L, u, &useq);
    const int tiles_per_page = C.page / 16;

    while (u < u1) {
        const int64_t len = L.len(s), su = (len + kDecodeUnit - 1) / kDecodeUnit;
        if (su == 0) { ++s; continue; }
        const int64_t e = min(u1, useq + su);  // this block's units of the sequence: [u, e)
        // ---- the query, in the order the key pieces are laid out
        uint32_t qf[kSteps][2];
        float qs0, qs1;  // score factor of heads 2t, 2t + 1 (base-2 logs)
        {
            const __nv_bfloat16* qp = q + (int64_t)s * A.sq + (int64_t)(kv * A.G + g0 + min(g, ng - 1)) * D;
            uint32_t w[D / 8];  // pairs of elements
            if constexpr (E4M3) {
#pragma unroll
                for (int i = 0; i < kKp; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *reinterpret_cast<uint4*>(w + i * 8 + x * 4) =
                            __ldg(reinterpret_cast<const uint4*>(qp + (i * 4 + t) * 16) + x);
            } else {
#pragma unroll
                for (int i = 0; i < kKp; ++i)
                    *reinterpret_cast<uint4*>(w + i * 4) = __ldg(reinterpret_cast<const uint4*>(qp + (i * 4 + t) * 8));
            }
            float qscale = A.scale * kLog2e;
            if constexpr (E4M3) {
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_at(w[i], 0)), fabsf(bf16_at(w[i], 1))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = max(-126, min(126, (int)(__float_as_uint(top) >> 23) - 127));
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                qscale *= __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    w[i] = pack2<true>(bf16_at(w[i], 0) * down, bf16_at(w[i], 1) * down);
            }
            if (g >= ng) qscale = 0.f;
#pragma unroll
            for (int x = 0; x < kSteps; ++x) {
                qf[x][0] = g < ng ? w[2 * x] : 0u;
                qf[x][1] = g < ng ? w[2 * x + 1] : 0u;
            }
            qs0 = __shfl_sync(0xffffffffu, qscale, 8 * t);
            qs1 = __shfl_sync(0xffffffffu, qscale, 8 * t + 4);
        }
        float o[kMt][4];
#pragma unroll
        for (int x = 0; x < kMt; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
        float M0 = -INFINITY, M1 = -INFINITY, T0 = -INFINITY, T1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        // cache row of key 0 of tile i of the sequence; -1: no such tile or page
        auto page_of = [&](int64_t i) -> int {
            return i * 16 < len ? __ldg(c.page_table + (int64_t)s * C.max_pages + i / tiles_per_page) : -1;
        };
        auto row_of = [&](int64_t i, int page) -> int64_t {
            if (i * 16 >= len) return -1;
            if (page < 0 || page >= C.n_pages) {
                if (lane == 0) atomicExch(c.err, kErrState);
                return -1;
            }
            return ((int64_t)page * C.Hkv + kv) * C.page + (i % tiles_per_page) * 16;
        };
        uint4 kx[2][kKp];
        uint32_t vx[4][kVw];
        int ek0 = 0, ek1 = 0, ev0 = 0, ev1 = 0;
        auto load_k = [&](int64_t row) {
            if (row < 0) return;
            const char* p = static_cast<const char*>(c.k) + (row + g) * kRow + t * 16;
#pragma unroll
            for (int i = 0; i < kKp; ++i) {
                kx[0][i] = __ldcs(reinterpret_cast<const uint4*>(p + i * 64));
                kx[1][i] = __ldcs(reinterpret_cast<const uint4*>(p + 8 * kRow + i * 64));
            }
            if constexpr (E4M3) {
                ek0 = c.k_exp[row + g];
                ek1 = c.k_exp[row + g + 8];
                ev0 = c.v_exp[row + g];
                ev1 = c.v_exp[row + g + 8];
            }
        };
        auto load_v = [&](int64_t row, int n) {  // n: keys of the tile; the rows behind them are zeros
            if (row < 0) return;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 2 * t + (x & 1) + 8 * (x >> 1);
                const char* p = static_cast<const char*>(c.v) + (row + key) * kRow;
                if constexpr (kVw == 2) {  // 64 one-byte values: 8 bytes per lane
                    uint2 y = make_uint2(0u, 0u);
                    if (key < n) y = __ldcs(reinterpret_cast<const uint2*>(p + g * 8));
                    vx[x][0] = y.x;
                    vx[x][1] = y.y;
                } else {
#pragma unroll
                    for (int i = 0; i < kVw / 4; ++i) {
                        uint4 y = make_uint4(0u, 0u, 0u, 0u);
                        if (key < n) y = __ldcs(reinterpret_cast<const uint4*>(p + i * 128 + g * 16));
                        vx[x][4 * i] = y.x;
                        vx[x][4 * i + 1] = y.y;
                        vx[x][4 * i + 2] = y.z;
                        vx[x][4 * i + 3] = y.w;
                    }
                }
            }
        };
        // tiles of this warp: 4 unit + warp
        int64_t i = (u - useq) * 4 + warp;
        const int64_t iend = (e - useq) * 4;
        int64_t row = row_of(i, page_of(i));
        int page_next = page_of(i + 4);
        load_k(row);
        load_v(row, (int)min((int64_t)16, len - i * 16));
        for (; i < iend && i * 16 < len; i += 4) {
            const int n = (int)min((int64_t)16, len - i * 16);
            const bool more = i + 4 < iend;
            const int64_t row_next = more ? row_of(i + 4, page_next) : -1;
            page_next = more ? page_of(i + 8) : -1;
            const int n_next = (int)min((int64_t)16, len - (i + 4) * 16);
            if (row >= 0) {
                float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < kKp; ++x) {
                    const uint32_t a[4] = {kx[0][x].x, kx[0][x].y, kx[0][x].z, kx[0][x].w};
                    const uint32_t b[4] = {kx[1][x].x, kx[1][x].y, kx[1][x].z, kx[1][x].w};
                    if constexpr (E4M3) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            mma16816<true>(w & 1 ? sd : sc, h2_from_e4m3(a[w] & 0xffffu), h2_from_e4m3(b[w] & 0xffffu),
                                           h2_from_e4m3(a[w] >> 16), h2_from_e4m3(b[w] >> 16), qf[x * 4 + w][0],
                                           qf[x * 4 + w][1]);
                    } else {
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            mma16816<false>(w & 1 ? sd : sc, a[2 * w], b[2 * w], a[2 * w + 1], b[2 * w + 1],
                                            qf[x * 2 + w][0], qf[x * 2 + w][1]);
                    }
                }
                float f0 = 1.f, f1 = 1.f;  // the key rows' powers of two
                float v0 = 0.f, v1 = 0.f;  // the value rows' exponents
                if constexpr (E4M3) {
                    f0 = ek0 ? __uint_as_float((uint32_t)ek0 << 23) : __uint_as_float(0x400000u);
                    f1 = ek1 ? __uint_as_float((uint32_t)ek1 << 23) : __uint_as_float(0x400000u);
                    v0 = (float)(ev0 - 127);
                    v1 = (float)(ev1 - 127);
                }
                load_k(row_next);
                const bool on0 = g < n, on1 = g + 8 < n;
                float x0 = on0 ? (sc[0] + sd[0]) * f0 * qs0 : -INFINITY, x1 = on0 ? (sc[1] + sd[1]) * f0 * qs1 : -INFINITY;
                float x2 = on1 ? (sc[2] + sd[2]) * f1 * qs0 : -INFINITY, x3 = on1 ? (sc[3] + sd[3]) * f1 * qs1 : -INFINITY;
                float h0 = fmaxf(x0, x2), h1 = fmaxf(x1, x3);
                float t0 = h0, t1 = h1;
                if constexpr (E4M3) {
                    t0 = fmaxf(x0 + v0, x2 + v1);
                    t1 = fmaxf(x1 + v0, x3 + v1);
                }
                bool grow = h0 > M0 + kLazy || h1 > M1 + kLazy;
                if constexpr (E4M3) grow |= t0 > T0 + kLazy || t1 > T1 + kLazy;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) {
                        h0 = fmaxf(h0, __shfl_xor_sync(0xffffffffu, h0, sh));
                        h1 = fmaxf(h1, __shfl_xor_sync(0xffffffffu, h1, sh));
                        if constexpr (E4M3) {
                            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, sh));
                            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, sh));
                        }
                    }
                    const float m0 = fmaxf(M0, h0), m1 = fmaxf(M1, h1);
                    l0 *= M0 == -INFINITY ? 0.f : exp2f(M0 - m0);
                    l1 *= M1 == -INFINITY ? 0.f : exp2f(M1 - m1);
                    M0 = m0;
                    M1 = m1;
                    float r0, r1;
                    if constexpr (E4M3) {
                        const float y0 = fmaxf(T0, t0), y1 = fmaxf(T1, t1);
                        r0 = T0 == -INFINITY ? 0.f : exp2f(T0 - y0);
                        r1 = T1 == -INFINITY ? 0.f : exp2f(T1 - y1);
                        T0 = y0;
                        T1 = y1;
                    } else {
                        r0 = T0 == -INFINITY ? 0.f : exp2f(T0 - m0);
                        r1 = T1 == -INFINITY ? 0.f : exp2f(T1 - m1);
                        T0 = m0;
                        T1 = m1;
                    }
#pragma unroll
                    for (int x = 0; x < kMt; ++x) {
                        o[x][0] *= r0;
                        o[x][1] *= r1;
                        o[x][2] *= r0;
                        o[x][3] *= r1;
                    }
                }
                const float ref0 = safe_ref(M0), ref1 = safe_ref(M1);
                float p0 = exp2f(x0 - ref0), p1 = exp2f(x1 - ref1), p2 = exp2f(x2 - ref0), p3 = exp2f(x3 - ref1);
                l0 += p0 + p2;
                l1 += p1 + p3;
                if constexpr (E4M3) {
                    const float y0 = safe_ref(T0), y1 = safe_ref(T1);
                    p0 = exp2f(x0 + v0 - y0);
                    p1 = exp2f(x1 + v0 - y1);
                    p2 = exp2f(x2 + v1 - y0);
                    p3 = exp2f(x3 + v1 - y1);
                }
                const uint32_t b0 = transpose8(pack2<E4M3>(p0, p1)), b1 = transpose8(pack2<E4M3>(p2, p3));
#pragma unroll
                for (int w = 0; w < kVw; ++w) {
                    if constexpr (E4M3) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t lo = __byte_perm(vx[0][w], vx[1][w], y ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(vx[2][w], vx[3][w], y ? 0x7362 : 0x5140);
                            mma16816<true>(o[2 * w + y], h2_from_e4m3(lo & 0xffffu), h2_from_e4m3(lo >> 16),
                                           h2_from_e4m3(hi & 0xffffu), h2_from_e4m3(hi >> 16), b0, b1);
                        }
                    } else {
                        mma16816<false>(o[w], __byte_perm(vx[0][w], vx[1][w], 0x5410),
                                        __byte_perm(vx[0][w], vx[1][w], 0x7632), __byte_perm(vx[2][w], vx[3][w], 0x5410),
                                        __byte_perm(vx[2][w], vx[3][w], 0x7632), b0, b1);
                    }
                }
            } else {
                load_k(row_next);
            }
            load_v(row_next, n_next);
            row = row_next;
        }
        // ---- join the warps
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
            l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
        }
        __syncthreads();  // the previous sequence's sums have been read
        if (g == 0) {
            refs[warp][2 * t][0] = M0;
            refs[warp][2 * t][1] = l0;
            refs[warp][2 * t][2] = T0;
            refs[warp][2 * t + 1][0] = M1;
            refs[warp][2 * t + 1][1] = l1;
            refs[warp][2 * t + 1][2] = T1;
        }
#pragma unroll
        for (int x = 0; x < kMt; ++x) {
            // even and odd element of tile x for this lane's g
            int d0;
            if constexpr (E4M3) d0 = g * (D / 8) + 2 * x;
            else d0 = ((x >> 2) * 8 + g) * 8 + 2 * (x & 3);
            *reinterpret_cast<float2*>(&osum[warp][2 * t][d0]) = make_float2(o[x][0], o[x][2]);
            *reinterpret_cast<float2*>(&osum[warp][2 * t + 1][d0]) = make_float2(o[x][1], o[x][3]);
        }
        __syncthreads();
        const bool whole = u == useq && e == useq + su;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (u == u0 ? 0 : 1);
        for (int h = warp; h < ng; h += kWarps) {
            float m = -INFINITY, tt = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                m = fmaxf(m, refs[w][h][0]);
                tt = fmaxf(tt, refs[w][h][2]);
            }
            float l = 0.f, acc[D / 32];
#pragma unroll
            for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (refs[w][h][1] == 0.f) continue;  // no keys
                l = fmaf(refs[w][h][1], exp2f(refs[w][h][0] - m), l);
                const float f = exp2f(refs[w][h][2] - tt);
                float y[D / 32];
                load_vec<D / 32>(&osum[w][h][lane * (D / 32)], y);
#pragma unroll
                for (int x = 0; x < D / 32; ++x) acc[x] = fmaf(f, y[x], acc[x]);
            }
            const int64_t hq = kv * A.G + g0 + h;
            if (whole) {
                // exp2f(tt - m): a value row's exponent at most, within +-127
                const float f = l > 0.f ? exp2f(tt - m) / l : (l == 0.f ? 0.f : l);
                __nv_bfloat16* dst = out + ((int64_t)s * A.Hq + hq) * D + lane * (D / 32);
#pragma unroll
                for (int x = 0; x < D / 32; x += 2)
                    *reinterpret_cast<__nv_bfloat162*>(dst + x) = __floats2bfloat162_rn(acc[x] * f, acc[x + 1] * f);
            } else {
                float* dst = part.o + (slot * A.Hq + hq) * D + lane * (D / 32);
#pragma unroll
                for (int x = 0; x < D / 32; x += 2) *reinterpret_cast<float2*>(dst + x) = make_float2(acc[x], acc[x + 1]);
                if (lane == 0)
                    *reinterpret_cast<float4*>(part.st + (slot * A.Hq + hq) * 4) = make_float4(m, l, tt, 0.f);
            }
        }
        u = e;
        useq += su;
        ++s;
    }
}

// ---- join -------------------------------------------------------------------

// Sequences cut over several blocks: their slots added in order (fixed, so
// results do not depend on timing); sequences without keys: zeros.
template <typename T>
__global__ void __launch_bounds__(128)
decode_join_kernel(AttnDims A, DecodeLine L, int n_blocks, DecodePart part, T* __restrict__ out) {
    const int s = blockIdx.x;
    int64_t first;
    const int64_t U = line_units(L, s, &first), n = L.units(s);
    pdl_wait();
    for (int h = blockIdx.y * 4 + (threadIdx.x >> 5); h < A.Hq; h += gridDim.y * 4) {
        const int lane = threadIdx.x & 31;
        T* dst = out + ((int64_t)s * A.Hq + h) * A.d;
        if (n == 0) {
            for (int x = lane; x < A.d; x += 32) dst[x] = from_f32<T>(0.f);
            continue;
        }
        const int64_t nb = min((int64_t)n_blocks, U);
        const int64_t c0 = ((first + 1) * nb - 1) / U, c1 = ((first + n) * nb - 1) / U;
        if (c0 == c1) continue;  // finished by its block
        auto slot = [&](int64_t c) { return 2 * c + (c * U / nb < first ? 1 : 0); };
        float m = -INFINITY;
        for (int64_t c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, part.st[(slot(c) * A.Hq + h) * 4]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
        const int per = A.d / 32;
        for (int64_t c = c0; c <= c1; ++c) {
            const int64_t i = slot(c) * A.Hq + h;
            const float4 st = *reinterpret_cast<const float4*>(part.st + i * 4);
            if (st.y == 0.f) continue;  // no keys
            l = fmaf(exp2f(st.x - m), st.y, l);
            const float w = exp2f(st.z - m);
            const float* o = part.o + i * A.d + lane * per;
            for (int x = 0; x < per; ++x) acc[x] = fmaf(w, o[x], acc[x]);
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        for (int x = 0; x < per; ++x) dst[lane * per + x] = from_f32<T>(acc[x] * inv);
    }
}

// Thread blocks per kv head and head group: enough to fill the SMs with the
// resident blocks of the kernel, whatever the lengths turn out to be.
int blocks_per_head(int n_sm, int resident, int Hkv, int groups) {
    return std::max(1, n_sm * resident / (Hkv * groups));
}
constexpr int kMaxResident = 8, kMaxSm = 160;

}  // namespace

// Slots for the most blocks any kernel here runs.
size_t attention_decode_ws_bytes(int Hq, int Hkv, int d) {
    const size_t groups = (size_t)(Hq / Hkv + kGroup - 1) / kGroup;
    const size_t blocks = std::max<size_t>(1, (size_t)kMaxSm * kMaxResident / ((size_t)Hkv * groups));
    return 2 * blocks * (size_t)Hq * (size_t)(d + 4) * sizeof(float);
}

template <typename T>
cudaError_t launch_attention_decode(const AttnDims& A, const CacheDims& C, bool e4m3, const hla_cache& c, const T* q,
                                    const int64_t* lens, T* out, float* ws, cudaStream_t st) {
    static DeviceCache cache;
    int n_sm = 0;
    cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
    if (e != cudaSuccess) return e;
    n_sm = std::min(n_sm, kMaxSm);
    const int groups = (A.G + kGroup - 1) / kGroup;
    const DecodeLine L = {lens, A.n_seqs, (int64_t)C.max_pages * C.page};
    int n = 0;
    DecodePart part = {};
    auto run = [&](auto kernel, DeviceCache& occupancy) {
        int resident = 0;
        cudaError_t r = device_cached(occupancy, &resident, [&](int, int* v) {
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kernel, kThreads, 0);
        });
        if (r != cudaSuccess) return r;
        n = blocks_per_head(n_sm, std::max(1, std::min(resident, kMaxResident)), A.Hkv, groups);
        part = {ws, ws + 2 * (size_t)n * A.Hq * A.d};
        kernel<<<dim3((unsigned)n, (unsigned)A.Hkv, (unsigned)groups), kThreads, 0, st>>>(A, C, c, q, L, out, part);
        return cudaGetLastError();
    };
    static DeviceCache occ[4];
    if constexpr (sizeof(T) == 4) {
        if (A.d == 128)
            e = e4m3 ? run(decode_f32_kernel<true, 128>, occ[0]) : run(decode_f32_kernel<false, 128>, occ[1]);
        else
            e = e4m3 ? run(decode_f32_kernel<true, 64>, occ[2]) : run(decode_f32_kernel<false, 64>, occ[3]);
    } else {
        if (A.d == 128)
            e = e4m3 ? run(decode_mma_kernel<true, 128>, occ[0]) : run(decode_mma_kernel<false, 128>, occ[1]);
        else
            e = e4m3 ? run(decode_mma_kernel<true, 64>, occ[2]) : run(decode_mma_kernel<false, 64>, occ[3]);
    }
    if (e != cudaSuccess) return e;
    LaunchCfg lc(dim3((unsigned)A.n_seqs, (unsigned)std::min(65535, (A.Hq + 3) / 4)), dim3(128), 0, st, true);
    return cudaLaunchKernelEx(&lc.cfg, decode_join_kernel<T>, A, L, n, part, out);
}
template cudaError_t launch_attention_decode<float>(const AttnDims&, const CacheDims&, bool, const hla_cache&,
                                                    const float*, const int64_t*, float*, float*, cudaStream_t);
template cudaError_t launch_attention_decode<__nv_bfloat16>(const AttnDims&, const CacheDims&, bool, const hla_cache&,
                                                            const __nv_bfloat16*, const int64_t*, __nv_bfloat16*,
                                                            float*, cudaStream_t);

}  // namespace hla
