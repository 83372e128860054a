// Decode step of a full softmax layer: one query token per sequence over the
// paged cache.  See attention_decode.cuh for the cut over blocks.
//
// bf16 layers are bound by the cache's bytes.  32/8 heads of 128: 64 sequences of 8192 tokens of 8-bit rows in 182 us
// (5.9 TB/s; heads of 64 122 us, 4.5), of bf16 rows in 305 us (7.0); one sequence of 131072 in 55 us (8-bit) and 86 us
// (bf16).  8-bit rows take two conversions per four values on the way to the products, which is what keeps them behind
// bf16's rate.  The join takes 7 to 8 us of these.  fp32 layers wait at four barriers per 64 keys with nothing on its way
// across them: 8 x 8192 tokens of fp32 rows 132 us (4.1 TB/s), of 8-bit rows, whose conversions come on top, 209 us (0.65).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "attention_decode.cuh"

namespace hla {

namespace {

constexpr int kThreads = 128;
constexpr int kGroup = 8;  // query heads of a kv head per block
constexpr int kDecodeUnit = 64;  // keys the fp32 kernel takes at a time

// ---- fp32 layers ------------------------------------------------------------
//
// Scores: eight lanes per key, D / 8 values each, partial dot products joined
// by three shuffles.  Values: a thread per column pair, the weights read from
// shared memory.  All in fp32.
template <int E> __device__ __forceinline__ void load_e4m3(const uint8_t* p, float* f) {
    uint32_t w[E < 4 ? 1 : E / 4];
    if constexpr (E == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
    else if constexpr (E == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (E == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int x = 0; x < E; x += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[x / 4] >> (8 * (x & 2))), __NV_E4M3);
        const float2 g = __half22float2(__half2(h));
        f[x] = g.x;
        f[x + 1] = g.y;
    }
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(kThreads)
decode_f32_kernel(AttnDims A, CacheDims C, hla_cache c, const float* __restrict__ q, DecodeLine L,
                  float* __restrict__ out, DecodePart part) {
    constexpr int E = D / 8;  // elements of a key per lane
    __shared__ alignas(16) float qs[kGroup][D];
    __shared__ alignas(16) float ps[kGroup][kDecodeUnit];  // scores, then weights
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
        float mrun = -INFINITY, lrun = 0.f;  // of head tid / 16
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
            {  // four keys per lane group, all on their way at once
                constexpr int kN = kDecodeUnit / (kThreads / 8);
                float kx[kN][E];
#pragma unroll
                for (int y = 0; y < kN; ++y) {
                    const int64_t r = rows[tid / 8 + y * (kThreads / 8)];
                    if (r < 0) {
#pragma unroll
                        for (int x = 0; x < E; ++x) kx[y][x] = 0.f;
                    } else if constexpr (E4M3) {
                        const float ks = exp2f((float)((int)c.k_exp[r] - 127));
                        load_e4m3<E>(static_cast<const uint8_t*>(c.k) + r * D + (tid & 7) * E, kx[y]);
#pragma unroll
                        for (int x = 0; x < E; ++x) kx[y][x] *= ks;
                    } else {
                        const float* src = static_cast<const float*>(c.k) + r * D + (tid & 7) * 4;
#pragma unroll
                        for (int x = 0; x < E; x += 4) load_vec<4>(src + x * 8, kx[y] + x);
                    }
                }
                for (int g = 0; g < ng; ++g) {
                    float d[kN];
#pragma unroll
                    for (int y = 0; y < kN; ++y) d[y] = 0.f;
#pragma unroll
                    for (int x = 0; x < E; x += 4) {
                        // the lane's elements: E in a row (8-bit rows), else four of every 32
                        const float4 qv = *reinterpret_cast<const float4*>(&qs[g][E4M3 ? (tid & 7) * E + x : (tid & 7) * 4 + x * 8]);
#pragma unroll
                        for (int y = 0; y < kN; ++y) {
                            d[y] = fmaf(qv.x, kx[y][x], d[y]);
                            d[y] = fmaf(qv.y, kx[y][x + 1], d[y]);
                            d[y] = fmaf(qv.z, kx[y][x + 2], d[y]);
                            d[y] = fmaf(qv.w, kx[y][x + 3], d[y]);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < kN; ++y) {
#pragma unroll
                        for (int o = 4; o; o >>= 1) d[y] += __shfl_xor_sync(0xffffffffu, d[y], o);
                        const int j = tid / 8 + y * (kThreads / 8);
                        if ((tid & 7) == 0) ps[g][j] = rows[j] >= 0 ? d[y] : -INFINITY;
                    }
                }
            }
            __syncthreads();
            {  // 16 lanes per head, four keys each
                const int g = tid >> 4, j = (tid & 15) * 4;
                const float4 x = *reinterpret_cast<const float4*>(&ps[g][j]);
                float v[4] = {x.x, x.y, x.z, x.w}, top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if (j + y >= n || g >= ng) v[y] = -INFINITY;
                    top = fmaxf(top, v[y]);
                }
#pragma unroll
                for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float m = fmaxf(mrun, top), corr = mrun == -INFINITY ? 0.f : exp2f(mrun - m);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    v[y] = v[y] == -INFINITY ? 0.f : exp2f(v[y] - m);
                    sum += v[y];
                }
#pragma unroll
                for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                *reinterpret_cast<float4*>(&ps[g][j]) = make_float4(v[0], v[1], v[2], v[3]);
                lrun = lrun * corr + sum;
                mrun = m;
                if ((tid & 15) == 0) stats[g][1] = corr;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kGroup; ++g)
                if (g < ng)
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) acc[g][x] *= stats[g][1];
            // values: a warp takes every fourth key, eight on their way at once
            constexpr int kE = D / 32, kN = 8;
            for (int j0 = warp; j0 < n; j0 += kN * (kThreads / 32)) {
                float vx[kN][kE];
#pragma unroll
                for (int y = 0; y < kN; ++y) {
                    const int j = j0 + y * (kThreads / 32);
                    const int64_t r = j < n ? rows[j] : -1;
#pragma unroll
                    for (int x = 0; x < kE; ++x) vx[y][x] = 0.f;
                    if (r < 0) continue;
                    if constexpr (E4M3) load_e4m3<kE>(static_cast<const uint8_t*>(c.v) + r * D + lane * kE, vx[y]);
                    else load_vec<kE>(static_cast<const float*>(c.v) + r * D + lane * kE, vx[y]);
                }
#pragma unroll
                for (int y = 0; y < kN; ++y) {
                    const int j = min(j0 + y * (kThreads / 32), kDecodeUnit - 1);
                    const float scale = vs[j];
#pragma unroll
                    for (int x = 0; x < kE; ++x) vx[y][x] *= scale;
#pragma unroll
                    for (int g = 0; g < kGroup; ++g)
                        if (g < ng) {
                            const float p = j0 + y * (kThreads / 32) < n ? ps[g][j] : 0.f;
#pragma unroll
                            for (int x = 0; x < kE; ++x) acc[g][x] = fmaf(p, vx[y][x], acc[g][x]);
                        }
                }
            }
        }
        // join the warps; the block's part of the sequence
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
            if (g < ng)
#pragma unroll
                for (int x = 0; x < D / 32; ++x) osum[warp][g][lane * (D / 32) + x] = acc[g][x];
        __syncthreads();  // the last corrections have been read
        if ((tid & 15) == 0) {
            stats[tid >> 4][0] = mrun;
            stats[tid >> 4][1] = lrun;
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
            t[0] = stats[tid][0];
            t[1] = stats[tid][1];
            t[2] = stats[tid][0];
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
// value row's into the exponent of its weight, 2^x with x = s + ev - Mt and a
// reference Mt of their own.  Weights are fp16 too: 11 bits of them from
// 2^(kTop + 1) down to 2^-14 (x = -kBand), steps of 2^-24 below.  A weight's error there, 2^-39 of
// Mt's, is 2^-31 of the sum of weights at most while the value rows' exponents are
// within kLike of each other.  But a key whose value row is large in one column sets Mt
// for all of them, and the weights that this leaves too few bits may be all that the
// other columns have: a warp whose rows differ by more goes over them again, kBand powers
// of two of weights at a time (64 x 8192 tokens 182 -> 348 us, part of it read from L2).
// (Always exact, by values and two-part weights in bf16, to which no instruction
// converts: 64 x 8192 tokens, timed one by one, 186 -> 273 us, where this takes 191; light weights looked for
// one by one: 223, for want of registers.)  bf16 caches: products in bf16,
// weights in two bf16 parts (with one, outputs of a few heads were off by up to
// 1.5 times the rounding of the result; the second costs nothing beside the loads).
//
// A warp takes 32 keys at a time (16 of 256 bytes), so that the 12 to 16 warps
// of an SM keep some 60 KB on their way.
//
// References are raised only when a score exceeds them by 2^8 (8-bit rows: 2), by a
// vote per tile, no reduction.

constexpr float kLazy = 8.0f, kLazyT = 1.0f;
constexpr float kTop = 14.0f, kBand = 28.0f, kLeast = -126.0f;  // weights of 2^kLeast of the reference and less are 0
constexpr uint32_t kLike = 8;
constexpr uint32_t kNoRow = 0xffffffffu;

// Tiles of 16 keys per page, and division by it: i / tiles = i mul >> shift for i < 2^31 (mul = ceil(2^shift /
// tiles), shift = 31 + ceil(log2 tiles); the excess of mul adds less than 1 / tiles to the quotient).
struct PageDiv {
    uint32_t tiles, mul, shift;
    explicit PageDiv(int page) : tiles((uint32_t)page / 16), shift(31) {
        while ((1ull << (shift - 31)) < tiles) ++shift;
        mul = (uint32_t)(((1ull << shift) + tiles - 1) / tiles);
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t i) const { return (uint32_t)(((uint64_t)i * mul) >> shift); }
};
__device__ __forceinline__ float ex2(float x) {  // 2 ulp; below 2^-126: 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four e4m3 values to fp16: the first two, the last two.
__device__ __forceinline__ void h2_from_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
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
// A weight >= 0 in two bf16 parts: its upper half (of a pair), and what that leaves; not 0, so that an infinite value
// times either is that infinity.
__device__ __forceinline__ uint32_t top2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float p) {
    const float r = fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xffff0000u), 1.17549435e-38f);
    return p == 0.f ? 0.f : r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float safe_ref(float m) { return m == -INFINITY ? 0.f : m; }

template <bool E4M3, int D>
__global__ void __launch_bounds__(kThreads, D == 64 && E4M3 ? 4 : 3)
decode_mma_kernel(AttnDims A, CacheDims C, PageDiv pd, hla_cache c, const __nv_bfloat16* __restrict__ q, DecodeLine L,
                  __nv_bfloat16* __restrict__ out, DecodePart part) {
    constexpr int kRow = D * (E4M3 ? 1 : 2);      // bytes of a cache row
    constexpr int kKp = kRow / 64;                // 16-byte pieces of a key row per lane
    constexpr int kVw = kRow / 32;                // 32-bit words of a value row per lane
    constexpr int kSteps = D / 16, kMt = D / 16;  // k steps of the scores; d tiles of the output
    constexpr int kWarps = kThreads / 32;
    constexpr int kSub = kRow == 256 ? 1 : 2, kUnit = 16 * kSub * kWarps;  // sub-tiles of 16 keys per warp; keys of a unit
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
    while (u < u1) {
        const int64_t len = L.len(s), su = (len + kUnit - 1) / kUnit;
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
        float o[kMt][4], M0, M1, T0, T1, l0, l1;
        uint32_t spread = 0u;  // of the value rows' exponents (bytes): the largest, and 256 less the smallest but 0

        // tiles of 16 keys: the page a tile lies in (-1: past the last key), its cache row (kNoRow: no such page)
        const uint32_t n_tiles = (uint32_t)((len + 15) / 16);
        const int32_t* pages = c.page_table + (int64_t)s * C.max_pages;
        auto page_of = [&](uint32_t i, uint32_t* at) -> int {
            const uint32_t p = pd.quotient(i);
            *at = (i - p * pd.tiles) * 16;
            return i < n_tiles ? __ldg(pages + p) : -1;
        };
        auto row_of = [&](uint32_t i, int page, uint32_t at) -> uint32_t {
            if (i >= n_tiles) return kNoRow;
            if ((uint32_t)page >= (uint32_t)C.n_pages) {
                if (lane == 0) atomicExch(c.err, kErrState);
                return kNoRow;
            }
            return ((uint32_t)page * C.Hkv + kv) * C.page + at;
        };
        uint4 kx[kSub][2][kKp];
        uint32_t vx[kSub][4][kVw];
        // exponent bytes of both tiles: of tile lane / 16, keys' (bit 3 of the lane 0) or values', keys 2 (lane % 8) and the next
        uint32_t ex = 0u;
        const uint8_t* ex_base = (lane & 8 ? c.v_exp : c.k_exp) + 2 * (lane & 7);
        auto load_ex = [&](const uint32_t (&r)[kSub]) {
            const uint32_t mine = lane < 16 ? r[0] : r[kSub - 1];
            return mine == kNoRow ? 0u : (uint32_t)*reinterpret_cast<const uint16_t*>(ex_base + mine);
        };
        auto ex_of = [&](int y, int kind, int key) {  // keys g and g + 8: key 0 and 8
            return __byte_perm(__shfl_sync(0xffffffffu, ex, y * 16 + kind * 8 + (g + key) / 2), 0u, 0x4440 + (g & 1));
        };
        auto load_k = [&](int y, uint32_t row) {
            if (row == kNoRow) return;
            const char* p = static_cast<const char*>(c.k) + (size_t)(row + g) * kRow + t * 16;
#pragma unroll
            for (int i = 0; i < kKp; ++i) {
                kx[y][0][i] = __ldcs(reinterpret_cast<const uint4*>(p + i * 64));
                kx[y][1][i] = __ldcs(reinterpret_cast<const uint4*>(p + 8 * kRow + i * 64));
            }
        };
        auto load_v = [&](int y, uint32_t row, int n) {  // n: keys of the tile; the rows behind them are zeros
            if (row == kNoRow) return;
            const char* p0 = static_cast<const char*>(c.v) + (size_t)(row + 2 * t) * kRow;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 2 * t + (x & 1) + 8 * (x >> 1);
                const char* p = p0 + ((x & 1) + 8 * (x >> 1)) * kRow;
                if constexpr (kVw == 2) {  // 64 one-byte values: 8 bytes per lane
                    uint2 w = make_uint2(0u, 0u);
                    if (key < n) w = __ldcs(reinterpret_cast<const uint2*>(p + g * 8));
                    vx[y][x][0] = w.x;
                    vx[y][x][1] = w.y;
                } else {
#pragma unroll
                    for (int i = 0; i < kVw / 4; ++i) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (key < n) w = __ldcs(reinterpret_cast<const uint4*>(p + i * 128 + g * 16));
                        vx[y][x][4 * i] = w.x;
                        vx[y][x][4 * i + 1] = w.y;
                        vx[y][x][4 * i + 2] = w.z;
                        vx[y][x][4 * i + 3] = w.w;
                    }
                }
            }
        };
        // tiles of this warp: kSub in a row from (4 unit + warp) kSub
        constexpr uint32_t kStep = kWarps * kSub;
        const uint32_t iend = min((uint32_t)(e - useq) * kStep, n_tiles);
        auto keys_of = [&](uint32_t j) { return (int)min((int64_t)16, len - (int64_t)j * 16); };
        // One pass over them.  BANDS: of the weights with x in (-kBand, 0] - up only (all above, with up = 0); whether there
        // are lighter ones.
        auto walk = [&](auto bands, float up) {
            constexpr bool BANDS = decltype(bands)::value;
            bool lighter = false;
#pragma unroll
            for (int x = 0; x < kMt; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
            M0 = M1 = T0 = T1 = -INFINITY;
            l0 = l1 = 0.f;
            uint32_t i = (uint32_t)((u - useq) * kWarps + warp) * kSub;
            uint32_t row[kSub], at_next[kSub];
            int page_next[kSub];
#pragma unroll
            for (int y = 0; y < kSub; ++y) {
                uint32_t at;
                const int page = page_of(i + y, &at);
                row[y] = row_of(i + y, page, at);
                page_next[y] = page_of(i + kStep + y, &at_next[y]);
                load_k(y, row[y]);
                load_v(y, row[y], keys_of(i + y));
            }
            if constexpr (E4M3) ex = load_ex(row);
            for (; i < iend; i += kStep) {
                const bool more = i + kStep < iend;
                uint32_t row_next[kSub];
#pragma unroll
                for (int y = 0; y < kSub; ++y) {
                    row_next[y] = more ? row_of(i + kStep + y, page_next[y], at_next[y]) : kNoRow;
                    if (more) page_next[y] = page_of(i + 2 * kStep + y, &at_next[y]);
                }
                uint32_t ex_next = 0u;
                if constexpr (E4M3) {
                    ex_next = load_ex(row_next);
                    // (bytes of rows behind the last key count as 0)
                    const int n = min(2, keys_of(i + (lane >> 4)) - 2 * (lane & 7));
                    const uint32_t a = lane & 8 && n > 0 ? ex & 0xffu : 0u, b = lane & 8 && n > 1 ? ex >> 8 : 0u;
                    spread = max_u16x2(spread, max(a, b) | max(256u - a & 0xffu, 256u - b & 0xffu) << 16);
                }
                // ---- scores of every sub-tile (base-2 logs), and the exponents of its value rows
                float sc[kSub][4], ve[kSub][2];
                float h0 = -INFINITY, h1 = -INFINITY, t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int y = 0; y < kSub; ++y) {
                    float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
                    const int n = row[y] != kNoRow ? keys_of(i + y) : 0;
#pragma unroll
                    for (int x = 0; x < kKp; ++x) {
                        const uint32_t a[4] = {kx[y][0][x].x, kx[y][0][x].y, kx[y][0][x].z, kx[y][0][x].w};
                        const uint32_t b[4] = {kx[y][1][x].x, kx[y][1][x].y, kx[y][1][x].z, kx[y][1][x].w};
                        if constexpr (E4M3) {
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                uint32_t al, ah, bl, bh;
                                h2_from_e4m3(a[w], al, ah);
                                h2_from_e4m3(b[w], bl, bh);
                                mma16816<true>(w & 1 ? a1 : a0, al, bl, ah, bh, qf[x * 4 + w][0], qf[x * 4 + w][1]);
                            }
                        } else {
#pragma unroll
                            for (int w = 0; w < 2; ++w)
                                mma16816<false>(w & 1 ? a1 : a0, a[2 * w], b[2 * w], a[2 * w + 1], b[2 * w + 1],
                                                qf[x * 2 + w][0], qf[x * 2 + w][1]);
                        }
                    }
                    float f0 = 1.f, f1 = 1.f;  // the key rows' powers of two
                    ve[y][0] = ve[y][1] = 0.f;
                    if constexpr (E4M3) {
                        const uint32_t e0 = ex_of(y, 0, 0), e1 = ex_of(y, 0, 8);
                        f0 = e0 ? __uint_as_float(e0 << 23) : __uint_as_float(0x400000u);
                        f1 = e1 ? __uint_as_float(e1 << 23) : __uint_as_float(0x400000u);
                        ve[y][0] = (float)((int)ex_of(y, 1, 0) - 127);
                        ve[y][1] = (float)((int)ex_of(y, 1, 8) - 127);
                    }
                    load_k(y, row_next[y]);
                    // (the factors' product first: a sum of 8-bit products times either may leave the range that the score does not)
                    const bool on0 = g < n, on1 = g + 8 < n;
                    sc[y][0] = on0 ? (a0[0] + a1[0]) * (f0 * qs0) : -INFINITY;
                    sc[y][1] = on0 ? (a0[1] + a1[1]) * (f0 * qs1) : -INFINITY;
                    sc[y][2] = on1 ? (a0[2] + a1[2]) * (f1 * qs0) : -INFINITY;
                    sc[y][3] = on1 ? (a0[3] + a1[3]) * (f1 * qs1) : -INFINITY;
                    h0 = fmaxf(h0, fmaxf(sc[y][0], sc[y][2]));
                    h1 = fmaxf(h1, fmaxf(sc[y][1], sc[y][3]));
                    if constexpr (E4M3) {
                        t0 = fmaxf(t0, fmaxf(sc[y][0] + ve[y][0], sc[y][2] + ve[y][1]));
                        t1 = fmaxf(t1, fmaxf(sc[y][1] + ve[y][0], sc[y][3] + ve[y][1]));
                    }
                }
                bool grow = h0 > M0 + kLazy || h1 > M1 + kLazy;
                if constexpr (E4M3) grow |= t0 > T0 + kLazyT || t1 > T1 + kLazyT;
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
                    const float n0 = E4M3 ? fmaxf(T0, t0) : m0, n1 = E4M3 ? fmaxf(T1, t1) : m1;
                    l0 *= M0 == -INFINITY ? 0.f : exp2f(M0 - m0);
                    l1 *= M1 == -INFINITY ? 0.f : exp2f(M1 - m1);
                    const float r0 = T0 == -INFINITY ? 0.f : exp2f(T0 - n0), r1 = T1 == -INFINITY ? 0.f : exp2f(T1 - n1);
                    M0 = m0;
                    M1 = m1;
                    T0 = n0;
                    T1 = n1;
#pragma unroll
                    for (int x = 0; x < kMt; ++x) {
                        o[x][0] *= r0;
                        o[x][1] *= r1;
                        o[x][2] *= r0;
                        o[x][3] *= r1;
                    }
                }
                // ---- weights, and the values they go to
                const float ref0 = safe_ref(M0), ref1 = safe_ref(M1), ret0 = safe_ref(T0) - kTop, ret1 = safe_ref(T1) - kTop;
#pragma unroll
                for (int y = 0; y < kSub; ++y) {
                    float p0 = ex2(sc[y][0] - ref0), p1 = ex2(sc[y][1] - ref1);
                    float p2 = ex2(sc[y][2] - ref0), p3 = ex2(sc[y][3] - ref1);
                    l0 += p0 + p2;
                    l1 += p1 + p3;
                    if constexpr (E4M3) {
                        auto weight = [&](float s, float p, float ev, float top) {
                            const float z = s + (ev - top) + up;
                            if constexpr (!BANDS) return ex2(z);
                            lighter |= z <= kTop - kBand && z - up > kTop + kLeast && p > 0.f;
                            return z <= kTop - kBand || (z > kTop && up > 0.f) ? 0.f : ex2(z);
                        };
                        p0 = weight(sc[y][0], p0, ve[y][0], ret0);
                        p1 = weight(sc[y][1], p1, ve[y][0], ret1);
                        p2 = weight(sc[y][2], p2, ve[y][1], ret0);
                        p3 = weight(sc[y][3], p3, ve[y][1], ret1);
                    }
                    uint32_t b0, b1, c0 = 0u, c1 = 0u;  // bf16 weights in two parts
                    if constexpr (E4M3) {
                        b0 = transpose8(pack2<true>(p0, p1));
                        b1 = transpose8(pack2<true>(p2, p3));
                    } else {
                        b0 = transpose8(top2(p0, p1));
                        b1 = transpose8(top2(p2, p3));
                        c0 = transpose8(pack2<false>(rest(p0), rest(p1)));
                        c1 = transpose8(pack2<false>(rest(p2), rest(p3)));
                    }
                    if (row[y] != kNoRow) {
#pragma unroll
                        for (int w = 0; w < kVw; ++w) {
                            if constexpr (E4M3) {
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    const uint32_t sel = z ? 0x7362 : 0x5140;
                                    uint32_t a0, a1, a2, a3;
                                    h2_from_e4m3(__byte_perm(vx[y][0][w], vx[y][1][w], sel), a0, a1);
                                    h2_from_e4m3(__byte_perm(vx[y][2][w], vx[y][3][w], sel), a2, a3);
                                    mma16816<true>(o[2 * w + z], a0, a1, a2, a3, b0, b1);
                                }
                            } else {
                                const uint32_t a0 = __byte_perm(vx[y][0][w], vx[y][1][w], 0x5410);
                                const uint32_t a1 = __byte_perm(vx[y][0][w], vx[y][1][w], 0x7632);
                                const uint32_t a2 = __byte_perm(vx[y][2][w], vx[y][3][w], 0x5410);
                                const uint32_t a3 = __byte_perm(vx[y][2][w], vx[y][3][w], 0x7632);
                                mma16816<false>(o[w], a0, a1, a2, a3, c0, c1);
                                mma16816<false>(o[w], a0, a1, a2, a3, b0, b1);
                            }
                        }
                    }
                    load_v(y, row_next[y], keys_of(i + kStep + y));
                    row[y] = row_next[y];
                }
                ex = ex_next;
            }
            return lighter;
        };
        walk(std::false_type{}, 0.f);
        if constexpr (E4M3) {
            if (__reduce_max_sync(0xffffffffu, spread & 0xffffu) + __reduce_max_sync(0xffffffffu, spread >> 16) > 256u + kLike) {
                volatile float kept[kMt * 4];  // in local memory
                for (int x = 0; x < kMt * 4; ++x) kept[x] = 0.f;
                float down = 1.f;
                bool more = true;
                for (float up = 0.f; more; up += kBand, down *= 0x1p-28f) {
                    more = __any_sync(0xffffffffu, walk(std::true_type{}, up));
#pragma unroll
                    for (int x = 0; x < kMt * 4; ++x) kept[x] = fmaf(down, o[x / 4][x % 4], kept[x]);
                }
#pragma unroll
                for (int x = 0; x < kMt * 4; ++x) o[x / 4][x % 4] = kept[x];
            }
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
            constexpr float f = E4M3 ? 0x1p-14f : 1.f;  // 2^-kTop
            *reinterpret_cast<float2*>(&osum[warp][2 * t][d0]) = make_float2(o[x][0] * f, o[x][2] * f);
            *reinterpret_cast<float2*>(&osum[warp][2 * t + 1][d0]) = make_float2(o[x][1] * f, o[x][3] * f);
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

// Sequences cut over several blocks: W warps per sequence and query head take
// the slots in turn, four in flight each, then are joined in order (fixed, so results do not depend on timing).  Sequences without
// keys: zeros.
constexpr int kJoinWarps = 8;
template <typename T, int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32)
decode_join_kernel(AttnDims A, DecodeLine L, int n_blocks, DecodePart part, T* __restrict__ out) {
    constexpr int E = D / 32;
    __shared__ float osum[W][D], lsum[W];
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
    const int h = W == 1 ? blockIdx.y * kJoinWarps + (threadIdx.x >> 5) : blockIdx.y;
    if (h >= A.Hq) return;
    int64_t first;
    const int64_t U = line_units(L, s, &first), n = L.units(s);
    pdl_wait();
    T* dst = out + ((int64_t)s * A.Hq + h) * D;
    if (n == 0) {
        for (int x = warp * 32 + lane; x < D; x += W * 32) dst[x] = from_f32<T>(0.f);
        return;
    }
    const int64_t nb = min((int64_t)n_blocks, U);
    const int c0 = (int)(((first + 1) * nb - 1) / U), c1 = (int)(((first + n) * nb - 1) / U);
    if (c0 == c1) return;  // finished by its block
    // slot of block c: 2 c, or 2 c + 1 for the one that reached the sequence from another
    const int late = c0 * U / nb < first ? 1 : 0;
    auto at = [&](int c) { return (int64_t)(2 * c + (c == c0 ? late : 0)) * A.Hq + h; };
    float m = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, __ldg(part.st + at(c) * 4));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[E], l = 0.f;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = 0.f;
    for (int c = c0 + warp; c <= c1; c += 4 * W) {
        float4 st[4];
        float o[4][E];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            st[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + y * W > c1) continue;
            const int64_t i = at(c + y * W);
            st[y] = __ldg(reinterpret_cast<const float4*>(part.st + i * 4));
            load_vec<E>(part.o + i * D + lane * E, o[y]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (st[y].y == 0.f) continue;  // no keys
            l = fmaf(exp2f(st[y].x - m), st[y].y, l);
            const float w = exp2f(st[y].z - m);
#pragma unroll
            for (int x = 0; x < E; ++x) acc[x] = fmaf(w, o[y][x], acc[x]);
        }
    }
    if constexpr (W == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int x = 0; x < E; ++x) dst[lane * E + x] = from_f32<T>(acc[x] * inv);
    } else {
#pragma unroll
        for (int x = 0; x < E; ++x) osum[warp][lane * E + x] = acc[x];
        if (lane == 0) lsum[warp] = l;
        __syncthreads();
        if (threadIdx.x < D) {
            float o = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                o += osum[w][threadIdx.x];
                sum += lsum[w];
            }
            dst[threadIdx.x] = from_f32<T>(sum == 0.f ? 0.f : o / sum);
        }
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
    // keys of a unit: what the kernel's four warps take at a time
    const int unit = sizeof(T) == 4 || (A.d == 128 && !e4m3) ? kDecodeUnit : 2 * kDecodeUnit;
    // a table beyond 2^31 tiles of 16 positions is more than any memory holds: positions past that are cut as well
    const DecodeLine L = {lens, A.n_seqs, std::min((int64_t)C.max_pages * C.page, ((int64_t)INT32_MAX - 4096) * 16), unit};
    const PageDiv pd(C.page);
    int n = 0;
    DecodePart part = {};
    auto run = [&](auto kernel, DeviceCache& occupancy, auto... page) {
        int resident = 0;
        cudaError_t r = device_cached(occupancy, &resident, [&](int, int* v) {
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kernel, kThreads, 0);
        });
        if (r != cudaSuccess) return r;
        n = blocks_per_head(n_sm, std::max(1, std::min(resident, kMaxResident)), A.Hkv, groups);
        part = {ws, ws + 2 * (size_t)n * A.Hq * A.d};
        kernel<<<dim3((unsigned)n, (unsigned)A.Hkv, (unsigned)groups), kThreads, 0, st>>>(A, C, page..., c, q, L,
                                                                                                 out, part);
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
            e = e4m3 ? run(decode_mma_kernel<true, 128>, occ[0], pd) : run(decode_mma_kernel<false, 128>, occ[1], pd);
        else
            e = e4m3 ? run(decode_mma_kernel<true, 64>, occ[2], pd) : run(decode_mma_kernel<false, 64>, occ[3], pd);
    }
    if (e != cudaSuccess) return e;
    // a sequence of average length lies in n / n_seqs + 2 blocks or fewer: with few, a warp adds them; with many, a
    // block does (one sequence of 131072 keys in 57 blocks: join 35 -> 4 us; 64 sequences of 100: 16 -> 12 us in all)
    const bool few = n / A.n_seqs + 2 <= 8;
    LaunchCfg lc(dim3((unsigned)A.n_seqs, few ? (unsigned)((A.Hq + kJoinWarps - 1) / kJoinWarps) : (unsigned)A.Hq),
                 dim3(kJoinWarps * 32), 0, st, true);
    auto join = [&](auto kernel) { return cudaLaunchKernelEx(&lc.cfg, kernel, A, L, n, part, out); };
    if (A.d == 128) return few ? join(decode_join_kernel<T, 128, 1>) : join(decode_join_kernel<T, 128, kJoinWarps>);
    return few ? join(decode_join_kernel<T, 64, 1>) : join(decode_join_kernel<T, 64, kJoinWarps>);
}
template cudaError_t launch_attention_decode<float>(const AttnDims&, const CacheDims&, bool, const hla_cache&,
                                                    const float*, const int64_t*, float*, float*, cudaStream_t);
template cudaError_t launch_attention_decode<__nv_bfloat16>(const AttnDims&, const CacheDims&, bool, const hla_cache&,
                                                            const __nv_bfloat16*, const int64_t*, __nv_bfloat16*,
                                                            float*, cudaStream_t);

}  // namespace hla
