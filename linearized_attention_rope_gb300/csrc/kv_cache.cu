// Paged key / value cache: rows quantised as they are written, and read back.
//
// A row (token, kv head) of d values is kept as 8-bit floats (e4m3) of
// x 2^-e with e the smallest integer that keeps |x| <= 448 2^e.  A power of
// two: the scaling is exact, so the one rounding is the 8-bit float's, the
// decode step can fold 2^e into its scores by an exponent, and one byte holds
// it.  (The relative step of a floating point value does not depend on the
// scale; a full-precision scale would gain at most one bit of range.)
//
// Memory bound: a block takes a few tokens; one thread per token finds its
// sequence and page, then d / 8 lanes hold a row, 8 values each (16-byte loads
// of bf16 rows, 8-byte stores), the largest magnitude by shuffles; every thread
// has four rows in flight.  Per-row searches and 64-bit divisions in place of
// the per-token step took three times as long.
#include <cuda_fp8.h>

#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

template <typename T> struct Row8;  // 8 values of a row
template <> struct Row8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Row8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float* f) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// Where packed token t goes: the cache row of head 0 (head h: h pages' rows of
// one head further, h * page), or -1 (out of range, flagged); listed: whether
// it belongs to a sequence at all.
__device__ __forceinline__ int64_t token_row(const CacheDims& C, const hla_cache& c, const int32_t* __restrict__ cu,
                                             const int64_t* __restrict__ start, int64_t t, bool* listed) {
    const int s = seq_of_token(cu, C.n_seqs, t);
    int64_t a, n;
    seq_range(cu, s, C.total, &a, &n);
    *listed = t >= a && t < a + n;
    if (!*listed) return -1;
    const int64_t p = __ldg(start + s) + (t - a);
    int page = -1;
    if (p >= 0 && p / C.page < C.max_pages) page = __ldg(c.page_table + (int64_t)s * C.max_pages + p / C.page);
    if (page < 0 || page >= C.n_pages) {
        atomicExch(c.err, kErrState);
        return -1;
    }
    return (int64_t)page * C.Hkv * C.page + p % C.page;
}

// Smallest e >= -127 with top <= 448 2^e (top finite, >= 0), from the bits.
__device__ __forceinline__ int row_exponent(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
    return max(e, -127);
}
__device__ __forceinline__ float pow2(int e) {  // -127 <= e <= 127
    return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x400000u);
}

// d / 8 consecutive lanes per row; rows of a token: Hkv of k, then Hkv of v.
constexpr int kMaxTokens = 32;  // tokens of a block
template <typename T, bool E4M3, bool READ, int LPR>
__global__ void __launch_bounds__(kThreads)
cache_kernel(CacheDims C, hla_cache c, T* k, T* v, const int32_t* __restrict__ cu, const int64_t* __restrict__ start,
             int tokens) {
    constexpr int D = LPR * 8, kRows = kThreads / LPR;  // rows the block handles at once
    __shared__ int64_t base[kMaxTokens];                // cache row of head 0 (-1: none)
    __shared__ bool listed[kMaxTokens];
    const int lane8 = (threadIdx.x % LPR) * 8, per = 2 * C.Hkv;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, C.total - t0), rows = nt * per;
    if (blockIdx.x == 0) attn_check_table(cu, C.n_seqs, C.total, c.err);
    if ((int)threadIdx.x < nt) {
        bool in;
        base[threadIdx.x] = token_row(C, c, cu, start, t0 + threadIdx.x, &in);
        listed[threadIdx.x] = in;
    }
    __syncthreads();
    for (int r0 = threadIdx.x / LPR; r0 - (int)(threadIdx.x / LPR) < rows; r0 += kRows * kBatch) {  // whole block together
        Row8<T> x[kBatch];
        int64_t at[kBatch], own[kBatch];  // cache row (-1: none), row of k or v (-1: none)
        uint2 q8[kBatch];
        int eb[kBatch];
        bool isv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRows;
            at[i] = own[i] = -1;
            isv[i] = false;
            if (r >= rows) continue;
            const int t = r / per, hh = r - t * per, h = hh < C.Hkv ? hh : hh - C.Hkv;
            isv[i] = hh >= C.Hkv;
            if (base[t] >= 0) at[i] = base[t] + (int64_t)h * C.page;
            if (listed[t]) own[i] = (t0 + t) * C.Hkv + h;
            if constexpr (!READ) {
                if (at[i] >= 0) x[i].load((isv[i] ? v : k) + own[i] * D + lane8);
            } else if (at[i] >= 0) {
                const void* src = isv[i] ? c.v : c.k;
                if constexpr (E4M3) {
                    q8[i] = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(src) + at[i] * D + lane8));
                    eb[i] = (isv[i] ? c.v_exp : c.k_exp)[at[i]];
                } else {
                    x[i].load(static_cast<const T*>(src) + at[i] * D + lane8);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float f[8];
            if constexpr (!READ) {
                if constexpr (E4M3) {
                    float top = 0.f;
                    if (at[i] >= 0) {
                        x[i].get(f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float m = fabsf(f[j]);
                            top = fmaxf(top, m < INFINITY ? m : 0.f);
                        }
                    }
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (at[i] < 0) continue;
                    const int e = row_exponent(top);
                    const float inv = pow2(-e);
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE,
                                                        __NV_E4M3);
                    uint8_t* dst = static_cast<uint8_t*>(isv[i] ? c.v : c.k) + at[i] * D + lane8;
                    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
                    if (lane8 == 0) (isv[i] ? c.v_exp : c.k_exp)[at[i]] = (uint8_t)(e + 127);
                } else {
                    if (at[i] >= 0) x[i].store(static_cast<T*>(isv[i] ? c.v : c.k) + at[i] * D + lane8);
                }
            } else {
                if (own[i] < 0) continue;
                T* dst = (isv[i] ? v : k) + own[i] * D + lane8;
                if (at[i] < 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = 0.f;
                    x[i].set(f);
                } else if constexpr (E4M3) {
                    const float s = pow2(eb[i] - 127);
                    const uint32_t w[2] = {q8[i].x, q8[i].y};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j & 1))), __NV_E4M3);
                        const float2 g = __half22float2(__half2(h));
                        f[2 * j] = g.x * s;
                        f[2 * j + 1] = g.y * s;
                    }
                    x[i].set(f);
                }
                x[i].store(dst);
            }
        }
    }
}

template <typename T, bool READ>
cudaError_t launch_cache(const CacheDims& C, bool e4m3, const hla_cache& c, T* k, T* v, const int32_t* cu,
                         const int64_t* start, cudaStream_t st) {
    static DeviceCache cache;
    int n_sm = 0;
    cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* x) { return sm_count(dev, x); });
    if (e != cudaSuccess) return e;
    if (C.total <= 0) return cudaSuccess;
    // Tokens per block: four batches of rows for every thread, fewer where that would leave SMs without a block.
    const int at_once = kThreads / (C.d / 8) * kBatch;  // rows in flight in a block
    const int64_t want = std::max<int64_t>(1, 4 * at_once / (2 * C.Hkv)), spread = std::max<int64_t>(1, C.total / (2 * n_sm));
    const int tokens = (int)std::min<int64_t>(kMaxTokens, std::min(want, spread));
    const int64_t blocks = (C.total + tokens - 1) / tokens;
    auto run = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, st>>>(C, c, k, v, cu, start, tokens);
        return cudaGetLastError();
    };
    if (C.d == 128) return e4m3 ? run(cache_kernel<T, true, READ, 16>) : run(cache_kernel<T, false, READ, 16>);
    return e4m3 ? run(cache_kernel<T, true, READ, 8>) : run(cache_kernel<T, false, READ, 8>);
}

}  // namespace

template <typename T>
cudaError_t launch_cache_write(const CacheDims& C, bool e4m3, const hla_cache& c, const T* k, const T* v,
                               const int32_t* cu, const int64_t* start, cudaStream_t st) {
    return launch_cache<T, false>(C, e4m3, c, const_cast<T*>(k), const_cast<T*>(v), cu, start, st);
}
template <typename T>
cudaError_t launch_cache_read(const CacheDims& C, bool e4m3, const hla_cache& c, T* k, T* v, const int32_t* cu,
                              const int64_t* start, cudaStream_t st) {
    return launch_cache<T, true>(C, e4m3, c, k, v, cu, start, st);
}
#define HLA_INST(T)                                                                                               \
    template cudaError_t launch_cache_write<T>(const CacheDims&, bool, const hla_cache&, const T*, const T*,      \
                                               const int32_t*, const int64_t*, cudaStream_t);                     \
    template cudaError_t launch_cache_read<T>(const CacheDims&, bool, const hla_cache&, T*, T*, const int32_t*,   \
                                              const int64_t*, cudaStream_t);
HLA_INST(float)
HLA_INST(__nv_bfloat16)
#undef HLA_INST

}  // namespace hla
