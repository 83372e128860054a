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
// sequence and page, then d / 16 lanes hold a row, eight values of each half
// each (16-byte loads of bf16 rows, 8-byte stores), the largest magnitude by
// integer maxima and shuffles; every thread has four bf16 rows in flight.
// 32575 tokens, 8 heads of 128, bf16: written in 34 us (5.9 TB/s), read back in
// 35 us (5.7 TB/s).  With eight values per lane, a division per row and fp32
// maxima that leave out infinities one by one, the kernel was bound by its
// instructions (53 and 43 us); with a search and 64-bit divisions per row in
// place of the per-token step it took three times as long again.
#include <cuda_fp8.h>

#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 8;  // rows in flight per thread: this by the bytes of a value

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

// Largest finite magnitude of a row, its P pieces over LPR lanes.  By integer maxima of the values' bits (two at a time
// for bf16); rows with infinities or NaN again, value by value.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t top_bits(const Row8<__nv_bfloat16>& x) {  // two maxima
    return max_u16x2(max_u16x2(x.r.x & 0x7fff7fffu, x.r.y & 0x7fff7fffu), max_u16x2(x.r.z & 0x7fff7fffu, x.r.w & 0x7fff7fffu));
}
__device__ __forceinline__ uint32_t top_bits(const Row8<float>& x) {
    float f[8];
    x.get(f);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    return m;
}
template <typename T, int P, int LPR>
__device__ __forceinline__ float row_top(const Row8<T> (&x)[P], bool on) {
    constexpr bool kPair = sizeof(T) == 2;
    uint32_t m = 0;
    if (on)
#pragma unroll
        for (int p = 0; p < P; ++p) m = kPair ? max_u16x2(m, top_bits(x[p])) : max(m, top_bits(x[p]));
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) {
        const uint32_t y = __shfl_xor_sync(0xffffffffu, m, o);
        m = kPair ? max_u16x2(m, y) : max(m, y);
    }
    if (kPair) m = max(m << 16, m & 0xffff0000u);
    if (!__any_sync(0xffffffffu, m >= 0x7f800000u)) return __uint_as_float(m);
    float top = 0.f;
    if (on)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float f[8];
            x[p].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]) < INFINITY ? fabsf(f[j]) : 0.f);
        }
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}

// d / 16 consecutive lanes per row, each with eight values of each half; rows of a token: Hkv of k, then Hkv of v.
constexpr int kMaxTokens = 64;  // tokens of a block
template <typename T, bool E4M3, bool READ, int LPR>
__global__ void __launch_bounds__(kThreads)
cache_kernel(CacheDims C, hla_cache c, T* k, T* v, const int32_t* __restrict__ cu, const int64_t* __restrict__ start,
             int tokens) {
    constexpr int P = 2, D = LPR * 8 * P, kRows = kThreads / LPR;  // rows the block handles at once
    constexpr int kBatch = kInFlight / (int)sizeof(T);
    __shared__ int64_t base[kMaxTokens];  // cache row of head 0 (-1: none)
    __shared__ bool listed[kMaxTokens];
    const int lane8 = (threadIdx.x % LPR) * 8, per = 2 * C.Hkv;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, C.total - t0);
    if (blockIdx.x == 0) attn_check_table(cu, C.n_seqs, C.total, c.err);
    if ((int)threadIdx.x < nt) {
        bool in;
        base[threadIdx.x] = token_row(C, c, cu, start, t0 + threadIdx.x, &in);
        listed[threadIdx.x] = in;
    }
    __syncthreads();
    // a thread's rows: every kRows-th, as (token, row of the token)
    const int dt = kRows / per, dh = kRows - dt * per;
    int t = (int)(threadIdx.x / LPR) / per, hh = (int)(threadIdx.x / LPR) - t * per;
    for (int r0 = 0; r0 < nt * per; r0 += kRows * kBatch) {  // the whole block together
        Row8<T> x[kBatch][P];
        uint2 q8[kBatch][P];
        int eb[kBatch];
        T* own[kBatch];        // values of k or v (null: none)
        int64_t at[kBatch];    // cache row (-1: none)
        bool isv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            own[i] = nullptr;
            at[i] = -1;
            isv[i] = hh >= C.Hkv;
            if (t < nt && listed[t]) {
                const int h = isv[i] ? hh - C.Hkv : hh;
                own[i] = (isv[i] ? v : k) + ((t0 + t) * C.Hkv + h) * D + lane8;
                if (base[t] >= 0) at[i] = base[t] + (int64_t)h * C.page;
            }
            if (at[i] >= 0) {
                if constexpr (!READ) {
#pragma unroll
                    for (int p = 0; p < P; ++p) x[i][p].load(own[i] + p * (D / 2));
                } else if constexpr (E4M3) {
                    const uint8_t* src = static_cast<const uint8_t*>(isv[i] ? c.v : c.k) + at[i] * D + lane8;
#pragma unroll
                    for (int p = 0; p < P; ++p) q8[i][p] = __ldcs(reinterpret_cast<const uint2*>(src + p * (D / 2)));
                    eb[i] = (isv[i] ? c.v_exp : c.k_exp)[at[i]];
                } else {
                    const T* src = static_cast<const T*>(isv[i] ? c.v : c.k) + at[i] * D + lane8;
#pragma unroll
                    for (int p = 0; p < P; ++p) x[i][p].load(src + p * (D / 2));
                }
            }
            t += dt;
            hh += dh;
            if (hh >= per) {
                hh -= per;
                ++t;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if constexpr (!READ && E4M3) {
                const float top = row_top<T, P, LPR>(x[i], at[i] >= 0);
                if (at[i] < 0) continue;
                const int e = row_exponent(top);
                const float inv = pow2(-e);
                uint8_t* dst = static_cast<uint8_t*>(isv[i] ? c.v : c.k) + at[i] * D + lane8;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float f[8];
                    x[i][p].get(f);
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE,
                                                        __NV_E4M3);
                    *reinterpret_cast<uint2*>(dst + p * (D / 2)) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
                }
                if (lane8 == 0) (isv[i] ? c.v_exp : c.k_exp)[at[i]] = (uint8_t)(e + 127);
            } else if constexpr (!READ) {
                if (at[i] < 0) continue;
                T* dst = static_cast<T*>(isv[i] ? c.v : c.k) + at[i] * D + lane8;
#pragma unroll
                for (int p = 0; p < P; ++p) x[i][p].store(dst + p * (D / 2));
            } else {
                if (!own[i]) continue;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float f[8];
                    if (at[i] < 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = 0.f;
                        x[i][p].set(f);
                    } else if constexpr (E4M3) {
                        const float s = pow2(eb[i] - 127);
                        const uint32_t w[2] = {q8[i][p].x, q8[i][p].y};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j & 1)));
                            const float2 g = __half22float2(__half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3))));
                            f[2 * j] = g.x * s;
                            f[2 * j + 1] = g.y * s;
                        }
                        x[i][p].set(f);
                    }
                    x[i][p].store(own[i] + p * (D / 2));
                }
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
    // Tokens per block: two batches of rows for every thread (one or four: up to 4 % more for 32575 tokens), fewer where
    // that would leave SMs without a block.
    const int at_once = kThreads / (C.d / 16) * (kInFlight / (int)sizeof(T));  // rows in flight in a block
    const int64_t want = std::max<int64_t>(1, 2 * at_once / (2 * C.Hkv)), spread = std::max<int64_t>(1, C.total / (2 * n_sm));
    const int tokens = (int)std::min<int64_t>(kMaxTokens, std::min(want, spread));
    const int64_t blocks = (C.total + tokens - 1) / tokens;
    auto run = [&](auto kernel) {
        kernel<<<(unsigned)blocks, kThreads, 0, st>>>(C, c, k, v, cu, start, tokens);
        return cudaGetLastError();
    };
    if (C.d == 128) return e4m3 ? run(cache_kernel<T, true, READ, 8>) : run(cache_kernel<T, false, READ, 8>);
    return e4m3 ? run(cache_kernel<T, true, READ, 4>) : run(cache_kernel<T, false, READ, 4>);
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
