// Root-mean-square norms with the residual's addition, and their gradient.
//
//   s = x + residual (rounded to the layer's type, kept),
//   y = s r (offset + w),  r = 1 / sqrt(mean s^2 + eps)
//   ds = r (w dy - s r^2 mean(w dy s)) + dsum,   dw = sum over rows of dy s r
//
// Memory bound: a row is read once into registers, reduced, and written once.
// A row of up to 32 pieces of 16 bytes is taken by 4 to 32 lanes of a warp, a
// longer one by a block with up to four pieces a thread (sixteen single values
// where a row does not start on 16 bytes), rows past that by a block that
// reads them twice.
// The gradient's blocks stay and walk the rows, so that a thread adds up dw of
// its own columns in registers; the blocks' sums are added in order by a second
// launch.  A thread has one piece of a row where 1024 threads can (then the next
// row is on its way while this one is reduced), else two or four that it reads
// again behind the reduction, from L2: registers are what a row's length is
// limited by.
#include <algorithm>

#include "layer.cuh"

namespace hla {

namespace {

constexpr int kNarrow = 128;  // threads of a block whose rows take a warp or less

// The sum of v over the tpr threads of a row (tpr a power of two up to 32, or all threads of the block).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float* sm) {
    for (int o = min(tpr, 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = tpr >> 5;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) sm[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float y = lane < n ? sm[i * 32 + lane] : 0.f;
        for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        v[i] = y;
    }
}

__device__ __forceinline__ float row_max(float v, int tpr, float* sm) {
    for (int o = min(tpr, 32) / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr <= 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) sm[warp] = v;
    __syncthreads();
    v = lane < (tpr >> 5) ? sm[lane] : 0.f;
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float finite_size(float y) {  // |y|, 0 for infinities and NaN
    const uint32_t b = __float_as_uint(y) & 0x7fffffffu;
    return b < 0x7f800000u ? __uint_as_float(b) : 0.f;
}

template <int V>
__device__ __forceinline__ void store_8_bits(uint8_t* p, const float* y, float inv) {
    if constexpr (V >= 4) {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i] * inv, y[4 * i + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2] * inv, y[4 * i + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | hi << 16;
        }
        if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
        *p = (uint8_t)__nv_cvt_float_to_fp8(*y * inv, __NV_SATFINITE, __NV_E4M3);
    }
}

// Where a row starts, given the token stride.
__device__ __forceinline__ int64_t row_at(const NormDims& N, int64_t row, int64_t stride) {
    if (N.heads == 1) return row * stride;
    const int64_t token = row / N.heads;
    return token * stride + (row - token * N.heads) * N.cols;
}

template <int V, int P> struct Bound {
    static constexpr int threads = V == 1 || P > 1 ? 1024 : 256;
    static constexpr int blocks = (V > 1 && P == 1 ? 1536 : 1024) / threads;
};

// A row's P pieces of V values per thread, piece p at (p tpr + thread) V.  Eight bits: a group's values lie in
// neighbouring lanes of one piece index (its pieces are a power of two that divides 32, and tpr is a multiple of it).
template <typename T, int V, int P, bool E4M3>
__global__ void __launch_bounds__(Bound<V, P>::threads, Bound<V, P>::blocks)
norm_kernel(const NormDims N, const T* x, const T* residual, const T* __restrict__ weight, T* out, uint8_t* out8,
            uint8_t* exps, T* sum, int tpr) {
    using Pc = Piece<T, V>;
    __shared__ float sm[64];
    const int group = tpr > 32 ? 0 : threadIdx.x / tpr, lane = threadIdx.x - group * tpr;
    const int64_t row = tpr > 32 ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / tpr) + group;
    const bool on = row < N.rows;
    const T* xr = x + (on ? row_at(N, row, N.sx) : 0);
    const int64_t dense = (on ? row : 0) * N.cols;
    Pc a[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * tpr + lane) * V;
        a[p] = on && e < N.cols ? *reinterpret_cast<const Pc*>(xr + e) : Pc{};
    }
    if (residual) {
        const T* rr = residual + (on ? row_at(N, row, N.sr) : 0);
        Pc b[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            b[p] = on && e < N.cols ? *reinterpret_cast<const Pc*>(rr + e) : Pc{};
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < V; ++j) a[p].x[j] = from_f32<T>(to_f32(a[p].x[j]) + to_f32(b[p].x[j]));
    }
    float v[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < V; ++j) v[0] += to_f32(a[p].x[j]) * to_f32(a[p].x[j]);
    row_sum(v, tpr, sm);
    const float r = 1.f / sqrtf(v[0] / (float)N.cols + N.eps);
    // the sum is written once the whole row has been read: it may lie where x or the residual does
    if (sum) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            if (on && e < N.cols) *reinterpret_cast<Pc*>(sum + dense + e) = a[p];
        }
    }
    auto values = [&](int p, int e, float (&y)[V]) {
        if (weight) {
            const Pc w = e < N.cols ? *reinterpret_cast<const Pc*>(weight + e) : Pc{};
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = to_f32(a[p].x[j]) * r * (N.offset + to_f32(w.x[j]));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = to_f32(a[p].x[j]) * r;
        }
    };
    if constexpr (!E4M3) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            if (!on || e >= N.cols) continue;
            float y[V];
            values(p, e, y);
            Pc o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.x[j] = from_f32<T>(y[j]);
            *reinterpret_cast<Pc*>(out + dense + e) = o;
        }
    } else {
        const int per = N.group ? N.cols / N.group : 1;  // exponents of a row
        auto store = [&](int e, const float (&y)[V], float top) {
            if (!on || e >= N.cols) return;
            const int q = group_exponent(top);
            store_8_bits<V>(out8 + dense + e, y, group_pow2(-q));
            if (N.group ? e % N.group == 0 : e == 0) exps[row * per + (N.group ? e / N.group : 0)] = (uint8_t)(q + 127);
        };
        auto size = [&](const float (&y)[V]) {  // (columns past the row's are 0)
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) top = fmaxf(top, finite_size(y[j]));
            return top;
        };
        float y[V];
        if (N.group) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * tpr + lane) * V;
                values(p, e, y);
                float top = on && e < N.cols ? size(y) : 0.f;
                for (int o = N.group / V / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                store(e, y, top);
            }
        } else {
            float all = 0.f;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * tpr + lane) * V;
                values(p, e, y);
                if (on && e < N.cols) all = fmaxf(all, size(y));
            }
            all = row_max(all, tpr, sm + 32);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * tpr + lane) * V;
                values(p, e, y);
                store(e, y, all);
            }
        }
    }
}

// Rows too long for the registers of a block: the sum of squares, then the row again (from the sums just written, each
// by the thread that reads it).
template <typename T, bool E4M3>
__global__ void __launch_bounds__(1024)
norm_long_kernel(const NormDims N, const T* x, const T* residual, const T* __restrict__ weight, T* out, uint8_t* out8,
                 uint8_t* exps, T* sum) {
    __shared__ float sm[64];
    const int64_t row = blockIdx.x, token = row / N.heads, dense = row * N.cols;
    const int head = (int)(row - token * N.heads);
    const T* xr = x + token * N.sx + (int64_t)head * N.cols;
    const T* rr = residual + token * N.sr + (int64_t)head * N.cols;
    auto stored = [&](int e) { return residual ? from_f32<T>(to_f32(xr[e]) + to_f32(rr[e])) : xr[e]; };
    float v[1] = {0.f};
    for (int e = threadIdx.x; e < N.cols; e += blockDim.x) {
        const T s = stored(e);
        if (sum) sum[dense + e] = s;
        v[0] += to_f32(s) * to_f32(s);
    }
    const T* sr = sum ? sum + dense : xr;
    row_sum(v, 1024, sm);
    const float r = 1.f / sqrtf(v[0] / (float)N.cols + N.eps);
    auto value = [&](int e) { return to_f32(sr[e]) * r * (weight ? N.offset + to_f32(weight[e]) : 1.f); };
    if constexpr (!E4M3) {
        for (int e = threadIdx.x; e < N.cols; e += blockDim.x) out[dense + e] = from_f32<T>(value(e));
    } else {
        const int group = N.group ? N.group : N.cols, per = N.cols / group;
        if (N.group) {  // a warp per group
            for (int g = threadIdx.x >> 5; g < per; g += 32) {
                float top = 0.f;
                for (int e = g * group + (threadIdx.x & 31); e < (g + 1) * group; e += 32) top = fmaxf(top, finite_size(value(e)));
                top = row_max(top, 32, sm);
                const int q = group_exponent(top);
                for (int e = g * group + (threadIdx.x & 31); e < (g + 1) * group; e += 32) {
                    const float y = value(e);
                    store_8_bits<1>(out8 + dense + e, &y, group_pow2(-q));
                }
                if ((threadIdx.x & 31) == 0) exps[row * per + g] = (uint8_t)(q + 127);
            }
        } else {
            float top = 0.f;
            for (int e = threadIdx.x; e < N.cols; e += blockDim.x) top = fmaxf(top, finite_size(value(e)));
            top = row_max(top, 1024, sm + 32);
            const int q = group_exponent(top);
            for (int e = threadIdx.x; e < N.cols; e += blockDim.x) {
                const float y = value(e);
                store_8_bits<1>(out8 + dense + e, &y, group_pow2(-q));
            }
            if (threadIdx.x == 0) exps[row] = (uint8_t)(q + 127);
        }
    }
}

// The gradient.  part [gridDim.x][cols]: this block's sums of dy s r.
// MOST: threads of a block, at most.
template <typename T, int V, int P, int MOST>
__global__ void __launch_bounds__(MOST, MOST == kNarrow ? 6 : 1)
norm_backward_kernel(const NormDims N, const T* s, const T* __restrict__ weight, const T* dout, const T* dsum, T* dx,
                     float* part, int tpr) {
    using Pc = Piece<T, V>;
    constexpr bool kAgain = P * V * sizeof(T) > 16;                             // pieces are read again, not held
    constexpr bool kAhead = P == 1 && V * (MOST == 1024 ? 8 / sizeof(T) : 1) <= 8;  // the next row's are loaded early
    constexpr int H = kAgain ? 1 : P;
    __shared__ float sm[2][64];
    extern __shared__ float cols_sm[];  // rows of a warp or less: the sums of every group of lanes
    const int groups = tpr > 32 ? 1 : blockDim.x / tpr, group = tpr > 32 ? 0 : threadIdx.x / tpr;
    const int lane = threadIdx.x - group * tpr;
    const float inv = 1.f / (float)N.cols;
    Pc w[H];
    float acc[P][V];
    auto factor = [&](int p, int e) {
        return weight && e < N.cols ? *reinterpret_cast<const Pc*>(weight + e) : Pc{};
    };
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (!kAgain) w[kAgain ? 0 : p] = factor(p, (p * tpr + lane) * V);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[p][j] = 0.f;
    }
    const float one = weight ? N.offset : 1.f;  // (without a weight w is 0)
    const int64_t step = (int64_t)gridDim.x * groups;
    Pc a[H], d[H], g[H];
    auto load = [&](int64_t row, int p, Pc& a, Pc& d, Pc& g, bool with_sum) {
        const int e = (p * tpr + lane) * V;
        const bool on = row < N.rows && e < N.cols;
        a = on ? *reinterpret_cast<const Pc*>(s + row_at(N, row, N.sx) + e) : Pc{};
        d = on ? *reinterpret_cast<const Pc*>(dout + row * N.cols + e) : Pc{};
        if (with_sum) g = on && dsum ? *reinterpret_cast<const Pc*>(dsum + row * N.cols + e) : Pc{};
    };
    if (kAhead) load((int64_t)blockIdx.x * groups + group, 0, a[0], d[0], g[0], true);
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < N.rows; row0 += step, turn ^= 1) {
        const int64_t row = row0 + group;
        Pc a1, d1, g1;
        if constexpr (kAhead) load(row + step, 0, a1, d1, g1, true);
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int h = kAgain ? 0 : p;
            if constexpr (!kAhead) load(row, p, a[h], d[h], g[h], !kAgain);
            if constexpr (kAgain) w[h] = factor(p, (p * tpr + lane) * V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = to_f32(a[h].x[j]);
                v[0] += x * x;
                v[1] += (one + to_f32(w[h].x[j])) * to_f32(d[h].x[j]) * x;
            }
        }
        row_sum(v, tpr, sm[turn]);  // (sums of the row before last have been read by all)
        const float r = 1.f / sqrtf(v[0] * inv + N.eps), c = v[1] * inv * r * r;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V, h = kAgain ? 0 : p;
            if constexpr (kAgain) {
                load(row, p, a[h], d[h], g[h], true);
                w[h] = factor(p, e);
            }
            Pc o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = to_f32(a[h].x[j]), dy = to_f32(d[h].x[j]);
                o.x[j] = from_f32<T>(((one + to_f32(w[h].x[j])) * dy - x * c) * r + to_f32(g[h].x[j]));
                acc[p][j] += dy * (x * r);
            }
            if (row < N.rows && e < N.cols) *reinterpret_cast<Pc*>(dx + row * N.cols + e) = o;
        }
        if constexpr (kAhead) {
            a[0] = a1;
            d[0] = d1;
            g[0] = g1;
        }
    }
    if (!part) return;
    float* mine = part + (int64_t)blockIdx.x * N.cols;
    if (groups == 1) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            if (e >= N.cols) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) mine[e + j] = acc[p][j];
        }
        return;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * tpr + lane) * V;
        if (e >= N.cols) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) cols_sm[group * N.cols + e + j] = acc[p][j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < N.cols; e += blockDim.x) {
        float y = 0.f;
        for (int k = 0; k < groups; ++k) y += cols_sm[k * N.cols + e];
        mine[e] = y;
    }
}

// Rows too long for registers: twice over the row; a block's sums of dw lie in its own row of part.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_backward_long_kernel(const NormDims N, const T* s, const T* __restrict__ weight, const T* dout, const T* dsum,
                          T* dx, float* part) {
    __shared__ float sm[64];
    const float inv = 1.f / (float)N.cols;
    float* mine = part + (int64_t)blockIdx.x * N.cols;
    bool first = true;
    for (int64_t row = blockIdx.x; row < N.rows; row += gridDim.x) {
        const int64_t token = row / N.heads, dense = row * N.cols;
        const T* sr = s + token * N.sx + (row - token * N.heads) * N.cols;
        float v[2] = {0.f, 0.f};
        for (int e = threadIdx.x; e < N.cols; e += blockDim.x) {
            const float x = to_f32(sr[e]);
            v[0] += x * x;
            v[1] += (weight ? N.offset + to_f32(weight[e]) : 1.f) * to_f32(dout[dense + e]) * x;
        }
        row_sum(v, 1024, sm);
        const float r = 1.f / sqrtf(v[0] * inv + N.eps), c = v[1] * inv * r * r;
        for (int e = threadIdx.x; e < N.cols; e += blockDim.x) {
            const float x = to_f32(sr[e]), dy = to_f32(dout[dense + e]);
            const float f = weight ? N.offset + to_f32(weight[e]) : 1.f;
            const T o = from_f32<T>((f * dy - x * c) * r + (dsum ? to_f32(dsum[dense + e]) : 0.f));
            dx[dense + e] = o;
            if (part) mine[e] = (first ? 0.f : mine[e]) + dy * (x * r);
        }
        first = false;
        __syncthreads();  // sm is written again
    }
}

// dweight[c] = sum over parts, in order: 32 columns a block, 32 runs of parts side by side.
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* __restrict__ part, int parts, int cols,
                                                          float* __restrict__ dweight) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int per = (parts + 31) / 32, k1 = min(parts, (run + 1) * per);
    float y = 0.f;
    if (c < cols)
        for (int k = run * per; k < k1; ++k) y += part[(int64_t)k * cols + c];
    sm[run][lane] = y;
    __syncthreads();
    if (run == 0 && c < cols) {
        y = 0.f;
        for (int k = 0; k < 32; ++k) y += sm[k][lane];
        dweight[c] = y;
    }
}

// Threads of a row and pieces of a thread for `pieces` pieces; 0 threads: the long kernel.
struct RowShape {
    int tpr, p;
};
RowShape row_shape(int pieces, bool single, bool backward) {
    if (pieces <= 32) {
        int t = 4;
        while (t < pieces) t *= 2;
        return {t, 1};
    }
    auto threads = [&](int p) { return ((pieces + p - 1) / p + 31) / 32 * 32; };
    if (single) return pieces <= 4096 ? RowShape{threads(4), 4} : pieces <= 16384 ? RowShape{threads(16), 16} : RowShape{0, 0};
    if (pieces <= (backward ? 1024 : 256)) return {threads(1), 1};
    if (pieces <= 2048) return {threads(2), 2};
    return pieces <= 4096 ? RowShape{threads(4), 4} : RowShape{0, 0};
}

template <typename T, int V, int P>
cudaError_t forward(const NormDims& N, const T* x, const T* residual, const T* weight, T* out, uint8_t* out8,
                    uint8_t* exps, T* sum, int tpr, cudaStream_t st) {
    const int threads = tpr <= 32 ? kNarrow : tpr, per = threads / tpr;
    const int64_t blocks = (N.rows + per - 1) / per;
    if constexpr (V > 1)
        if (out8) {
            norm_kernel<T, V, P, true><<<(unsigned)blocks, threads, 0, st>>>(N, x, residual, weight, out, out8, exps, sum, tpr);
            return cudaGetLastError();
        }
    norm_kernel<T, V, P, false><<<(unsigned)blocks, threads, 0, st>>>(N, x, residual, weight, out, out8, exps, sum, tpr);
    return cudaGetLastError();
}

template <typename T, int V, int P>
cudaError_t backward(const NormDims& N, const T* s, const T* weight, const T* dout, const T* dsum, T* dx, float* part,
                     int tpr, int* blocks, cudaStream_t st) {
    static DeviceCache cache;
    int n_sm = 0;
    cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
    if (e != cudaSuccess) return e;
    const int threads = tpr <= 32 ? kNarrow : tpr, groups = threads / tpr;
    const int resident = std::max(1, 768 / threads);
    *blocks = (int)std::min<int64_t>({(N.rows + groups - 1) / groups, (int64_t)n_sm * resident, kNormParts});
    const size_t sm = groups > 1 ? (size_t)groups * N.cols * sizeof(float) : 0;  // at most 128 threads x 8 values
    auto go = [&](auto most) {
        norm_backward_kernel<T, V, P, decltype(most)::value><<<*blocks, threads, sm, st>>>(N, s, weight, dout, dsum, dx, part, tpr);
        return cudaGetLastError();
    };
    if constexpr (V > 1 && P == 1) {
        if (threads <= kNarrow) return go(std::integral_constant<int, kNarrow>());
        if (threads <= 768) return go(std::integral_constant<int, 768>());
    }
    return go(std::integral_constant<int, 1024>());
}

template <typename T>
bool wide(const NormDims& N, uintptr_t p) {  // 16-byte pieces everywhere
    constexpr int V = 16 / (int)sizeof(T);
    return p % 16 == 0 && (N.cols | N.sx | N.sr) % V == 0;
}

}  // namespace

template <typename T>
cudaError_t launch_norm(const NormDims& N, const T* x, const T* residual, const T* weight, T* out, uint8_t* out8,
                        uint8_t* exps, T* sum, cudaStream_t st) {
    if (N.rows == 0) return cudaSuccess;
    constexpr int V = 16 / (int)sizeof(T);
    const uintptr_t a = (uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)out | (uintptr_t)sum;
    const bool vec = wide<T>(N, a);
    const RowShape r = row_shape(vec ? N.cols / V : N.cols, !vec, false);
    auto run = [&](auto v, auto p) {
        return forward<T, decltype(v)::value, decltype(p)::value>(N, x, residual, weight, out, out8, exps, sum, r.tpr, st);
    };
    using One = std::integral_constant<int, 1>;
    using Vec = std::integral_constant<int, V>;
    if (r.tpr == 0) {
        if (out8) norm_long_kernel<T, true><<<(unsigned)N.rows, 1024, 0, st>>>(N, x, residual, weight, out, out8, exps, sum);
        else norm_long_kernel<T, false><<<(unsigned)N.rows, 1024, 0, st>>>(N, x, residual, weight, out, out8, exps, sum);
        return cudaGetLastError();
    }
    if (!vec) return r.p == 1 ? run(One(), One()) : r.p == 4 ? run(One(), std::integral_constant<int, 4>()) : run(One(), std::integral_constant<int, 16>());
    return r.p == 1 ? run(Vec(), One()) : r.p == 2 ? run(Vec(), std::integral_constant<int, 2>()) : run(Vec(), std::integral_constant<int, 4>());
}

template <typename T>
cudaError_t launch_norm_backward(const NormDims& N, const T* s, const T* weight, const T* dout, const T* dsum, T* dx,
                                 float* dweight, float* part, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!dweight) part = nullptr;
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (N.rows > 0) {
        const uintptr_t a = (uintptr_t)s | (uintptr_t)weight | (uintptr_t)dout | (uintptr_t)dsum | (uintptr_t)dx;
        const bool vec = wide<T>(N, a);
        const RowShape r = row_shape(vec ? N.cols / V : N.cols, !vec, true);
        auto run = [&](auto v, auto p) {
            return backward<T, decltype(v)::value, decltype(p)::value>(N, s, weight, dout, dsum, dx, part, r.tpr, &blocks, st);
        };
        using One = std::integral_constant<int, 1>;
        using Vec = std::integral_constant<int, V>;
        if (r.tpr == 0) {
            blocks = (int)std::min<int64_t>(N.rows, 304);
            norm_backward_long_kernel<T><<<blocks, 1024, 0, st>>>(N, s, weight, dout, dsum, dx, part);
            e = cudaGetLastError();
        } else if (!vec) {
            e = r.p == 1 ? run(One(), One()) : r.p == 4 ? run(One(), std::integral_constant<int, 4>()) : run(One(), std::integral_constant<int, 16>());
        } else {
            e = r.p == 1 ? run(Vec(), One()) : r.p == 2 ? run(Vec(), std::integral_constant<int, 2>()) : run(Vec(), std::integral_constant<int, 4>());
        }
    }
    if (e != cudaSuccess || !dweight) return e;
    norm_parts_kernel<<<(unsigned)((N.cols + 31) / 32), 1024, 0, st>>>(part, blocks, N.cols, dweight);
    return cudaGetLastError();
}

#define HLA_NORM(T)                                                                                                  \
    template cudaError_t launch_norm<T>(const NormDims&, const T*, const T*, const T*, T*, uint8_t*, uint8_t*, T*,   \
                                        cudaStream_t);                                                               \
    template cudaError_t launch_norm_backward<T>(const NormDims&, const T*, const T*, const T*, const T*, T*,        \
                                                 float*, float*, cudaStream_t);
HLA_NORM(float)
HLA_NORM(__nv_bfloat16)

}  // namespace hla
