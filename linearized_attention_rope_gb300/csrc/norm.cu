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
// launch.  Rows come through a ring in shared memory, filled by bulk copies, in
// the gradient and where the norm of 16-bit rows has more than three rows a
// block: loads go on while a row is reduced.
// Measured: 32767 rows of 5120 bf16 with the residual 213 us, 94 % of the copy
// rate (a block a row: 259); 4097 rows of 4096 fp32 42 us, 96 %; gradients: 524352
// heads of 128 bf16 72 us (83 %), 4097 rows of 4096 fp32 with the stream's 48 us
// (84 %), 32767 rows of 5120 bf16 296 us (68 %: two pieces a thread, whose sums of
// dw and factors take the registers).
// Spilled at the 64 registers that blocks of up to 1024 threads leave (bytes stored
// and loaded a thread): gradients of bf16 rows in two pieces 72 and 144, in four 104
// and 104; norms of bf16 rows in four 56 to 84 and 116 to 280; sixteen single
// values a thread 44 to 60 and 76 to 100, their gradient 660 and 764.
#include <algorithm>

#include "layer.cuh"
#include "tma.cuh"
#include "umma.cuh"

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

template <typename T, int V> __device__ __forceinline__ void add_to(Piece<T, V>& a, const Piece<T, V>& b) {
#pragma unroll
    for (int j = 0; j < V; ++j) a.x[j] = from_f32<T>(to_f32(a.x[j]) + to_f32(b.x[j]));
}

// A ring of row buffers that bulk copies fill.  Every wait ends; after one that ran out a block loads no more and its rows
// are NaN.
constexpr int kStages = 8;
constexpr uint32_t kPolls = 1u << 22;
__device__ __forceinline__ void start_ring(uint64_t* full, int stages, int* dead) {
    if (threadIdx.x == 0) {
        *dead = 0;
        for (int i = 0; i < stages; ++i) umma::mbar_init(umma::smem_addr(full + i), 1);
        umma::fence_mbar_init();
    }
    __syncthreads();
}
__device__ __forceinline__ bool wait_ring(uint64_t* full, uint32_t turn, int* dead) {
    const uint32_t bar = umma::smem_addr(full);
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (umma::mbar_try_wait(bar, turn)) return true;
    if (!*(volatile int*)dead && umma::mbar_wait(bar, turn, kPolls)) return true;
    *dead = 1;
    return false;
}
// Copies in flight end before the block does.  (After a wait that ran out; else every buffer has been waited for.)
__device__ __forceinline__ void end_ring(uint64_t* full, int stages, int dead) {
    if (!dead) return;
    for (int i = 0; i < 2 * stages; ++i) umma::mbar_wait(umma::smem_addr(full + i % stages), i / stages, kPolls / 8, 100000000ull);
}

// A row's P pieces of V values per thread, piece p at (p tpr + thread) V: the sum of squares, then the sum and the outputs.
// Eight bits: a group's values lie in neighbouring lanes of one piece index (its pieces are a power of two that divides
// 32, and tpr is a multiple of it).  `between` runs once every thread of the row has its pieces.
template <typename T, int V, int P, bool E4M3, typename F>
__device__ __forceinline__ void norm_row(const NormDims& N, Piece<T, V> (&a)[P], const T* __restrict__ weight, T* out,
                                         uint8_t* out8, uint8_t* exps, T* sum, int64_t row, bool on, int lane, int tpr,
                                         float* sm, F between) {
    using Pc = Piece<T, V>;
    const int64_t dense = (on ? row : 0) * N.cols;
    float v[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < V; ++j) v[0] += to_f32(a[p].x[j]) * to_f32(a[p].x[j]);
    row_sum(v, tpr, sm);
    between();
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
        for (int p = 0; p < P; ++p) add_to(a[p], b[p]);
    }
    norm_row<T, V, P, E4M3>(N, a, weight, out, out8, exps, sum, row, on, lane, tpr, sm, [] {});
}

// Many rows of a block each: blocks stay, and the rows to come are on their way into a ring in shared memory (x, then the
// residual), so that loads do not stop while a row is reduced.
template <typename T, int V, int P, bool E4M3>
__global__ void __launch_bounds__(P == 1 ? 256 : 1024, P == 1 ? 4 : 1)
norm_ring_kernel(const NormDims N, const T* x, const T* residual, const T* __restrict__ weight, T* out, uint8_t* out8,
                 uint8_t* exps, T* sum, int stages) {
    using Pc = Piece<T, V>;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][64];
    __shared__ alignas(8) uint64_t full[kStages];
    __shared__ int dead;
    const int lane = threadIdx.x, tpr = blockDim.x;
    const uint32_t bytes = (uint32_t)N.cols * sizeof(T), each = residual ? 2 * bytes : bytes;
    auto load = [&](int64_t row, int st) {
        if (row >= N.rows) return;
        const uint32_t bar = umma::smem_addr(full + st), at = umma::smem_addr(ring) + st * each;
        tma::expect_tx(bar, each);
        tma::bulk_load(at, x + row_at(N, row, N.sx), bytes, bar);
        if (residual) tma::bulk_load(at + bytes, residual + row_at(N, row, N.sr), bytes, bar);
    };
    start_ring(full, stages, &dead);
    if (threadIdx.x == 0)
        for (int i = 0; i < stages; ++i) load(blockIdx.x + (int64_t)i * gridDim.x, i);
    int st = 0, turn = 0, odd = 0;
    for (int64_t row = blockIdx.x; row < N.rows; row += gridDim.x) {
        const bool there = wait_ring(full + st, turn, &dead);
        const T* xr = reinterpret_cast<const T*>(ring + (size_t)st * each);
        Pc a[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            a[p] = Pc{};
            if (e < N.cols) {
                a[p] = *reinterpret_cast<const Pc*>(xr + e);
                if (residual) add_to(a[p], *reinterpret_cast<const Pc*>(xr + N.cols + e));
                if (!there) a[p].x[0] = from_f32<T>(__int_as_float(0x7fc00000));
            }
        }
        norm_row<T, V, P, E4M3>(N, a, weight, out, out8, exps, sum, row, true, lane, tpr, sm[odd], [&] {
            if (threadIdx.x == 0 && !dead) load(row + (int64_t)stages * gridDim.x, st);
        });
        odd ^= 1;
        if (++st == stages) {
            st = 0;
            turn ^= 1;
        }
    }
    end_ring(full, stages, dead);
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
// A block's sums of dw, one group of lanes after the other, to its own row of part.
template <int V, int P>
__device__ __forceinline__ void put_part(const float (&acc)[P][V], float* part, int cols, int groups, int group, int lane, int tpr,
                                         float* cols_sm) {
    if (!part) return;
    float* mine = part + (int64_t)blockIdx.x * cols;
    float* to = groups == 1 ? mine : cols_sm + group * cols;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = (p * tpr + lane) * V;
        if (e >= cols) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) to[e + j] = acc[p][j];
    }
    if (groups == 1) return;
    __syncthreads();
    for (int e = threadIdx.x; e < cols; e += blockDim.x) {
        float y = 0.f;
        for (int k = 0; k < groups; ++k) y += cols_sm[k * cols + e];
        mine[e] = y;
    }
}

template <typename T, int V, int P>
__global__ void __launch_bounds__(1024, 1)
norm_backward_kernel(const NormDims N, const T* s, const T* __restrict__ weight, const T* dout, const T* dsum, T* dx,
                     float* part, int tpr) {
    using Pc = Piece<T, V>;
    __shared__ float sm[2][64];
    extern __shared__ float cols_sm[];  // rows of a warp or less: the sums of every group of lanes
    const int groups = tpr > 32 ? 1 : blockDim.x / tpr, group = tpr > 32 ? 0 : threadIdx.x / tpr;
    const int lane = threadIdx.x - group * tpr;
    const float inv = 1.f / (float)N.cols;
    float acc[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[p][j] = 0.f;
    const float one = weight ? N.offset : 1.f;  // (without a weight w is 0)
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < N.rows; row0 += (int64_t)gridDim.x * groups, turn ^= 1) {
        const int64_t row = row0 + group;
        auto load = [&](int e, Pc& a, Pc& d, Pc& w) {
            const bool on = row < N.rows && e < N.cols;
            a = on ? *reinterpret_cast<const Pc*>(s + row_at(N, row, N.sx) + e) : Pc{};
            d = on ? *reinterpret_cast<const Pc*>(dout + row * N.cols + e) : Pc{};
            w = on && weight ? *reinterpret_cast<const Pc*>(weight + e) : Pc{};
        };
        Pc a, d, w;
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
            load((p * tpr + lane) * V, a, d, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = to_f32(a.x[j]);
                v[0] += x * x;
                v[1] += (one + to_f32(w.x[j])) * to_f32(d.x[j]) * x;
            }
        }
        row_sum(v, tpr, sm[turn]);  // (sums of the row before last have been read by all)
        const float r = 1.f / sqrtf(v[0] * inv + N.eps), c = v[1] * inv * r * r;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * tpr + lane) * V;
            if (P > 1) load(e, a, d, w);
            const bool on = row < N.rows && e < N.cols;
            const Pc g = on && dsum ? *reinterpret_cast<const Pc*>(dsum + row * N.cols + e) : Pc{};
            Pc o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = to_f32(a.x[j]), dy = to_f32(d.x[j]);
                o.x[j] = from_f32<T>(((one + to_f32(w.x[j])) * dy - x * c) * r + to_f32(g.x[j]));
                acc[p][j] += on ? dy * (x * r) : 0.f;  // (without eps r is infinite where there is no row)
            }
            if (on) *reinterpret_cast<Pc*>(dx + row * N.cols + e) = o;
        }
    }
    put_part<V, P>(acc, part, N.cols, groups, group, lane, tpr, cols_sm);
}

// A piece in fp32, two values at a time.
template <typename T, int V> __device__ __forceinline__ void pairs(const Piece<T, V>& a, float2 (&o)[V / 2]) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(a.x)[j];
            o[j] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
            o[j] = make_float2(a.x[2 * j], a.x[2 * j + 1]);
        }
    }
}

// The same from a ring of row buffers (s, dout and dsum), which both passes over a row read.  NARROW: a warp or less takes
// a row, and a buffer holds `per` dense rows; else one.  SMALL: a block of up to 128 threads, which keep their piece of the
// row in registers between the passes (100000 rows of 512 bf16: 121 us, read again 149); larger blocks read it again and are
// twice as many (65536 rows of 1024 fp32: 180 us, kept 231).
template <typename T, int P, bool NARROW, bool SMALL>
__global__ void __launch_bounds__(SMALL ? kNarrow : P == 1 ? 256 : 1024, NARROW ? 6 : SMALL || P == 1 ? 4 : 1)
norm_backward_ring_kernel(const NormDims N, const T* s, const T* __restrict__ weight, const T* dout, const T* dsum, T* dx,
                          float* part, int tpr, int stages, int per) {
    constexpr int V = 16 / (int)sizeof(T);
    using Pc = Piece<T, V>;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][64];
    __shared__ alignas(8) uint64_t full[kStages];
    __shared__ int dead;
    const int groups = NARROW ? blockDim.x / tpr : 1, group = NARROW ? threadIdx.x / tpr : 0;
    const int lane = threadIdx.x - group * tpr;
    const float inv = 1.f / (float)N.cols;
    const uint32_t row_bytes = (uint32_t)N.cols * sizeof(T), each = row_bytes * per;
    const int n_in = dsum ? 3 : 2;
    const int64_t items = (N.rows + per - 1) / per;
    auto load = [&](int64_t item, int st) {
        if (item >= items) return;
        const int64_t row = item * per;
        const uint32_t n = (uint32_t)min((int64_t)per, N.rows - row) * row_bytes;
        const uint32_t bar = umma::smem_addr(full + st), at = umma::smem_addr(ring) + st * n_in * each;
        tma::expect_tx(bar, n * n_in);
        tma::bulk_load(at, s + row_at(N, row, N.sx), n, bar);
        tma::bulk_load(at + each, dout + row * N.cols, n, bar);
        if (dsum) tma::bulk_load(at + 2 * each, dsum + row * N.cols, n, bar);
    };
    start_ring(full, stages, &dead);
    if (threadIdx.x == 0)
        for (int i = 0; i < stages; ++i) load(blockIdx.x + (int64_t)i * gridDim.x, i);
    constexpr bool kHold = P * V <= 8, kRow = SMALL;  // the factors, the row stay in registers between the passes
    constexpr int H = V / 2;
    constexpr int K = kHold ? P : 1;
    float2 f[K][H], x[H], dy[H], acc[P][H];
    const float one = weight ? N.offset : 1.f;
    auto factors = [&](int h, int e) {
        const Pc w = weight && e < N.cols ? *reinterpret_cast<const Pc*>(weight + e) : Pc{};
#pragma unroll
        for (int j = 0; j < H; ++j) f[h][j] = make_float2(one + to_f32(w.x[2 * j]), one + to_f32(w.x[2 * j + 1]));
    };
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < H; ++j) acc[p][j] = make_float2(0.f, 0.f);
    if (kHold)
#pragma unroll
        for (int p = 0; p < K; ++p) factors(p, (p * tpr + lane) * V);
    int st = 0, turn = 0, odd = 0;
    int64_t before = -1;  // the item whose buffer can be filled again, its stage the one before
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const bool there = wait_ring(full + st, turn, &dead);
        const T* base = reinterpret_cast<const T*>(ring + (size_t)st * n_in * each);
        const int64_t row0 = item * per;
        for (int k = 0; k < per; k += groups) {
            const int at = k + group;
            const bool on = at < per && row0 + at < N.rows;
            const T* sr = base + (size_t)(on ? at : 0) * N.cols;
            const T* dr = sr + (size_t)per * N.cols;
            auto take = [&](int h, int e) {
                const Pc a = *reinterpret_cast<const Pc*>(sr + e), d = *reinterpret_cast<const Pc*>(dr + e);
                pairs<T, V>(a, x);
                pairs<T, V>(d, dy);
                if (!kHold) factors(h, e);
            };
            float2 v0 = make_float2(there ? 0.f : __int_as_float(0x7fc00000), 0.f), v1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * tpr + lane) * V, h = kHold ? p : 0;
                if (e >= N.cols) continue;
                take(h, e);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    v0 = ffma2(x[j], x[j], v0);
                    v1 = ffma2(mul2(f[h][j], dy[j]), x[j], v1);
                }
            }
            float v[2] = {v0.x + v0.y, v1.x + v1.y};
            row_sum(v, tpr, sm[odd]);
            odd ^= 1;
            if (!NARROW && threadIdx.x == 0 && before >= 0 && !dead)  // every thread has left the buffer before
                load(before + (int64_t)stages * gridDim.x, (st ? st : stages) - 1);
            // c: mean of f dy x r, which is of dy's size whatever the row's (r^3 for x would pass fp32's range for small rows)
            const float r = rsqrtf(v[0] * inv + N.eps), c = -v[1] * inv * r;
            const float2 r2 = make_float2(r, r), c2 = make_float2(c, c);
            const int64_t to = (row0 + at) * N.cols;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int e = (p * tpr + lane) * V, h = kHold ? p : 0;
                if (!on || e >= N.cols) continue;
                if (!kRow) take(h, e);
                float2 g[H];
                if (dsum) pairs<T, V>(*reinterpret_cast<const Pc*>(dr + (size_t)per * N.cols + e), g);
                Pc o;
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const float2 u = mul2(x[j], r2), t = ffma2(u, c2, mul2(f[h][j], dy[j]));
                    const float2 y = dsum ? ffma2(t, r2, g[j]) : mul2(t, r2);
                    acc[p][j] = ffma2(dy[j], u, acc[p][j]);
                    o.x[2 * j] = from_f32<T>(y.x);
                    o.x[2 * j + 1] = from_f32<T>(y.y);
                }
                *reinterpret_cast<Pc*>(dx + to + e) = o;
            }
        }
        if (NARROW) {
            __syncthreads();
            if (threadIdx.x == 0 && !dead) load(item + (int64_t)stages * gridDim.x, st);
        }
        before = item;
        if (++st == stages) {
            st = 0;
            turn ^= 1;
        }
    }
    if (NARROW) __syncthreads();  // the ring's memory is used again
    float sums[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < H; ++j) {
            sums[p][2 * j] = acc[p][j].x;
            sums[p][2 * j + 1] = acc[p][j].y;
        }
    put_part<V, P>(sums, part, N.cols, groups, group, lane, tpr, reinterpret_cast<float*>(ring));
    end_ring(full, stages, dead);
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
RowShape row_shape(int pieces, bool single) {
    if (pieces <= 32) {
        int t = 4;
        while (t < pieces) t *= 2;
        return {t, 1};
    }
    auto threads = [&](int p) { return ((pieces + p - 1) / p + 31) / 32 * 32; };
    if (single) return pieces <= 4096 ? RowShape{threads(4), 4} : pieces <= 16384 ? RowShape{threads(16), 16} : RowShape{0, 0};
    if (pieces <= 256) return {threads(1), 1};
    if (pieces <= 2048) return {threads(2), 2};
    return pieces <= 4096 ? RowShape{threads(4), 4} : RowShape{0, 0};
}

// A ring's stages and blocks an SM for rows of `each` bytes in all: `resident` threads' worth of blocks, of two stages at least.
struct RingShape {
    int stages, blocks;
};
constexpr size_t kRingBytes = 204800;
RingShape ring_shape(int threads, size_t each, int resident) {
    const int blocks = (int)std::max<size_t>(1, std::min<size_t>(resident / threads, kRingBytes / (2 * each)));
    return {(int)std::min<size_t>(kStages, kRingBytes / blocks / each), blocks};
}

template <typename T, int P>
cudaError_t forward_ring(const NormDims& N, const T* x, const T* residual, const T* weight, T* out, uint8_t* out8,
                         uint8_t* exps, T* sum, int threads, const RingShape& ring, int n_sm, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const size_t sm = (size_t)ring.stages * N.cols * sizeof(T) * (residual ? 2 : 1);
    const int blocks = n_sm * ring.blocks;
    auto go = [&](auto eight) {
        const auto kernel = norm_ring_kernel<T, V, P, decltype(eight)::value>;
        static DeviceCache cache;
        cudaError_t e = device_cached(cache, nullptr, [&](int, int*) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
        });
        if (e != cudaSuccess) return e;
        kernel<<<blocks, threads, sm, st>>>(N, x, residual, weight, out, out8, exps, sum, ring.stages);
        return cudaGetLastError();
    };
    return out8 ? go(std::true_type()) : go(std::false_type());
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
                     int tpr, int n_sm, int* blocks, cudaStream_t st) {
    const int threads = tpr <= 32 ? kNarrow : tpr, groups = threads / tpr;
    *blocks = (int)std::min<int64_t>({(N.rows + groups - 1) / groups, (int64_t)n_sm * (1024 / threads), norm_parts(N.cols)});
    const size_t sm = groups > 1 ? (size_t)groups * N.cols * sizeof(float) : 0;  // at most 128 threads x 8 values
    norm_backward_kernel<T, V, P><<<*blocks, threads, sm, st>>>(N, s, weight, dout, dsum, dx, part, tpr);
    return cudaGetLastError();
}

template <typename T, int P, bool NARROW, bool SMALL>
cudaError_t backward_ring(const NormDims& N, const T* s, const T* weight, const T* dout, const T* dsum, T* dx, float* part,
                          int threads, int tpr, int stages, int resident, int per, int n_sm, int* blocks, cudaStream_t st) {
    const auto kernel = norm_backward_ring_kernel<T, P, NARROW, SMALL>;
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
    });
    if (e != cudaSuccess) return e;
    *blocks = (int)std::min<int64_t>({(N.rows + per - 1) / per, (int64_t)n_sm * resident, norm_parts(N.cols)});
    size_t sm = (size_t)stages * per * N.cols * sizeof(T) * (dsum ? 3 : 2);
    if (NARROW) sm = std::max(sm, (size_t)(threads / tpr) * N.cols * sizeof(float));
    kernel<<<*blocks, threads, sm, st>>>(N, s, weight, dout, dsum, dx, part, tpr, stages, per);
    return cudaGetLastError();
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
    const RowShape r = row_shape(vec ? N.cols / V : N.cols, !vec);
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
    if constexpr (sizeof(T) == 2) if (vec && r.tpr > 32) {
        static DeviceCache cache;
        int n_sm = 0;
        const cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
        if (e != cudaSuccess) return e;
        const int p = N.cols / V <= 256 ? 1 : 2, threads = (N.cols / V + 32 * p - 1) / (32 * p) * 32;
        const RingShape ring = ring_shape(threads, (size_t)N.cols * sizeof(T) * (residual ? 2 : 1), 1024);
        // Up to three rows a block a block a row starts sooner (640 rows of 4096: 8.4 and 8.4 us, 7680: 44 with the ring, 52
        // without); rows of fp32 go through registers as fast (65536 of 1024: 156 us, 169 with the ring).
        if (threads <= 1024 && ring.stages >= 2 && N.rows > (int64_t)3 * n_sm * ring.blocks) {
            auto go = [&](auto pp) {
                return forward_ring<T, decltype(pp)::value>(N, x, residual, weight, out, out8, exps, sum, threads, ring, n_sm, st);
            };
            return p == 1 ? go(One()) : go(std::integral_constant<int, 2>());
        }
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
    auto finish = [&](cudaError_t e) {  // the blocks' sums
        if (e != cudaSuccess || !dweight) return e;
        norm_parts_kernel<<<(unsigned)((N.cols + 31) / 32), 1024, 0, st>>>(part, blocks, N.cols, dweight);
        return cudaGetLastError();
    };
    if (N.rows > 0) {
        const uintptr_t a = (uintptr_t)s | (uintptr_t)weight | (uintptr_t)dout | (uintptr_t)dsum | (uintptr_t)dx;
        const bool vec = wide<T>(N, a);
        static DeviceCache cache;
        int n_sm = 0;
        e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
        if (e != cudaSuccess) return e;
        const int pieces = vec ? N.cols / V : N.cols, n_in = dsum ? 3 : 2;
        const RowShape r = row_shape(pieces, !vec);
        const size_t row_bytes = (size_t)N.cols * sizeof(T);
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        using Four = std::integral_constant<int, 4>;
        auto run = [&](auto v, auto p) {
            return backward<T, decltype(v)::value, decltype(p)::value>(N, s, weight, dout, dsum, dx, part, r.tpr, n_sm, &blocks, st);
        };
        if (vec && r.tpr <= 32 && r.tpr > 0 && N.heads == 1 && N.sx == N.cols) {
            // buffers of about 8 KB a tensor, a multiple of the rows that the block's lanes take at once
            const int groups = kNarrow / r.tpr, per = std::max<int>(groups, (int)(8192 / row_bytes) / groups * groups);
            const int stages = 2;
            const int resident = (int)std::min<size_t>(6, kRingBytes / (stages * per * row_bytes * n_in + 1024));
            return finish(backward_ring<T, 1, true, true>(N, s, weight, dout, dsum, dx, part, kNarrow, r.tpr, stages, resident, per, n_sm,
                                                    &blocks, st));
        }
        if (vec && r.tpr > 32) {
            const int p = pieces <= 256 ? 1 : 2, threads = (pieces + 32 * p - 1) / (32 * p) * 32;
            const RingShape ring = ring_shape(threads, row_bytes * n_in, threads <= kNarrow ? 512 : 1024);
            if (threads <= 1024 && ring.stages >= 2) {
                auto go = [&](auto pp, auto small) {
                    return backward_ring<T, decltype(pp)::value, false, decltype(small)::value>(N, s, weight, dout, dsum, dx, part, threads, threads, ring.stages,
                                                                        ring.blocks, 1, n_sm, &blocks, st);
                };
                return finish(p == 1 ? (threads <= kNarrow ? go(One(), std::true_type()) : go(One(), std::false_type()))
                              : go(Two(), std::false_type()));
            }
        }
        if (r.tpr == 0) {
            blocks = (int)std::min<int64_t>(N.rows, norm_parts(N.cols));
            norm_backward_long_kernel<T><<<blocks, 1024, 0, st>>>(N, s, weight, dout, dsum, dx, part);
            e = cudaGetLastError();
        } else if (!vec) {
            e = r.p == 1 ? run(One(), One()) : r.p == 4 ? run(One(), Four()) : run(One(), std::integral_constant<int, 16>());
        } else {
            e = r.p == 1 ? run(std::integral_constant<int, V>(), One()) : run(std::integral_constant<int, V>(), Four());
        }
    }
    return finish(e);
}

#define HLA_NORM(T)                                                                                                  \
    template cudaError_t launch_norm<T>(const NormDims&, const T*, const T*, const T*, T*, uint8_t*, uint8_t*, T*,   \
                                        cudaStream_t);                                                               \
    template cudaError_t launch_norm_backward<T>(const NormDims&, const T*, const T*, const T*, const T*, T*,        \
                                                 float*, float*, cudaStream_t);
HLA_NORM(float)
HLA_NORM(__nv_bfloat16)

}  // namespace hla
