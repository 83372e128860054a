// Packed causal attention and its gradient in fp32 on the CUDA cores: the path
// of fp32 layers, whose products the tensor cores do not form exactly.
//
// 64 x 64 tiles of (query, key) scores, 256 threads with 4 x 4 scores each,
// both operands in shared memory (key rows padded by 16 bytes so that 16
// consecutive rows are read without bank conflicts).  Forward: one pass over
// the keys with the running maximum and sum.  Gradient: the probabilities are
// recomputed from lse; one kernel per key block sums dk and dv over the query
// heads of the group and the query blocks, in order, another per query block
// sums dq.  7 products in place of the 5 that a single pass with atomics would
// take, for results that do not depend on the order of arrival.
// Bound by the fp32 FMA rate and shared-memory reads (two 16-byte reads per 4
// x 4 x 4 FMAs).
#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kB = 64;  // rows and keys of a tile
constexpr int kThreads = 256;

template <int D> constexpr int kPitch = D + 4;

// Rows [first, first + 64) of a head into shared memory as fp32; rows at or past n are zeros.
template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, const T* __restrict__ src, int64_t stride, int first, int n) {
    for (int i = threadIdx.x; i < kB * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (first + r < n) load_vec<4>(src + (int64_t)(first + r) * stride + c, x);
        *reinterpret_cast<float4*>(dst + r * kPitch<D> + c) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// s[i][j] = a row (ty 4 + i) . b row (tx + 16 j)
template <int D>
__device__ __forceinline__ void scores(const float* a, const float* b, int ty, int tx, float (&s)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * 4 + i) * kPitch<D> + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * kPitch<D> + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}

// acc[i][c] += sum_k p[row ty 4 + i][k] b[k][column], columns tx 4 + (64 c / 4); p: [64][kB + 4].  SKIP: terms with
// p = 0 are left out, for tiles in which some rows must not see what some of b's rows hold (0 times infinity).
template <int D, bool SKIP>
__device__ __forceinline__ void add_rows(const float* p, const float* b, int ty, int tx, float (&acc)[4][D / 16]) {
#pragma unroll 2
    for (int k = 0; k < kB; k += 4) {
        float w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(p + (ty * 4 + i) * (kB + 4) + k);
            w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 y = *reinterpret_cast<const float4*>(b + (k + kk) * kPitch<D> + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (SKIP && w[i][kk] == 0.f) continue;
                    acc[i][4 * c + 0] = fmaf(w[i][kk], y.x, acc[i][4 * c + 0]);
                    acc[i][4 * c + 1] = fmaf(w[i][kk], y.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(w[i][kk], y.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(w[i][kk], y.w, acc[i][4 * c + 3]);
                }
            }
    }
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int D>
__device__ __forceinline__ void store_rows(T* __restrict__ dst, int64_t stride, int first, int n, int ty, int tx,
                                           const float (&acc)[4][D / 16], const float* mul) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (first + ty * 4 + i >= n) continue;
        T* row = dst + (int64_t)(first + ty * 4 + i) * stride + tx * 4;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) row[64 * c + x] = from_f32<T>(acc[i][4 * c + x] * mul[i]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_fwd_simt_kernel(AttnDims A, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, T* __restrict__ out,
                     float* __restrict__ lse, int32_t* __restrict__ err) {
    extern __shared__ float sm[];
    float *qs = sm, *ks = qs + kB * kPitch<D>, *vs = ks + kB * kPitch<D>, *ps = vs + kB * kPitch<D>;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, kB, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, kv = h / A.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + kB, B.lq) + off);  // keys some row sees: [0, end)
    load_rows<T, D>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq);
    const float cs = A.scale * kLog2e;
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = 0; j0 < end; j0 += kB) {
        __syncthreads();
        // keys that no row of the tile sees are loaded as zeros: what they hold stays out of the sums
        load_rows<T, D>(ks, k + B.k0 * A.sk + (int64_t)kv * D, A.sk, j0, end);
        load_rows<T, D>(vs, v + B.k0 * A.sv + (int64_t)kv * D, A.sv, j0, end);
        __syncthreads();
        float s[4][4];
        scores<D>(qs, ks, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = B.first + ty * 4 + i + off;  // last key the row sees
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                s[i][j] = key <= last && key < B.lk ? s[i][j] * cs : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            const float mn = fmaxf(m[i], max16(top));
            const float corr = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - mn);
                sum += p;
                ps[(ty * 4 + i) * (kB + 4) + tx + 16 * j] = p;
            }
            l[i] = l[i] * corr + sum16(sum);
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= corr;
        }
        __syncthreads();
        if (j0 + kB > B.first + off) add_rows<D, true>(ps, vs, ty, tx, acc);
        else add_rows<D, false>(ps, vs, ty, tx, acc);
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        inv[i] = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
        const int p = B.first + ty * 4 + i;
        if (tx == 0 && p < B.lq)
            lse[(B.q0 + p) * A.Hq + h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
    store_rows<T, D>(out + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, ty, tx, acc, inv);
}

// delta[row][h] = dout . out; one warp per row and head
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_delta_kernel(int64_t rows, const T* __restrict__ out, const T* __restrict__ dout, float* __restrict__ delta) {
    const int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= rows) return;
    float a[D / 32], b[D / 32], s = 0.f;
    load_vec<D / 32>(out + r * D + (threadIdx.x & 31) * (D / 32), a);
    load_vec<D / 32>(dout + r * D + (threadIdx.x & 31) * (D / 32), b);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) delta[r] = s;
}

// Probabilities and score gradients of a tile from its recomputed scores:
// s -> p, dp -> ds (times the scale).  lse and delta of rows ty 4 + i.
template <int N>
__device__ __forceinline__ void tile_grad(float (&s)[4][4], float (&dp)[4][4], const float (&lse2)[N],
                                          const float (&dl)[N], float cs, float scale, int row0, int key0, int ty,
                                          int tx, int off, int lq, int lk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = row0 + ty * 4 + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = key0 + tx + 16 * j;
            const bool on = row < lq && key < lk && key <= row + off;
            s[i][j] = on ? exp2f(fmaf(s[i][j], cs, -lse2[i])) : 0.f;
            dp[i][j] = on ? s[i][j] * (dp[i][j] - dl[i]) * scale : 0.f;
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dkdv_simt_kernel(AttnDims A, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ lse, const T* __restrict__ dout, const float* __restrict__ delta,
                      const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, T* __restrict__ dk,
                      T* __restrict__ dv, int32_t* __restrict__ err) {
    extern __shared__ float sm[];
    float *ks = sm, *vs = ks + kB * kPitch<D>, *qs = vs + kB * kPitch<D>, *os = qs + kB * kPitch<D>;
    float *pt = os + kB * kPitch<D>, *dt = pt + kB * (kB + 4);  // [key][row]
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, kB, blockIdx.x, true);
    if (!B.found) return;
    const int kv = blockIdx.y, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq;
    load_rows<T, D>(ks, k + B.k0 * A.sk + (int64_t)kv * D, A.sk, B.first, B.lk);
    load_rows<T, D>(vs, v + B.k0 * A.sv + (int64_t)kv * D, A.sv, B.first, B.lk);
    float ak[4][D / 16], av[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
    const float cs = A.scale * kLog2e;
    const int i0 = max(0, B.first - off) / kB * kB;  // first block of rows that see the block's first key
    for (int g = 0; g < A.G; ++g) {
        const int h = kv * A.G + g;
        for (int r0 = i0; r0 < B.lq; r0 += kB) {
            __syncthreads();
            load_rows<T, D>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, r0, B.lq);
            load_rows<T, D>(os, dout + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, r0, B.lq);
            float lse2[4], dl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = B.q0 + min(r0 + ty * 4 + i, B.lq - 1);
                lse2[i] = __ldg(lse + row * A.Hq + h) * kLog2e;
                dl[i] = __ldg(delta + row * A.Hq + h);
            }
            __syncthreads();
            float s[4][4], dp[4][4];
            scores<D>(qs, ks, ty, tx, s);
            scores<D>(os, vs, ty, tx, dp);
            tile_grad(s, dp, lse2, dl, cs, A.scale, r0, B.first, ty, tx, off, B.lq, B.lk);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pt[(tx + 16 * j) * (kB + 4) + ty * 4 + i] = s[i][j];
                    dt[(tx + 16 * j) * (kB + 4) + ty * 4 + i] = dp[i][j];
                }
            __syncthreads();
            if (r0 + off < B.first + kB) {
                add_rows<D, true>(pt, os, ty, tx, av);
                add_rows<D, true>(dt, qs, ty, tx, ak);
            } else {
                add_rows<D, false>(pt, os, ty, tx, av);
                add_rows<D, false>(dt, qs, ty, tx, ak);
            }
        }
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    const int64_t to = B.k0 * A.Hkv * D + (int64_t)kv * D;
    store_rows<T, D>(dk + to, (int64_t)A.Hkv * D, B.first, B.lk, ty, tx, ak, one);
    store_rows<T, D>(dv + to, (int64_t)A.Hkv * D, B.first, B.lk, ty, tx, av, one);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dq_simt_kernel(AttnDims A, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                    const float* __restrict__ lse, const T* __restrict__ dout, const float* __restrict__ delta,
                    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, T* __restrict__ dq) {
    extern __shared__ float sm[];
    float *qs = sm, *os = qs + kB * kPitch<D>, *ks = os + kB * kPitch<D>, *vs = ks + kB * kPitch<D>;
    float* ds = vs + kB * kPitch<D>;  // [row][key]
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, kB, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, kv = h / A.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + kB, B.lq) + off);
    load_rows<T, D>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq);
    load_rows<T, D>(os, dout + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq);
    float lse2[4], dl[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = B.q0 + min(B.first + ty * 4 + i, B.lq - 1);
        lse2[i] = __ldg(lse + row * A.Hq + h) * kLog2e;
        dl[i] = __ldg(delta + row * A.Hq + h);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    const float cs = A.scale * kLog2e;
    for (int j0 = 0; j0 < end; j0 += kB) {
        __syncthreads();
        load_rows<T, D>(ks, k + B.k0 * A.sk + (int64_t)kv * D, A.sk, j0, end);
        load_rows<T, D>(vs, v + B.k0 * A.sv + (int64_t)kv * D, A.sv, j0, end);
        __syncthreads();
        float s[4][4], dp[4][4];
        scores<D>(qs, ks, ty, tx, s);
        scores<D>(os, vs, ty, tx, dp);
        tile_grad(s, dp, lse2, dl, cs, A.scale, B.first, j0, ty, tx, off, B.lq, B.lk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ds[(ty * 4 + i) * (kB + 4) + tx + 16 * j] = dp[i][j];
        __syncthreads();
        if (j0 + kB > B.first + off) add_rows<D, true>(ds, ks, ty, tx, acc);
        else add_rows<D, false>(ds, ks, ty, tx, acc);
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    store_rows<T, D>(dq + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, ty, tx, acc, one);
}

template <int D> constexpr size_t fwd_smem() { return (3 * kB * kPitch<D> + kB * (kB + 4)) * sizeof(float); }
template <int D> constexpr size_t dq_smem() { return (4 * kB * kPitch<D> + kB * (kB + 4)) * sizeof(float); }
template <int D> constexpr size_t dkdv_smem() { return (4 * kB * kPitch<D> + 2 * kB * (kB + 4)) * sizeof(float); }

template <class K>
cudaError_t allow_smem(DeviceCache& cache, K kernel, size_t bytes) {
    return device_cached(cache, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    });
}

template <typename T, int D>
cudaError_t forward(const AttnDims& A, const T* q, const T* k, const T* v, const int32_t* cu_q, const int32_t* cu_k,
                    T* out, float* lse, int32_t* err, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_fwd_simt_kernel<T, D>, fwd_smem<D>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.total_q / kB + A.n_seqs), (unsigned)A.Hq);
    attn_fwd_simt_kernel<T, D><<<grid, kThreads, fwd_smem<D>(), st>>>(A, q, k, v, cu_q, cu_k, out, lse, err);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t backward(const AttnDims& A, const T* q, const T* k, const T* v, const T* out, const float* lse,
                     const T* dout, const int32_t* cu_q, const int32_t* cu_k, T* dq, T* dk, T* dv, float* delta,
                     int32_t* err, cudaStream_t st) {
    static DeviceCache c1, c2;
    cudaError_t e = allow_smem(c1, attn_dkdv_simt_kernel<T, D>, dkdv_smem<D>());
    if (e == cudaSuccess) e = allow_smem(c2, attn_dq_simt_kernel<T, D>, dq_smem<D>());
    if (e != cudaSuccess) return e;
    const int64_t rows = A.total_q * A.Hq;
    if (rows > 0) attn_delta_kernel<T, D><<<(unsigned)((rows + 7) / 8), kThreads, 0, st>>>(rows, out, dout, delta);
    if (A.total_k > 0)
        attn_dkdv_simt_kernel<T, D><<<dim3((unsigned)(A.total_k / kB + A.n_seqs), (unsigned)A.Hkv), kThreads,
                                      dkdv_smem<D>(), st>>>(A, q, k, v, lse, dout, delta, cu_q, cu_k, dk, dv, err);
    if (rows > 0)
        attn_dq_simt_kernel<T, D><<<dim3((unsigned)(A.total_q / kB + A.n_seqs), (unsigned)A.Hq), kThreads,
                                    dq_smem<D>(), st>>>(A, q, k, v, lse, dout, delta, cu_q, cu_k, dq);
    return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_attention_simt(const AttnDims& A, const T* q, const T* k, const T* v, const int32_t* cu_q,
                                  const int32_t* cu_k, T* out, float* lse, int32_t* err, cudaStream_t st) {
    if (A.total_q <= 0) return cudaSuccess;
    return A.d == 128 ? forward<T, 128>(A, q, k, v, cu_q, cu_k, out, lse, err, st)
                      : forward<T, 64>(A, q, k, v, cu_q, cu_k, out, lse, err, st);
}
template <typename T>
cudaError_t launch_attention_backward_simt(const AttnDims& A, const T* q, const T* k, const T* v, const T* out,
                                           const float* lse, const T* dout, const int32_t* cu_q,
                                           const int32_t* cu_k, T* dq, T* dk, T* dv, float* delta, int32_t* err,
                                           cudaStream_t st) {
    return A.d == 128 ? backward<T, 128>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, delta, err, st)
                      : backward<T, 64>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, delta, err, st);
}
#define HLA_INST(T)                                                                                                 \
    template cudaError_t launch_attention_simt<T>(const AttnDims&, const T*, const T*, const T*, const int32_t*,    \
                                                  const int32_t*, T*, float*, int32_t*, cudaStream_t);              \
    template cudaError_t launch_attention_backward_simt<T>(const AttnDims&, const T*, const T*, const T*, const T*, \
                                                           const float*, const T*, const int32_t*, const int32_t*,  \
                                                           T*, T*, T*, float*, int32_t*, cudaStream_t);
HLA_INST(float)
HLA_INST(__nv_bfloat16)
#undef HLA_INST

}  // namespace hla
