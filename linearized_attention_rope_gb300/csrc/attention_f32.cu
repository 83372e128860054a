// Packed causal attention and its gradient of fp32 layers, on the CUDA cores:
// the tensor cores do not form these products exactly.
//
// Forward: blocks of 64 or 32 query rows of a head walk 64-key tiles with the
// running maximum and sum; a thread holds 4 x 4 scores.  Gradient: the
// probabilities are recomputed from lse; one kernel per key block and query
// head sums dk and dv over the query tiles (over the heads of a group in a
// second step, in order), another per query block sums dq: 7 products in place
// of the 5 that a single pass with atomics would take, for results that do not
// depend on the order of arrival.
//
// Both operands of a product lie in shared memory, rows padded by 16 bytes so
// that 16 consecutive rows are read without bank conflicts; the next tile is
// copied (cp.async) while this one is worked on, where shared memory allows two
// (head dim 64, and the forward pass).  Bound by the fp32 FMA rate and
// shared-memory reads (two 16-byte reads per 4 x 4 x 4 FMAs); short sequences by
// the length of the walk, hence the blocks of 32 where 64 would leave SMs idle.
// 4096 tokens, 8/2 heads of 128: forward 1150 us (30 TFLOP/s of the 80 the FMAs
// could do), gradient 3853 us (31 of the 7 products done); 813 tokens, 4/2 heads
// of 64: 31 and 91 us.
#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kB = 64;  // keys of a forward tile, rows of a gradient tile
constexpr int kThreads = 256;

template <int D> constexpr int kPitch = D + 4;
constexpr int kPPitch = kB + 4;

__device__ __forceinline__ void copy_wait(int left) {
    if (left) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Rows [first, first + N) of a head to shared memory, asynchronously; rows at or past n are zeros.
template <int D, int N>
__device__ __forceinline__ void copy_rows(float* dst, const float* __restrict__ src, int64_t stride, int first, int n) {
    for (int i = threadIdx.x; i < N * (D / 4); i += blockDim.x) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const bool in = first + r < n;
        const float* from = src + (in ? (int64_t)(first + r) * stride : 0) + c;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * kPitch<D> + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
}

// s[i][j] = a row (ty MI + i) . b row (tx + 16 j)
template <int D, int MI, int NJ>
__device__ __forceinline__ void scores(const float* a, const float* b, int ty, int tx, float (&s)[MI][NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[MI], y[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * MI + i) * kPitch<D> + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * kPitch<D> + c);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}

// acc[i][c] += sum_k p[row ty MI + i][k] b[k][column], columns tx 4 + (64 c / 4), over 64 k.  skip: terms with p = 0 are
// left out, for tiles in which some rows must not see what some of b's rows hold (0 times infinity).
template <int D, int MI, bool SKIP>
__device__ __forceinline__ void add_rows(const float* p, const float* b, int ty, int tx, float (&acc)[MI][D / 16]) {
#pragma unroll 2
    for (int k = 0; k < kB; k += 4) {
        float w[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(p + (ty * MI + i) * kPPitch + k);
            w[i][0] = x.x; w[i][1] = x.y; w[i][2] = x.z; w[i][3] = x.w;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 y = *reinterpret_cast<const float4*>(b + (k + kk) * kPitch<D> + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    if (SKIP && w[i][kk] == 0.f) continue;
                    acc[i][4 * c + 0] = fmaf(w[i][kk], y.x, acc[i][4 * c + 0]);
                    acc[i][4 * c + 1] = fmaf(w[i][kk], y.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(w[i][kk], y.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(w[i][kk], y.w, acc[i][4 * c + 3]);
                }
            }
    }
}
template <int D, int MI>
__device__ __forceinline__ void add_rows(const float* p, const float* b, int ty, int tx, float (&acc)[MI][D / 16],
                                         bool skip) {
    if (skip) add_rows<D, MI, true>(p, b, ty, tx, acc);
    else add_rows<D, MI, false>(p, b, ty, tx, acc);
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

template <int D, int MI>
__device__ __forceinline__ void store_rows(float* __restrict__ dst, int64_t stride, int first, int n, int ty, int tx,
                                           const float (&acc)[MI][D / 16], const float* mul) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if (first + ty * MI + i >= n) continue;
        float* row = dst + (int64_t)(first + ty * MI + i) * stride + tx * 4;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<float4*>(row + 64 * c) = make_float4(acc[i][4 * c] * mul[i], acc[i][4 * c + 1] * mul[i],
                                                                   acc[i][4 * c + 2] * mul[i], acc[i][4 * c + 3] * mul[i]);
    }
}

// BM rows per block, 4 BM threads.
template <int D, int BM>
__global__ void __launch_bounds__(BM * 4)
attn_fwd_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ out,
                    float* __restrict__ lse, int32_t* __restrict__ err) {
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *kv = qs + BM * kPitch<D>, *ps = kv + 4 * kB * kPitch<D>;  // two stages of K and V
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BM, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + BM, B.lq) + off);  // keys some row sees: [0, end)
    const float *kb = k + B.k0 * A.sk + (int64_t)hk * D, *vb = v + B.k0 * A.sv + (int64_t)hk * D;
    auto load = [&](int stage, int j0) {  // keys that no row of the block sees are zeros: what they hold stays out
        copy_rows<D, kB>(kv + 2 * stage * kB * kPitch<D>, kb, A.sk, j0, end);
        copy_rows<D, kB>(kv + (2 * stage + 1) * kB * kPitch<D>, vb, A.sv, j0, end);
        copy_commit();
    };
    copy_rows<D, BM>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq);
    if (end > 0) load(0, 0);
    const float cs = A.scale * kLog2e;
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = 0, stage = 0; j0 < end; j0 += kB, stage ^= 1) {
        const bool more = j0 + kB < end;
        if (more) load(stage ^ 1, j0 + kB);
        copy_wait(more);
        __syncthreads();
        const float *ks = kv + 2 * stage * kB * kPitch<D>, *vs = ks + kB * kPitch<D>;
        float s[4][4];
        scores<D, 4, 4>(qs, ks, ty, tx, s);
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
                ps[(ty * 4 + i) * kPPitch + tx + 16 * j] = p;
            }
            l[i] = l[i] * corr + sum16(sum);
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= corr;
        }
        __syncwarp();  // a row's weights are written and read by one half of a warp
        add_rows<D, 4>(ps, vs, ty, tx, acc, j0 + kB > B.first + off);
        __syncthreads();
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        inv[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int p = B.first + ty * 4 + i;
        if (tx == 0 && p < B.lq) lse[(B.q0 + p) * A.Hq + h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
    copy_wait(0);
    store_rows<D, 4>(out + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, ty, tx, acc, inv);
}

// delta[row][h] = dout . out; one warp per row and head
template <int D>
__global__ void __launch_bounds__(kThreads)
attn_delta_kernel(int64_t rows, const float* __restrict__ out, const float* __restrict__ dout, float* __restrict__ delta) {
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
// s -> p, dp -> ds (times the scale).  lse and delta of rows ty MI + i.
template <int MI, int NJ>
__device__ __forceinline__ void tile_grad(float (&s)[MI][NJ], float (&dp)[MI][NJ], const float (&lse2)[MI],
                                          const float (&dl)[MI], float cs, float scale, int row0, int key0, int ty,
                                          int tx, int off, int lq, int lk) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int row = row0 + ty * MI + i;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int key = key0 + tx + 16 * j;
            const bool on = row < lq && key < lk && key <= row + off;
            s[i][j] = on ? exp2f(fmaf(s[i][j], cs, -lse2[i])) : 0.f;
            dp[i][j] = on ? s[i][j] * (dp[i][j] - dl[i]) * scale : 0.f;
        }
    }
}

// BN keys per block of one query head; ST stages of Q and dO.  dk, dv: [total_k][H][D], H heads of which this block
// writes head blockIdx.y.
template <int D, int BN, int ST>
__global__ void __launch_bounds__(kThreads)
attn_dkdv_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                     const float* __restrict__ lse, const float* __restrict__ dout, const float* __restrict__ delta,
                     const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ dk,
                     float* __restrict__ dv, int32_t* __restrict__ err) {
    constexpr int KN = BN / 16;
    extern __shared__ __align__(16) float sm[];
    float *ks = sm, *vs = ks + BN * kPitch<D>, *qo = vs + BN * kPitch<D>;  // ST stages of Q and dO
    float *pt = qo + ST * 2 * kB * kPitch<D>, *dt = pt + BN * kPPitch;     // [key][row]
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BN, blockIdx.x, true);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq;
    const float *qb = q + B.q0 * A.sq + (int64_t)h * D, *ob = dout + B.q0 * A.Hq * D + (int64_t)h * D;
    auto load = [&](int stage, int r0) {
        copy_rows<D, kB>(qo + 2 * stage * kB * kPitch<D>, qb, A.sq, r0, B.lq);
        copy_rows<D, kB>(qo + (2 * stage + 1) * kB * kPitch<D>, ob, (int64_t)A.Hq * D, r0, B.lq);
        copy_commit();
    };
    const int i0 = max(0, B.first - off) / kB * kB;  // first tile of rows that see the block's first key
    copy_rows<D, BN>(ks, k + B.k0 * A.sk + (int64_t)hk * D, A.sk, B.first, B.lk);
    copy_rows<D, BN>(vs, v + B.k0 * A.sv + (int64_t)hk * D, A.sv, B.first, B.lk);
    if (i0 < B.lq) load(0, i0);
    float ak[KN][D / 16], av[KN][D / 16];
#pragma unroll
    for (int i = 0; i < KN; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
    const float cs = A.scale * kLog2e;
    for (int r0 = i0, stage = 0; r0 < B.lq; r0 += kB, stage ^= ST - 1) {
        const bool more = r0 + kB < B.lq;
        if (ST == 2 && more) load(stage ^ 1, r0 + kB);
        float lse2[4], dl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = B.q0 + min(r0 + ty * 4 + i, B.lq - 1);
            lse2[i] = __ldg(lse + row * A.Hq + h) * kLog2e;
            dl[i] = __ldg(delta + row * A.Hq + h);
        }
        copy_wait(ST == 2 && more);
        __syncthreads();
        const float *qs = qo + 2 * stage * kB * kPitch<D>, *os = qs + kB * kPitch<D>;
        float s[4][KN], dp[4][KN];
        scores<D, 4, KN>(qs, ks, ty, tx, s);
        scores<D, 4, KN>(os, vs, ty, tx, dp);
        tile_grad(s, dp, lse2, dl, cs, A.scale, r0, B.first, ty, tx, off, B.lq, B.lk);
#pragma unroll
        for (int j = 0; j < KN; ++j) {
            *reinterpret_cast<float4*>(pt + (tx + 16 * j) * kPPitch + ty * 4) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
            *reinterpret_cast<float4*>(dt + (tx + 16 * j) * kPPitch + ty * 4) = make_float4(dp[0][j], dp[1][j], dp[2][j], dp[3][j]);
        }
        __syncthreads();
        const bool skip = r0 + off < B.first + BN;
        add_rows<D, KN>(pt, os, ty, tx, av, skip);
        add_rows<D, KN>(dt, qs, ty, tx, ak, skip);
        __syncthreads();
        if (ST == 1 && more) load(0, r0 + kB);
    }
    copy_wait(0);
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    const int64_t H = gridDim.y, to = B.k0 * H * D + (int64_t)h * D;
    store_rows<D, KN>(dk + to, H * D, B.first, B.lk, ty, tx, ak, one);
    store_rows<D, KN>(dv + to, H * D, B.first, B.lk, ty, tx, av, one);
}

// dk, dv of a kv head: the sums over its query heads, in order; rows of the sequences only.
template <int D>
__global__ void __launch_bounds__(kThreads)
attn_group_sum_kernel(AttnDims A, const int32_t* __restrict__ cu_k, const float* __restrict__ pk,
                      const float* __restrict__ pv, float* __restrict__ dk, float* __restrict__ dv) {
    const int64_t n = A.total_k * A.Hkv * (D / 4), i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t row = i / (D / 4), t = row / A.Hkv;
    int64_t a, len;
    seq_range(cu_k, seq_of_token(cu_k, A.n_seqs, t), A.total_k, &a, &len);
    if (t < a || t >= a + len) return;
    const float4 *sk = reinterpret_cast<const float4*>(pk) + row * A.G * (D / 4) + i % (D / 4);
    const float4 *sv = reinterpret_cast<const float4*>(pv) + row * A.G * (D / 4) + i % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int g = 0; g < A.G; ++g) {
        const float4 u = sk[g * (D / 4)], w = sv[g * (D / 4)];
        x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
        y = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
    }
    reinterpret_cast<float4*>(dk)[i] = x;
    reinterpret_cast<float4*>(dv)[i] = y;
}

template <int D, int BM, int ST>
__global__ void __launch_bounds__(BM * 4)
attn_dq_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                   const float* __restrict__ lse, const float* __restrict__ dout, const float* __restrict__ delta,
                   const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ dq) {
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *os = qs + BM * kPitch<D>, *kv = os + BM * kPitch<D>;  // ST stages of K and V
    float* ds = kv + ST * 2 * kB * kPitch<D>;                               // [row][key]
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BM, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + BM, B.lq) + off);
    const float *kb = k + B.k0 * A.sk + (int64_t)hk * D, *vb = v + B.k0 * A.sv + (int64_t)hk * D;
    auto load = [&](int stage, int j0) {
        copy_rows<D, kB>(kv + 2 * stage * kB * kPitch<D>, kb, A.sk, j0, end);
        copy_rows<D, kB>(kv + (2 * stage + 1) * kB * kPitch<D>, vb, A.sv, j0, end);
        copy_commit();
    };
    copy_rows<D, BM>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq);
    copy_rows<D, BM>(os, dout + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq);
    if (end > 0) load(0, 0);
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
    for (int j0 = 0, stage = 0; j0 < end; j0 += kB, stage ^= ST - 1) {
        const bool more = j0 + kB < end;
        if (ST == 2 && more) load(stage ^ 1, j0 + kB);
        copy_wait(ST == 2 && more);
        __syncthreads();
        const float *ks = kv + 2 * stage * kB * kPitch<D>, *vs = ks + kB * kPitch<D>;
        float s[4][4], dp[4][4];
        scores<D, 4, 4>(qs, ks, ty, tx, s);
        scores<D, 4, 4>(os, vs, ty, tx, dp);
        tile_grad(s, dp, lse2, dl, cs, A.scale, B.first, j0, ty, tx, off, B.lq, B.lk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ds[(ty * 4 + i) * kPPitch + tx + 16 * j] = dp[i][j];
        __syncwarp();
        add_rows<D, 4>(ds, ks, ty, tx, acc, j0 + kB > B.first + off);
        __syncthreads();
        if (ST == 1 && more) load(0, j0 + kB);
    }
    copy_wait(0);
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    store_rows<D, 4>(dq + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, ty, tx, acc, one);
}

template <int D, int BM> constexpr size_t fwd_smem() { return ((BM + 4 * kB) * kPitch<D> + BM * kPPitch) * sizeof(float); }
template <int D, int BM, int ST> constexpr size_t dq_smem() {
    return ((2 * BM + ST * 2 * kB) * kPitch<D> + BM * kPPitch) * sizeof(float);
}
template <int D, int BN, int ST> constexpr size_t dkdv_smem() {
    return ((2 * BN + ST * 2 * kB) * kPitch<D> + 2 * BN * kPPitch) * sizeof(float);
}

template <class K>
cudaError_t allow_smem(DeviceCache& cache, K kernel, size_t bytes) {
    return device_cached(cache, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    });
}

// Blocks of 32 rows (or keys) where 64 would give fewer than two blocks per SM: half the walk per block for a little
// more traffic (813 tokens, 4 heads, d 64: forward 54 -> 31 us; 1500 tokens, 32 heads, d 128, 768 blocks: 64 is faster).
bool small_blocks(int64_t total, int n_seqs, int heads) { return (total / kB + n_seqs) * heads < 2 * 152; }

template <int D, int BM>
cudaError_t forward(const AttnDims& A, const float* q, const float* k, const float* v, const int32_t* cu_q,
                    const int32_t* cu_k, float* out, float* lse, int32_t* err, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_fwd_f32_kernel<D, BM>, fwd_smem<D, BM>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.total_q / BM + A.n_seqs), (unsigned)A.Hq);
    attn_fwd_f32_kernel<D, BM><<<grid, BM * 4, fwd_smem<D, BM>(), st>>>(A, q, k, v, cu_q, cu_k, out, lse, err);
    return cudaGetLastError();
}

template <int D, int BN>
cudaError_t keys_backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* lse,
                          const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dk, float* dv, float* delta,
                          float* parts, int32_t* err, cudaStream_t st) {
    constexpr int ST = D == 64 ? 2 : 1;
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_dkdv_f32_kernel<D, BN, ST>, dkdv_smem<D, BN, ST>());
    if (e != cudaSuccess) return e;
    float *pk = A.G > 1 ? parts : dk, *pv = A.G > 1 ? parts + A.total_k * A.Hq * D : dv;
    attn_dkdv_f32_kernel<D, BN, ST><<<dim3((unsigned)(A.total_k / BN + A.n_seqs), (unsigned)A.Hq), kThreads,
                                      dkdv_smem<D, BN, ST>(), st>>>(A, q, k, v, lse, dout, delta, cu_q, cu_k, pk, pv, err);
    if (A.G > 1) {
        const int64_t n = A.total_k * A.Hkv * (D / 4);
        attn_group_sum_kernel<D><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(A, cu_k, pk, pv, dk, dv);
    }
    return cudaGetLastError();
}

template <int D, int BM>
cudaError_t rows_backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* lse,
                          const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dq, float* delta,
                          cudaStream_t st) {
    constexpr int ST = D == 64 ? 2 : 1;
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_dq_f32_kernel<D, BM, ST>, dq_smem<D, BM, ST>());
    if (e != cudaSuccess) return e;
    attn_dq_f32_kernel<D, BM, ST><<<dim3((unsigned)(A.total_q / BM + A.n_seqs), (unsigned)A.Hq), BM * 4,
                                    dq_smem<D, BM, ST>(), st>>>(A, q, k, v, lse, dout, delta, cu_q, cu_k, dq);
    return cudaGetLastError();
}

template <int D>
cudaError_t backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* out,
                     const float* lse, const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dq, float* dk,
                     float* dv, float* ws, int32_t* err, cudaStream_t st) {
    const int64_t rows = A.total_q * A.Hq;
    float *delta = ws, *parts = ws + (rows + 63) / 64 * 64;
    cudaError_t e = cudaSuccess;
    if (rows > 0) attn_delta_kernel<D><<<(unsigned)((rows + 7) / 8), kThreads, 0, st>>>(rows, out, dout, delta);
    if (A.total_k > 0)
        e = small_blocks(A.total_k, A.n_seqs, A.Hq)
                ? keys_backward<D, 32>(A, q, k, v, lse, dout, cu_q, cu_k, dk, dv, delta, parts, err, st)
                : keys_backward<D, 64>(A, q, k, v, lse, dout, cu_q, cu_k, dk, dv, delta, parts, err, st);
    if (e != cudaSuccess || rows == 0) return e;
    return small_blocks(A.total_q, A.n_seqs, A.Hq)
               ? rows_backward<D, 32>(A, q, k, v, lse, dout, cu_q, cu_k, dq, delta, st)
               : rows_backward<D, 64>(A, q, k, v, lse, dout, cu_q, cu_k, dq, delta, st);
}

// Rows of the sequences set to zero (and lse to -infinity): what attention and its gradient are without keys or queries.
template <typename T>
__global__ void __launch_bounds__(kThreads)
attn_empty_kernel(int64_t total, int64_t other, int n_seqs, const int32_t* __restrict__ cu,
                  const int32_t* __restrict__ cu_other, int heads, int d, T* x, T* y, float* lse, int32_t* err) {
    if (blockIdx.x == 0) {
        attn_check_table(cu, n_seqs, total, err);
        attn_check_table(cu_other, n_seqs, other, err);
    }
    const int64_t per = (int64_t)heads * d, n = total * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / per;
        int64_t a, len;
        seq_range(cu, seq_of_token(cu, n_seqs, t), total, &a, &len);
        if (t < a || t >= a + len) continue;
        x[i] = from_f32<T>(0.f);
        if (y) y[i] = from_f32<T>(0.f);
        if (lse && i % d == 0) lse[i / d] = -INFINITY;
    }
}

}  // namespace

cudaError_t launch_attention_f32(const AttnDims& A, const float* q, const float* k, const float* v, const int32_t* cu_q,
                                 const int32_t* cu_k, float* out, float* lse, int32_t* err, cudaStream_t st) {
    const bool small = small_blocks(A.total_q, A.n_seqs, A.Hq);
    if (A.d == 128)
        return small ? forward<128, 32>(A, q, k, v, cu_q, cu_k, out, lse, err, st)
                     : forward<128, 64>(A, q, k, v, cu_q, cu_k, out, lse, err, st);
    return small ? forward<64, 32>(A, q, k, v, cu_q, cu_k, out, lse, err, st)
                 : forward<64, 64>(A, q, k, v, cu_q, cu_k, out, lse, err, st);
}
size_t attention_backward_f32_floats(const AttnDims& A) {
    return (size_t)((A.total_q * A.Hq + 63) / 64 * 64 + (A.G > 1 ? 2 * A.total_k * A.Hq * A.d : 0));
}
cudaError_t launch_attention_backward_f32(const AttnDims& A, const float* q, const float* k, const float* v,
                                          const float* out, const float* lse, const float* dout, const int32_t* cu_q,
                                          const int32_t* cu_k, float* dq, float* dk, float* dv, float* ws, int32_t* err,
                                          cudaStream_t st) {
    return A.d == 128 ? backward<128>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, err, st)
                      : backward<64>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, err, st);
}

template <typename T>
cudaError_t launch_attention_empty(int64_t total, int64_t other, int n_seqs, const int32_t* cu, const int32_t* cu_other,
                                   int heads, int d, T* x, T* y, float* lse, int32_t* err, cudaStream_t st) {
    if (total <= 0) return cudaSuccess;
    const int64_t n = total * heads * d;
    attn_empty_kernel<T><<<(unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 4096), kThreads, 0, st>>>(
        total, other, n_seqs, cu, cu_other, heads, d, x, y, lse, err);
    return cudaGetLastError();
}
template cudaError_t launch_attention_empty<float>(int64_t, int64_t, int, const int32_t*, const int32_t*, int, int, float*,
                                                   float*, float*, int32_t*, cudaStream_t);
template cudaError_t launch_attention_empty<__nv_bfloat16>(int64_t, int64_t, int, const int32_t*, const int32_t*, int, int,
                                                           __nv_bfloat16*, __nv_bfloat16*, float*, int32_t*,
                                                           cudaStream_t);

}  // namespace hla
