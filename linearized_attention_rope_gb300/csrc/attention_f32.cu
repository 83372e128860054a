// Packed causal attention and its gradient of fp32 layers, on the CUDA cores:
// the tensor cores do not form these products exactly.  (Operands split into
// three bf16 parts, six products, were not tried.)
//
// Forward: blocks of 64, 32 or 16 query rows of a head walk 64-key tiles with the
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
// (head dim 64, and the forward pass).  A block of 32 or 16 has one warp per
// scheduler or less per group of threads, which waits for every load; so 4 groups
// (2 at head dim 128) take the tiles in turn and add their sums at the end, in
// order.
//
// Bound by shared-memory reads: eight of 16 bytes per 64 FMAs, at a quarter of a
// warp a cycle, which the 4 x 4 scores of a thread set (larger ones would need fewer).  4096 tokens, 8/2 heads of 128: forward 1141 us (30 TFLOP/s of
// the 80 the FMAs could do), gradient 3904 us (31 with the 7 products it forms);
// 813 tokens, 4/2 heads of 64, where the walk of one block is what takes the
// time: 24 and 63 us (blocks of 32 and one group: 31 and 91).
#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kB = 64;  // keys of a forward tile, rows of a gradient tile
constexpr int kThreads = 256;
constexpr int kPartTiles = 8;  // key tiles of a part, at least
template <int D> constexpr int kSmallGroups = D == 64 ? 4 : 2;  // groups of a smaller block: what shared memory holds

template <int D> constexpr int kPitch = D + 4;
constexpr int kPPitch = kB + 4;

__device__ __forceinline__ void copy_wait(int left) {
    if (left) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits for the T threads of group g.
template <int T> __device__ __forceinline__ void group_sync(int g) {
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(T) : "memory");
}

// Rows [first, first + N) of a head to shared memory, asynchronously, by T threads; rows at or past n are zeros.
template <int D, int N, int T>
__device__ __forceinline__ void copy_rows(float* dst, const float* __restrict__ src, int64_t stride, int first, int n,
                                          int tid) {
    for (int i = tid; i < N * (D / 4); i += T) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const bool in = first + r < n;
        const float* from = src + (in ? (int64_t)(first + r) * stride : 0) + c;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * kPitch<D> + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
}

// s[i][j] = a row (ty 4 + i) . b row (tx + NX j)
template <int D, int NX>
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
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + NX * j) * kPitch<D> + c);
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

// acc[i][4 c + e] += sum_k p[row ty MI + i][k] b[k][column 64 c + 4 tx + e], over 64 k.  skip: terms with p = 0 are left
// out, for tiles in which some rows must not see what some of b's rows hold (0 times infinity).
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

// Sums of the W groups' values, in order, in group 0; buf is free.
template <int W, int T, int N>
__device__ __forceinline__ void group_sums(float* buf, int g, int tid, float (&x)[N]) {
    if (W == 1) return;
    if (g > 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[((g - 1) * N + i) * T + tid] = x[i];
    __syncthreads();
    if (g == 0)
#pragma unroll
        for (int o = 0; o < W - 1; ++o)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += buf[(o * N + i) * T + tid];
    __syncthreads();
}

// Parts of a block's n key tiles: at least kPartTiles in each.
__device__ __forceinline__ int parts_of(int n, int parts) { return max(1, min(parts, n / kPartTiles)); }

// BM rows per block, W groups of 4 BM threads that take the key tiles in turn, ST stages of K and V each.  parts > 1:
// block z takes a part of whole tiles (those past the row's parts none) and leaves its results in out and lse, [parts][...].
template <int D, int BM, int W, int ST>
__global__ void __launch_bounds__(BM * 4 * W)
attn_fwd_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ out,
                    float* __restrict__ lse, int parts, int32_t* __restrict__ err) {
    extern __shared__ __align__(16) float sm[];
    constexpr int T = BM * 4, kGroup = ST * 2 * kB * kPitch<D> + BM * kPPitch;
    const int g = threadIdx.x / T, tid = threadIdx.x % T, ty = tid >> 4, tx = tid & 15;
    float *qs = sm, *kv = qs + BM * kPitch<D> + g * kGroup, *ps = kv + ST * 2 * kB * kPitch<D>;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BM, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + BM, B.lq) + off);  // keys some row sees: [0, end)
    int t0 = 0, t1 = (max(0, end) + kB - 1) / kB;                                 // this block's key tiles
    if (parts > 1) {
        const int n = t1, cut = parts_of(n, parts), z = blockIdx.z;
        t0 = z < cut ? n * z / cut : n;
        t1 = z < cut ? n * (z + 1) / cut : n;
        out += z * A.total_q * A.Hq * D;
        lse += z * A.total_q * A.Hq;
        if (t0 >= t1) {  // no tiles: the join looks at lse only
            const int p = B.first + (int)threadIdx.x;
            if ((int)threadIdx.x < BM && p < B.lq) lse[(B.q0 + p) * A.Hq + h] = -INFINITY;
            return;
        }
    }
    const float *kb = k + B.k0 * A.sk + (int64_t)hk * D, *vb = v + B.k0 * A.sv + (int64_t)hk * D;
    auto load = [&](int stage, int j0) {  // keys that no row of the block sees are zeros: what they hold stays out
        copy_rows<D, kB, T>(kv + 2 * stage * kB * kPitch<D>, kb, A.sk, j0, end, tid);
        copy_rows<D, kB, T>(kv + (2 * stage + 1) * kB * kPitch<D>, vb, A.sv, j0, end, tid);
        copy_commit();
    };
    copy_rows<D, BM, T * W>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq, threadIdx.x);
    copy_commit();
    load(0, (t0 + g) * kB);
    copy_wait(1);
    if (W > 1) __syncthreads();  // the query rows are every group's
    const float cs = A.scale * kLog2e;
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = (t0 + g) * kB, stage = 0; j0 < t1 * kB; j0 += W * kB, stage ^= ST - 1) {
        const bool more = j0 + W * kB < t1 * kB;
        if (ST == 2 && more) load(stage ^ 1, j0 + W * kB);
        copy_wait(ST == 2 && more);
        group_sync<T>(g);
        const float *ks = kv + 2 * stage * kB * kPitch<D>, *vs = ks + kB * kPitch<D>;
        float s[4][4];
        scores<D, 16>(qs, ks, ty, tx, s);
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
        group_sync<T>(g);
        if (ST == 1 && more) load(0, j0 + W * kB);
    }
    copy_wait(0);
    if (W > 1) {  // the groups' references made one, then their sums
        __syncthreads();
        float* ms = sm;
        if (tx == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) ms[g * BM + ty * 4 + i] = m[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mn = ms[ty * 4 + i];
#pragma unroll
            for (int o = 1; o < W; ++o) mn = fmaxf(mn, ms[o * BM + ty * 4 + i]);
            const float corr = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
            m[i] = mn;
            l[i] *= corr;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] *= corr;
        }
        group_sums<W, T>(sm + W * BM, g, tid, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) group_sums<W, T>(sm + W * BM, g, tid, acc[i]);
        if (g > 0) return;
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        inv[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int p = B.first + ty * 4 + i;
        if (tx == 0 && p < B.lq) lse[(B.q0 + p) * A.Hq + h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
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
// s -> p, dp -> ds (times the scale).  lse and delta of rows ty 4 + i, keys tx + NX j.
template <int NX>
__device__ __forceinline__ void tile_grad(float (&s)[4][4], float (&dp)[4][4], const float (&lse2)[4],
                                          const float (&dl)[4], float cs, float scale, int row0, int key0, int ty, int tx,
                                          int off, int lq, int lk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = row0 + ty * 4 + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = key0 + tx + NX * j;
            const bool on = row < lq && key < lk && key <= row + off;
            s[i][j] = on ? exp2f(fmaf(s[i][j], cs, -lse2[i])) : 0.f;
            dp[i][j] = on ? s[i][j] * (dp[i][j] - dl[i]) * scale : 0.f;
        }
    }
}

// BN keys per block of one query head; W groups take the query tiles in turn, ST stages of Q and dO each.  dk, dv:
// [total_k][H][D], H heads of which this block writes head blockIdx.y.
template <int D, int BN, int W, int ST>
__global__ void __launch_bounds__(BN * 4 * W)
attn_dkdv_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                     const float* __restrict__ lse, const float* __restrict__ dout, const float* __restrict__ delta,
                     const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ dk,
                     float* __restrict__ dv, int32_t* __restrict__ err) {
    constexpr int T = BN * 4, NX = BN / 4, kGroup = ST * 2 * kB * kPitch<D> + 2 * BN * kPPitch;
    extern __shared__ __align__(16) float sm[];
    const int g = threadIdx.x / T, tid = threadIdx.x % T, ty = tid >> 4, tx = tid & 15;  // of the gradients
    const int sy = tid / NX, sx = tid % NX;                                                // of the scores
    float *ks = sm, *vs = ks + BN * kPitch<D>, *qo = vs + BN * kPitch<D> + g * kGroup;
    float *pt = qo + ST * 2 * kB * kPitch<D>, *dt = pt + BN * kPPitch;  // [key][row]
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BN, blockIdx.x, true);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G, off = B.lk - B.lq;
    const float *qb = q + B.q0 * A.sq + (int64_t)h * D, *ob = dout + B.q0 * A.Hq * D + (int64_t)h * D;
    auto load = [&](int stage, int r0) {
        copy_rows<D, kB, T>(qo + 2 * stage * kB * kPitch<D>, qb, A.sq, r0, B.lq, tid);
        copy_rows<D, kB, T>(qo + (2 * stage + 1) * kB * kPitch<D>, ob, (int64_t)A.Hq * D, r0, B.lq, tid);
        copy_commit();
    };
    const int i0 = max(0, B.first - off) / kB * kB;  // first tile of rows that see the block's first key
    copy_rows<D, BN, T * W>(ks, k + B.k0 * A.sk + (int64_t)hk * D, A.sk, B.first, B.lk, threadIdx.x);
    copy_rows<D, BN, T * W>(vs, v + B.k0 * A.sv + (int64_t)hk * D, A.sv, B.first, B.lk, threadIdx.x);
    copy_commit();
    load(0, i0 + g * kB);
    copy_wait(1);
    if (W > 1) __syncthreads();
    float ak[4][D / 16], av[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
    const float cs = A.scale * kLog2e;
    for (int r0 = i0 + g * kB, stage = 0; r0 < B.lq; r0 += W * kB, stage ^= ST - 1) {
        const bool more = r0 + W * kB < B.lq;
        if (ST == 2 && more) load(stage ^ 1, r0 + W * kB);
        float lse2[4], dl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = B.q0 + min(r0 + sy * 4 + i, B.lq - 1);
            lse2[i] = __ldg(lse + row * A.Hq + h) * kLog2e;
            dl[i] = __ldg(delta + row * A.Hq + h);
        }
        copy_wait(ST == 2 && more);
        group_sync<T>(g);
        const float *qs = qo + 2 * stage * kB * kPitch<D>, *os = qs + kB * kPitch<D>;
        float s[4][4], dp[4][4];
        scores<D, NX>(qs, ks, sy, sx, s);
        scores<D, NX>(os, vs, sy, sx, dp);
        tile_grad<NX>(s, dp, lse2, dl, cs, A.scale, r0, B.first, sy, sx, off, B.lq, B.lk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float4*>(pt + (sx + NX * j) * kPPitch + sy * 4) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
            *reinterpret_cast<float4*>(dt + (sx + NX * j) * kPPitch + sy * 4) = make_float4(dp[0][j], dp[1][j], dp[2][j], dp[3][j]);
        }
        group_sync<T>(g);
        const bool skip = r0 + off < B.first + BN;
        add_rows<D, 4>(pt, os, ty, tx, av, skip);
        add_rows<D, 4>(dt, qs, ty, tx, ak, skip);
        group_sync<T>(g);
        if (ST == 1 && more) load(0, r0 + W * kB);
    }
    copy_wait(0);
    if (W > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            group_sums<W, T>(sm, g, tid, ak[i]);
            group_sums<W, T>(sm, g, tid, av[i]);
        }
        if (g > 0) return;
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    const int64_t H = gridDim.y, to = B.k0 * H * D + (int64_t)h * D;
    store_rows<D, 4>(dk + to, H * D, B.first, B.lk, ty, tx, ak, one);
    store_rows<D, 4>(dv + to, H * D, B.first, B.lk, ty, tx, av, one);
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

template <int D, int BM, int W, int ST>
__global__ void __launch_bounds__(BM * 4 * W)
attn_dq_f32_kernel(AttnDims A, const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                   const float* __restrict__ lse, const float* __restrict__ dout, const float* __restrict__ delta,
                   const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, float* __restrict__ dq, int parts) {
    extern __shared__ __align__(16) float sm[];
    constexpr int T = BM * 4, kGroup = ST * 2 * kB * kPitch<D> + BM * kPPitch;
    const int g = threadIdx.x / T, tid = threadIdx.x % T, ty = tid >> 4, tx = tid & 15;
    float *qs = sm, *os = qs + BM * kPitch<D>, *kv = os + BM * kPitch<D> + g * kGroup;
    float* ds = kv + ST * 2 * kB * kPitch<D>;  // [row][key]
    const AttnBlock B = attn_find_block(A, cu_q, cu_k, BM, blockIdx.x, false);
    if (!B.found) return;
    const int h = blockIdx.y, hk = h / A.G;
    const int off = B.lk - B.lq, end = min(B.lk, min(B.first + BM, B.lq) + off);
    int t0 = 0, t1 = (max(0, end) + kB - 1) / kB;  // this block's key tiles
    if (parts > 1) {                               // (the sum takes as many parts of the row's as have tiles)
        const int n = t1, cut = parts_of(n, parts), z = blockIdx.z;
        if (z >= cut) return;
        t0 = n * z / cut;
        t1 = n * (z + 1) / cut;
        dq += z * A.total_q * A.Hq * D;
    }
    const float *kb = k + B.k0 * A.sk + (int64_t)hk * D, *vb = v + B.k0 * A.sv + (int64_t)hk * D;
    auto load = [&](int stage, int j0) {
        copy_rows<D, kB, T>(kv + 2 * stage * kB * kPitch<D>, kb, A.sk, j0, end, tid);
        copy_rows<D, kB, T>(kv + (2 * stage + 1) * kB * kPitch<D>, vb, A.sv, j0, end, tid);
        copy_commit();
    };
    copy_rows<D, BM, T * W>(qs, q + B.q0 * A.sq + (int64_t)h * D, A.sq, B.first, B.lq, threadIdx.x);
    copy_rows<D, BM, T * W>(os, dout + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, threadIdx.x);
    copy_commit();
    load(0, (t0 + g) * kB);
    copy_wait(1);
    if (W > 1) __syncthreads();
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
    for (int j0 = (t0 + g) * kB, stage = 0; j0 < t1 * kB; j0 += W * kB, stage ^= ST - 1) {
        const bool more = j0 + W * kB < t1 * kB;
        if (ST == 2 && more) load(stage ^ 1, j0 + W * kB);
        copy_wait(ST == 2 && more);
        group_sync<T>(g);
        const float *ks = kv + 2 * stage * kB * kPitch<D>, *vs = ks + kB * kPitch<D>;
        float s[4][4], dp[4][4];
        scores<D, 16>(qs, ks, ty, tx, s);
        scores<D, 16>(os, vs, ty, tx, dp);
        tile_grad<16>(s, dp, lse2, dl, cs, A.scale, B.first, j0, ty, tx, off, B.lq, B.lk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ds[(ty * 4 + i) * kPPitch + tx + 16 * j] = dp[i][j];
        __syncwarp();
        add_rows<D, 4>(ds, ks, ty, tx, acc, j0 + kB > B.first + off);
        group_sync<T>(g);
        if (ST == 1 && more) load(0, j0 + W * kB);
    }
    copy_wait(0);
    if (W > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) group_sums<W, T>(sm, g, tid, acc[i]);
        if (g > 0) return;
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    store_rows<D, 4>(dq + B.q0 * A.Hq * D + (int64_t)h * D, (int64_t)A.Hq * D, B.first, B.lq, ty, tx, acc, one);
}

// dq of the sequences' rows from the parts of their blocks of BM rows, in order.
template <int D>
__global__ void __launch_bounds__(kThreads)
attn_dq_sum_kernel(AttnDims A, const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int bm, int parts,
                   const float* __restrict__ part, float* __restrict__ dq) {
    const int64_t per = (int64_t)A.Hq * (D / 4), n = A.total_q * per, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / per;
    const int s = seq_of_token(cu_q, A.n_seqs, t);
    int64_t a, lq, b, lk;
    seq_range(cu_q, s, A.total_q, &a, &lq);
    seq_range(cu_k, s, A.total_k, &b, &lk);
    if (t < a || t >= a + lq) return;
    const int64_t rows = min((t - a) / bm * bm + bm, lq), end = min(lk, rows + lk - lq);
    const int cut = parts_of((int)((max((int64_t)0, end) + kB - 1) / kB), parts);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < cut; ++z) {
        const float4 u = reinterpret_cast<const float4*>(part)[z * n + i];
        x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
    }
    reinterpret_cast<float4*>(dq)[i] = x;
}

template <int D, int BM, int W, int ST> constexpr size_t fwd_smem() {
    return (BM * kPitch<D> + W * (ST * 2 * kB * kPitch<D> + BM * kPPitch)) * sizeof(float);
}
template <int D, int BM, int W, int ST> constexpr size_t dq_smem() {
    return (2 * BM * kPitch<D> + W * (ST * 2 * kB * kPitch<D> + BM * kPPitch)) * sizeof(float);
}
template <int D, int BN, int W, int ST> constexpr size_t dkdv_smem() {
    return (2 * BN * kPitch<D> + W * (ST * 2 * kB * kPitch<D> + 2 * BN * kPPitch)) * sizeof(float);
}

template <class K>
cudaError_t allow_smem(DeviceCache& cache, K kernel, size_t bytes) {
    return device_cached(cache, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    });
}

// Rows (or keys) of a block.  64 unless that gives fewer than two blocks per SM, then 32 (half the walk per block, by
// several groups of threads, for a little more traffic), then, below `least` blocks, 16: half as many blocks as SMs
// for the forward pass, as many for the gradient.  Forward and gradient, in us:
//   1500 tokens, 32/8 heads of 128:     642 and 2147 with 64, 698 and 2692 with 32 (blocks of 64: 768)
//   226 tokens in 2, 32/8 heads of 128:  26 and 75 with 32, 36 and 98 with 16 (blocks of 32: 288)
//   813 tokens in 2, 4/2 heads of 64:    24 and 70 with 32, 25 and 63 with 16 (108)
//   1000 tokens, 2/1 heads of 128:       76 and 237 with 32, 53 and 158 with 16 (64)
int block_rows(int64_t total, int n_seqs, int heads, int least) {
    if ((total / 64 + n_seqs) * heads >= 2 * 152) return 64;
    return (total / 32 + n_seqs) * heads >= least ? 32 : 16;
}

// Parts that the keys of few rows (chunks behind earlier keys) are cut into at most, a block each, joined in order: one
// for every kPartTiles tiles that a single sequence could have, where the blocks would not fill the SMs twice.  How the keys
// are spread over the sequences is known on the device only: equal lengths lose a little by it, unequal ones gain much.  Forward:
// 186 rows in 5, one of them 31 behind 3506 keys, 8/4 heads of 128, 250 -> 58 us; 64 rows behind 8128, 32/8 of 128, 567 ->
// 289; one row of 3000, one head of 64, 77 -> 23; 5 x 100 behind 900, 4/2 of 64, 42 -> 43; 4 x 1 behind 2000, 32/8 of 128,
// 145 -> 158.  Gradient (dq): 327 -> 158, 1109 -> 1081, 107 -> 46, 98 -> 110, 689 -> 700.
int row_parts(const AttnDims& A) {
    const int64_t blocks = (A.total_q / 32 + A.n_seqs) * A.Hq;
    if (4 * A.total_q > A.total_k || blocks >= 2 * 152) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(32, A.total_k / (kPartTiles * kB)));
}

size_t part_bytes(const AttnDims& A, int64_t parts) {  // of the forward pass
    const int64_t rows = A.total_q * A.Hq;
    return parts > 1 ? (size_t)((parts * rows + 3) / 4 * 4 + parts * rows * A.d) * sizeof(float) : 0;
}
size_t backward_floats(const AttnDims& A, int64_t parts) {
    const int64_t rows = A.total_q * A.Hq;
    return (size_t)((rows + 63) / 64 * 64 + (A.G > 1 ? 2 * A.total_k * A.Hq * A.d : 0) + (parts > 1 ? parts * rows * A.d : 0));
}

template <int D, int BM, int W, int ST>
cudaError_t rows_forward(const AttnDims& A, const float* q, const float* k, const float* v, const int32_t* cu_q,
                         const int32_t* cu_k, float* out, float* lse, int parts, int32_t* err, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_fwd_f32_kernel<D, BM, W, ST>, fwd_smem<D, BM, W, ST>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.total_q / BM + A.n_seqs), (unsigned)A.Hq, (unsigned)parts);
    attn_fwd_f32_kernel<D, BM, W, ST><<<grid, BM * 4 * W, fwd_smem<D, BM, W, ST>(), st>>>(A, q, k, v, cu_q, cu_k, out, lse, parts,
                                                                                        err);
    return cudaGetLastError();
}

template <int D>
cudaError_t forward(const AttnDims& A, const float* q, const float* k, const float* v, const int32_t* cu_q,
                    const int32_t* cu_k, float* out, float* lse, float* part_ws, size_t room, int32_t* err,
                    cudaStream_t st) {
    const int qb = block_rows(A.total_q, A.n_seqs, A.Hq, 76);
    const int parts = parts_within(row_parts(A), room, [&](int p) { return part_bytes(A, p); });
    const int64_t rows = A.total_q * A.Hq;
    float *part_lse = part_ws, *part_o = part_ws + (parts * rows + 3) / 4 * 4;
    const cudaError_t e = (qb == 64   ? rows_forward<D, 64, 1, 2>
                           : qb == 32 ? rows_forward<D, 32, kSmallGroups<D>, 1>
                                      : rows_forward<D, 16, kSmallGroups<D>, 1>)(
        A, q, k, v, cu_q, cu_k, parts > 1 ? part_o : out, parts > 1 ? part_lse : lse, parts, err, st);
    if (e != cudaSuccess || parts == 1) return e;
    attention_join_kernel<D, float><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(A, cu_q, parts, part_o, part_lse, out, lse);
    return cudaGetLastError();
}

template <int D, int BN, int W, int ST>
cudaError_t keys_backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* lse,
                          const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dk, float* dv, float* delta,
                          float* parts, int32_t* err, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_dkdv_f32_kernel<D, BN, W, ST>, dkdv_smem<D, BN, W, ST>());
    if (e != cudaSuccess) return e;
    float *pk = A.G > 1 ? parts : dk, *pv = A.G > 1 ? parts + A.total_k * A.Hq * D : dv;
    attn_dkdv_f32_kernel<D, BN, W, ST><<<dim3((unsigned)(A.total_k / BN + A.n_seqs), (unsigned)A.Hq), BN * 4 * W,
                                      dkdv_smem<D, BN, W, ST>(), st>>>(A, q, k, v, lse, dout, delta, cu_q, cu_k, pk, pv, err);
    if (A.G > 1) {
        const int64_t n = A.total_k * A.Hkv * (D / 4);
        attn_group_sum_kernel<D><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(A, cu_k, pk, pv, dk, dv);
    }
    return cudaGetLastError();
}

template <int D, int BM, int W, int ST>
cudaError_t rows_backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* lse,
                          const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dq, float* delta,
                          float* part, int parts, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = allow_smem(cache, attn_dq_f32_kernel<D, BM, W, ST>, dq_smem<D, BM, W, ST>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(A.total_q / BM + A.n_seqs), (unsigned)A.Hq, (unsigned)parts);
    attn_dq_f32_kernel<D, BM, W, ST><<<grid, BM * 4 * W, dq_smem<D, BM, W, ST>(), st>>>(
        A, q, k, v, lse, dout, delta, cu_q, cu_k, parts > 1 ? part : dq, parts);
    if (parts > 1) {
        const int64_t n = A.total_q * A.Hq * (D / 4);
        attn_dq_sum_kernel<D><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(A, cu_q, cu_k, BM, parts, part,
                                                                                              dq);
    }
    return cudaGetLastError();
}

template <int D>
cudaError_t backward(const AttnDims& A, const float* q, const float* k, const float* v, const float* out,
                     const float* lse, const float* dout, const int32_t* cu_q, const int32_t* cu_k, float* dq, float* dk,
                     float* dv, float* ws, size_t room, int32_t* err, cudaStream_t st) {
    const int64_t rows = A.total_q * A.Hq;
    const int cut = parts_within(row_parts(A), room, [&](int p) { return backward_floats(A, p) * sizeof(float); });
    float *delta = ws, *parts = ws + (rows + 63) / 64 * 64;
    float* dq_part = parts + (A.G > 1 ? 2 * A.total_k * A.Hq * D : 0);
    const int kb = block_rows(A.total_k, A.n_seqs, A.Hq, 152), qb = block_rows(A.total_q, A.n_seqs, A.Hq, 152);
    attn_delta_kernel<D><<<(unsigned)((rows + 7) / 8), kThreads, 0, st>>>(rows, out, dout, delta);
    const cudaError_t e = (kb == 64   ? keys_backward<D, 64, 1, D == 64 ? 2 : 1>
                           : kb == 32 ? keys_backward<D, 32, kSmallGroups<D>, 1>
                                      : keys_backward<D, 16, kSmallGroups<D>, 1>)(A, q, k, v, lse, dout, cu_q, cu_k, dk, dv,
                                                                                  delta, parts, err, st);
    if (e != cudaSuccess) return e;
    return (qb == 64   ? rows_backward<D, 64, 1, D == 64 ? 2 : 1>
            : qb == 32 ? rows_backward<D, 32, kSmallGroups<D>, 1>
                       : rows_backward<D, 16, kSmallGroups<D>, 1>)(A, q, k, v, lse, dout, cu_q, cu_k, dq, delta, dq_part,
                                                                  cut, st);
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
                                 const int32_t* cu_k, float* out, float* lse, float* part_ws, size_t room, int32_t* err,
                                 cudaStream_t st) {
    return (A.d == 128 ? forward<128> : forward<64>)(A, q, k, v, cu_q, cu_k, out, lse, part_ws, room, err, st);
}
size_t attention_f32_part_bytes(const AttnDims& A) { return part_bytes(A, row_parts(A)); }
size_t attention_backward_f32_floats(const AttnDims& A, bool parts) { return backward_floats(A, parts ? row_parts(A) : 1); }
cudaError_t launch_attention_backward_f32(const AttnDims& A, const float* q, const float* k, const float* v,
                                          const float* out, const float* lse, const float* dout, const int32_t* cu_q,
                                          const int32_t* cu_k, float* dq, float* dk, float* dv, float* ws, size_t room,
                                          int32_t* err, cudaStream_t st) {
    return A.d == 128 ? backward<128>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, room, err, st)
                      : backward<64>(A, q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, ws, room, err, st);
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
