// Shared definitions of what stands around a layer's mixing: root-mean-square
// norms, the gated recurrence, products with 4-bit weights.
#pragma once

#include <cuda_fp8.h>

#include "hla_common.cuh"

namespace hla {

// Two fp32 values at once (with ffma2).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}

// V values in a row, loaded and stored at once.  At most 16 bytes: callers' rows are checked for 16 bytes and no more, and a
// wider type promises the compiler an alignment for which it may choose a wider access.
template <typename T, int V> struct alignas(V * sizeof(T)) Piece {
    static_assert(V * sizeof(T) <= 16, "a piece is one access of up to 16 bytes");
    T x[V];
};

// Groups of values as 8-bit floats (e4m3) times a power of two, as the cache
// keeps its rows: the smallest e >= -127 with top <= 448 2^e (top finite, >= 0).
__device__ __forceinline__ int group_exponent(float top) {
    const uint32_t b = __float_as_uint(top);
    return max((int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u), -127);
}
__device__ __forceinline__ float group_pow2(int e) {  // -127 <= e <= 127
    return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x400000u);
}

// Thread-block clusters along x.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Sum over the cluster's n blocks (1, 2, 4, 8), in their order, of the float at the same shared-memory offset as `local`.
__device__ __forceinline__ float ld_cluster(const float* local, uint32_t rank) {
    uint32_t a;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
template <int N> __device__ __forceinline__ float cluster_sum_of(const float* local) {
    float v[N], y = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] = ld_cluster(local, c);
#pragma unroll
    for (int c = 0; c < N; ++c) y += v[c];
    return y;
}
__device__ __forceinline__ float cluster_sum(const float* local, int n) {
    return n == 2 ? cluster_sum_of<2>(local) : n == 4 ? cluster_sum_of<4>(local) : cluster_sum_of<8>(local);
}
struct ClusterCfg {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    ClusterCfg(dim3 grid, int threads, size_t smem, cudaStream_t st, int blocks) {
        cfg.gridDim = grid;
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = blocks > 1 ? 1 : 0;
    }
    ClusterCfg(const ClusterCfg&) = delete;
    ClusterCfg& operator=(const ClusterCfg&) = delete;
};

struct NormDims {
    int64_t rows, sx, sr;  // rows of n_cols values; token strides of x and the residual
    int cols, heads, group;
    float eps, offset;
};
// out8: 8-bit rows with exponents exp (else out); residual, sum, weight may be null.
template <typename T>
cudaError_t launch_norm(const NormDims& N, const T* x, const T* residual, const T* weight, T* out, uint8_t* out8,
                        uint8_t* exp, T* sum, cudaStream_t st);
// part: fp32 [norm_parts(cols)][cols]
template <typename T>
cudaError_t launch_norm_backward(const NormDims& N, const T* s, const T* weight, const T* dout, const T* dsum, T* dx,
                                 float* dweight, float* part, cudaStream_t st);
// Blocks of a norm's gradient, at most.  Up to 1024 columns twelve an SM (of 152; rows of 512 bf16 take eight: 100000 of them
// 103 us, 122 with 1024 blocks in all), then as many as a block of cols / 16 threads leaves room for, six at most; two past
// 16384 columns, where rows are read twice.
constexpr int norm_parts(int cols) { return 152 * (cols <= 1024 ? 12 : cols > 16384 ? 2 : cols <= 2730 ? 6 : 16384 / cols); }

// The gated recurrence.  Gates: one per channel (gate_dim 1) or per gate_dim (64, 128) channels.
constexpr int kStateRows = 64;  // rows between the states that a gradient starts from
struct RecDims {
    int64_t total, sx, sg;  // rows; token strides of x and g
    int channels, gate_dim, n_seqs;
};
// Bytes of carries between tiles (0: one tile in time, or none), for both directions.
size_t recurrence_carry_bytes(const RecDims& R, bool f32);
template <typename T, typename G>
cudaError_t launch_recurrence(const RecDims& R, const G* g, const T* x, const float* h0, const int32_t* cu, T* out,
                              float* h_last, float* states, char* carry, int32_t* err, cudaStream_t st);
template <typename T, typename G>
cudaError_t launch_recurrence_backward(const RecDims& R, const G* g, const T* x, const float* h0, const float* states,
                                       const int32_t* cu, const T* dout, const float* dh_last, G* dg, T* dx,
                                       float* dh0, char* carry, int32_t* err, cudaStream_t st);
template <typename T, typename G>
cudaError_t launch_recurrence_step(const RecDims& R, const G* g, const T* x, float* h, T* out, cudaStream_t st);

// Products with 4-bit weights: w [n_out][n_in / 2] bytes, the even input in the low half; scales and offsets
// [n_out][n_in / group].  More than kFewRows rows of x as bf16 parts in
// `parts`, where they are not bf16 on 16-byte boundaries.
struct Linear4Dims {
    int64_t rows, sx;  // tokens; token stride of x in elements
    int n_in, n_out, group, x_group;
};
constexpr int64_t kFewRows = 16;  // that no rows are laid out for
// Blocks of a cluster that share a tile's inputs: of 1, 2, 4 and 8 the one with the least sum of rounds (of `blocks` at a
// time) by steps, where a block's start and end take as long as `ends` steps.
int linear4_split(int64_t tiles, int64_t stages, int64_t blocks, int64_t ends);
enum class Rows4 { kF32, kBf16, kE4m3 };
int linear4_parts(Rows4 kind);
template <typename T>
cudaError_t launch_linear4(const Linear4Dims& L, Rows4 kind, const void* x, const uint8_t* x_exp, const uint8_t* w,
                           const T* scales, const T* offsets, T* out, __nv_bfloat16* parts, cudaStream_t st);
// More than kFewRows rows: `parts` bf16 parts [parts][rows][n_in] (or one, sx apart) on 16-byte boundaries.
template <typename T>
cudaError_t launch_linear4_tc(const Linear4Dims& L, int parts, const __nv_bfloat16* x, const uint8_t* w, const T* scales,
                              const T* offsets, T* out, cudaStream_t st);
template <typename T>
cudaError_t launch_linear4_quantize(const Linear4Dims& L, const T* weight, uint8_t* w, T* scales, T* offsets,
                                    cudaStream_t st);

}  // namespace hla
