// What the tensor-core attention kernels share: query tiles of packed heads,
// exponentials, bounded waits.
//
// A query tile has 128 rows: `pack` query heads of one kv head (the largest
// power of two, at most 16, that divides the group) times 128 / pack
// positions, row = position * pack + head: the order a TMA box (64, pack, 128
// / pack) of a [tokens][heads][d] tensor lands in.  Packing heads keeps the
// causal edge of a tile short and a short sequence's rows in one tile.
#pragma once

#include <algorithm>

#include "attention.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace hla {
namespace attn_tc {

constexpr int kRows = 128;  // rows of a query tile, keys of a key tile
constexpr uint32_t kWaitLimit = 1u << 22;

// Registers of a block of three warpgroups: 168 a thread at launch; the third
// (loads and products) gives 96 a thread up, the softmax warpgroups take 48
// each.  The launcher checks that the kernel was compiled to that count: an
// increase beyond what the launch holds would never be granted.
constexpr int kBlock = 384, kLaunchRegs = 168, kSoftmaxRegs = 216, kIssueRegs = 72;
static_assert(2 * kSoftmaxRegs + kIssueRegs == 3 * kLaunchRegs, "register split");
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
template <class K>
cudaError_t prepare_kernel(K kernel, size_t smem) {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    if (a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

inline int pack_of(int G) {
    int p = 1;
    while (p < 16 && G % (2 * p) == 0) p *= 2;
    return p;
}

// 2^x by the PTX approximate base-2 exponential (2 ulp; 2^-inf = +0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    unsigned long long ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Waits with a bound (polls, and two seconds); a wait that runs out is recorded and ends the caller's role.
// Inlined: a function call would not leave its caller the registers of setmaxnreg.
__device__ __forceinline__ bool wait_or_flag(uint32_t mbar, uint32_t parity, int32_t* err) {
    if (umma::mbar_try_wait(mbar, parity)) return true;
    const uint64_t t0 = umma::global_ns();
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (umma::mbar_try_wait(mbar, parity)) return true;
        if (umma::global_ns() - t0 > 2000000000ull) break;
    }
    atomicExch(err, kErrTimeout);
    return false;
}

// Hardware barriers 1 .. 15 among some of the block's warps: `sync` waits,
// `arrive` does not.  A warp that waits this way takes no issue slots, where
// one that polls an mbarrier slows the warps beside it.  They cannot time out,
// so whoever arrives does so in every round, whatever has happened; only
// mbarrier waits, which are bounded, can fail.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Rows [first, 128) of a 128 x D 16-bit tile (128-byte-swizzled 64-column blocks) set to zero by one warp.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int first) {
    const int lane = threadIdx.x & 31, n = (kRows - first) * 8;  // 16-byte pieces of a column block
    for (int b = 0; b < D / 64; ++b)
        for (int i = lane; i < n; i += 32)
            *reinterpret_cast<uint4*>(tile + b * (kRows * 128) + first * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace attn_tc

bool attention_tc_supported(const AttnDims& A);
cudaError_t launch_attention_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out,
                                float* lse, int32_t* err, cudaStream_t st);
cudaError_t launch_attention_backward_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                         const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                         const __nv_bfloat16* dout, const int32_t* cu_q, const int32_t* cu_k,
                                         __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, float2* stats,
                                         int32_t* err, cudaStream_t st);

}  // namespace hla
