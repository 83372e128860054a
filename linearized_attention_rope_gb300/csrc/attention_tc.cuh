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
constexpr uint32_t kWaitLimit = 1u << 22;  // polls per second allowed

// Registers of a block of three warpgroups: 168 a thread at launch; the third
// (loads and products) gives 112 a thread up, the softmax warpgroups take 56
// each.  The launcher checks that the kernel was compiled to that count: an
// increase beyond what the launch holds would never be granted.
constexpr int kBlock = 384, kLaunchRegs = 168, kSoftmaxRegs = 224, kIssueRegs = 56;
static_assert(2 * kSoftmaxRegs + kIssueRegs == 3 * kLaunchRegs, "register split");
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;"); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
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

// Waits with a bound (polls, and two seconds); a wait that runs out is recorded, and the caller's role goes on without
// waiting.  The last poll comes after the time has been found to be up, so that a lane sees what the others of its warp
// saw before (a vote per wait: 4096 tokens with gradient 457 -> 469 us).  Inlined: a function call would not leave its
// caller the registers of setmaxnreg.
__device__ __forceinline__ bool wait_or_flag(uint32_t mbar, uint32_t parity, int32_t* err) {
    if (umma::mbar_try_wait(mbar, parity)) return true;
    const uint64_t t0 = umma::global_ns();
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitLimit * 2; ++i) {
        if (umma::mbar_try_wait(mbar, parity)) return true;
        if (umma::global_ns() - t0 > 2000000000ull) break;
    }
    if (umma::mbar_try_wait(mbar, parity)) return true;
    atomicExch(err, kErrTimeout);
    return false;
}
// A full warp's wait with a bound on the polls alone: time in which the whole block stands still does not count.
__device__ __forceinline__ bool wait_polls(uint32_t mbar, uint32_t parity, int32_t* err, uint32_t polls) {
#pragma unroll 1
    for (uint32_t i = 0; i < polls; ++i)
        if (__all_sync(0xffffffffu, umma::mbar_try_wait(mbar, parity))) return true;
    atomicExch(err, kErrTimeout);
    return false;
}

// Hardware barriers 1 .. 15 among some of the block's warps: `sync` waits,
// `arrive` does not.  A warp that waits this way takes no issue slots, where
// one that polls an mbarrier slows the warps beside it.  They cannot time out,
// so whoever arrives does so in every round of every item that is handed out,
// whatever has happened: only mbarrier waits, which are bounded, can fail, and a
// role whose wait failed goes on without waiting.  All roles must then see the
// same items (below).
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- persistent blocks ------------------------------------------------------
//
// The grid has a block per item (a tile or two of one head group), longest
// first; a block that runs takes over items of blocks that have not started
// (cluster launch control), so one block per SM does them all and the next
// free SM always takes the longest that is left.  A warp of its own asks for
// the next item, finds what it is, and hands it to the others through a short
// ring, so that every role runs ahead into the next item on its own: its loads
// start while the last products and results of this one are under way.
// The next item is asked for when the loads of this one come to an end, not
// before: items claimed early would be kept from blocks that are free sooner.
//
// A role that gave up waiting for an item which the others then get would leave
// them at a hardware barrier for ever.  So the roles wait longer than the
// scheduling warp can take to hand out an item or the end, all its own waits run out;
// and where it finds that a role has not taken the item before last, it hands out nothing
// more, so that no role does.

struct Item {
    int q0, k0;  // first query and key row of the sequence (of the item's part of the keys)
    int lq, lk;  // its lengths
    int first;   // first position of the tile(s)
    int head;    // first query head, or the kv head; -1: no more items
    int off;     // row i sees keys j <= i + off
    int part;    // which part of the keys; or the item's number (`numbered`)
};
constexpr int kItems = 2;       // entries of the ring
constexpr int kItemWarps = 11;  // warps that read them
constexpr uint32_t kItemPolls = 60 * kWaitLimit;    // of a wait of the scheduling warp: as long as an item may take
constexpr uint32_t kReaderPolls = 6 * kItemPolls;   // of a wait for an item
// at half the scheduling warp's rate: its waits for a free entry, for a request, and for the request's answer
static_assert(kReaderPolls / 2 > 2 * kItemPolls + 2 * kWaitLimit, "roles wait longer than the scheduling warp");
struct ItemRing {
    int4 word[kItems][2];
    uint4 answer;  // of a request for the next item
};

// Asks for an item of a block that has not started; the answer arrives on mbar.  (One lane.)
__device__ __forceinline__ void ask_item(uint32_t answer, uint32_t mbar) {
    tma::expect_tx(mbar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(mbar)
                 : "memory");
}
// The block whose item was taken over; -1: there is none left.
__device__ __forceinline__ int64_t taken_item(uint32_t answer) {
    uint32_t got, x;
    asm volatile(
        "{\n .reg .b128 a;\n .reg .pred p;\n ld.shared.b128 a, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n}\n"
        : "=r"(got), "=r"(x)
        : "r"(answer)
        : "memory");
    return got ? (int64_t)x : -1;
}

// The scheduling warp: `heads` head groups, `rows` positions per item, each in
// `parts` parts: of query positions, the visible keys are cut into parts of
// whole tiles, eight at least (the parts past those get none); of keys, the
// reader cuts the rows that see them.  Given a list (its length, then item numbers), the
// grid's blocks take its items in turn.
template <class HeadOf>
__device__ __forceinline__ void schedule_items(const AttnDims& A, const int32_t* cu_q, const int32_t* cu_k, int rows,
                                               int heads, bool by_key, ItemRing* ring, uint32_t bar_full,
                                               uint32_t bar_empty, uint32_t bar_ask, uint32_t bar_want, int32_t* err,
                                               HeadOf head_of, int parts = 1, bool numbered = false,
                                               const int* list = nullptr) {
    const int lane = threadIdx.x & 31;
    const uint32_t answer = umma::smem_addr(&ring->answer);
    int64_t x = blockIdx.x, listed = x;
    if (list) x = listed < list[0] ? list[1 + listed] : -1;
    bool more = true;
    for (int i = 0; more; ++i) {
        AttnBlock B = {};
        const int part = numbered ? (int)x : parts > 1 && x >= 0 ? (int)(x % parts) : 0;
        if (x >= 0) B = attn_find_block(A, cu_q, cu_k, rows, x / parts / heads, by_key);
        const int s = i % kItems;
        more = B.found;
        if (i >= kItems && !wait_polls(bar_empty + 8 * s, ((i / kItems) - 1) & 1, err, kItemPolls)) break;
        int k0 = (int)B.k0, lk = B.lk, off = B.lk - B.lq;
        if (parts > 1 && !by_key) {
            const int end = max(0, min(B.lk, min(B.first + rows, B.lq) + off)), n = (end + kRows - 1) / kRows;
            const int cut = max(1, min(parts, n / 8)), a = part < cut ? (int)((int64_t)n * part / cut) * kRows : end;
            const int b = part < cut ? (int)((int64_t)n * (part + 1) / cut) * kRows : end;
            k0 += a;
            lk = min(lk, b) - a;
            off -= a;
        }
        if (lane == 0) {
            ring->word[s][0] = make_int4((int)B.q0, k0, B.lq, lk);
            ring->word[s][1] = make_int4(B.first, more ? head_of((int)(x / parts % heads)) : -1, off, part);
        }
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(bar_full + 8 * s);
        if (!more) break;
        x = -1;
        if (wait_polls(bar_want, i & 1, err, kItemPolls)) {
            if (list) {
                listed += gridDim.x;
                if (listed < list[0]) x = list[1 + listed];
                continue;
            }
            if (lane == 0) ask_item(answer, bar_ask);
            if (__any_sync(0xffffffffu, wait_or_flag(bar_ask, i & 1, err))) x = taken_item(answer);
            __syncwarp();
            umma::fence_async_smem();
        }
    }
}

// The i-th item of this block (a full warp; each reader in order).
__device__ __forceinline__ Item next_item(const ItemRing* ring, int i, uint32_t bar_full, uint32_t bar_empty,
                                          int32_t* err) {
    const int s = i % kItems;
    Item it = {0, 0, 0, 0, 0, -1, 0, 0};
    if (wait_polls(bar_full + 8 * s, (i / kItems) & 1, err, kReaderPolls)) {
        const int4 a = ring->word[s][0], b = ring->word[s][1];
        it = Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) umma::mbar_arrive(bar_empty + 8 * s);
    return it;
}

// Position in a ring of n slots that is used over and over: slot, and the parity of its current round.
template <int N> struct RingPos {
    uint32_t slot = 0, par = 0;
    __device__ __forceinline__ RingPos next() {  // this use; moves on
        const RingPos u = *this;
        if (++slot == N) {
            slot = 0;
            par ^= 1u;
        }
        return u;
    }
};

// Infinities and NaN in rows [first, last) of a 128 x D bf16 tile
// (128-byte-swizzled 64-column blocks) set to zero by one warp: rows that some
// or all rows of the product must not see weigh 0 there, and 0 times infinity
// would reach them all the same.  found(row) for each row that held any.
// Looking costs less than clearing: 0 x + acc over a batch of pieces, one
// packed multiply-add per two elements, is 0 unless an x is infinite or NaN.
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {  // of each 16-bit half: all ones where it is finite
    return ((w & 0x7f80u) != 0x7f80u ? 0x0000ffffu : 0u) | ((w & 0x7f800000u) != 0x7f800000u ? 0xffff0000u : 0u);
}
__device__ __forceinline__ uint32_t add_zero_times(uint32_t x, uint32_t acc) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
}
template <int D, class Found>
__device__ __forceinline__ void clear_nonfinite(unsigned char* tile, int first, int last, Found found) {
    constexpr int kBatch = 8;  // pieces on their way
    const int lane = threadIdx.x & 31, n = max(0, last - first) * 8;  // 16-byte pieces of a column block
    for (int b = 0; b < D / 64; ++b) {
        uint4* p = reinterpret_cast<uint4*>(tile + b * (kRows * 128) + first * 128);
#pragma unroll 1
        for (int i0 = lane; i0 - lane < n; i0 += 32 * kBatch) {
            uint4 x[kBatch];
            uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                x[y] = make_uint4(0u, 0u, 0u, 0u);
                if (i0 + 32 * y < n) x[y] = p[i0 + 32 * y];
            }
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                acc[0] = add_zero_times(x[y].x, acc[0]);
                acc[1] = add_zero_times(x[y].y, acc[1]);
                acc[2] = add_zero_times(x[y].z, acc[2]);
                acc[3] = add_zero_times(x[y].w, acc[3]);
            }
            if (((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) == 0u) continue;
#pragma unroll 1
            for (int i = i0; i < min(n, i0 + 32 * kBatch); i += 32) {
                const uint4 w = p[i];
                const uint4 m = make_uint4(finite_mask(w.x), finite_mask(w.y), finite_mask(w.z), finite_mask(w.w));
                if ((m.x & m.y & m.z & m.w) == 0xffffffffu) continue;
                p[i] = make_uint4(w.x & m.x, w.y & m.y, w.z & m.z, w.w & m.w);
                found(first + (i >> 3));
            }
        }
    }
}

}  // namespace attn_tc

// The bytes of partial results of as many parts as suit the sizes (0: one part).  The launches take as many as fit into
// `room` bytes; the gradient needs those of one part (`parts` false) in any case: -lse and -D per row and head.
size_t attention_tc_part_bytes(const AttnDims& A);
cudaError_t launch_attention_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out,
                                float* lse, void* parts, size_t room, int32_t* err, cudaStream_t st);
size_t attention_backward_tc_bytes(const AttnDims& A, bool parts);
cudaError_t launch_attention_backward_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                         const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                         const __nv_bfloat16* dout, const int32_t* cu_q, const int32_t* cu_k,
                                         __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, void* ws, size_t room,
                                         int32_t* err, cudaStream_t st);

}  // namespace hla
