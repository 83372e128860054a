// How a decode step's keys are cut over the thread blocks, shared by its
// kernels and the join.
//
// The keys of all sequences, in units of 64 or 128, form one line of U units; with n
// blocks (at most U: the rest leave at once) block c takes units [c U / n,
// (c + 1) U / n) of it, for one kv head.  Blocks are equally
// loaded whatever the lengths, and only a block's first and last sequence can
// be shared with its neighbours: a sequence that lies in one block is finished
// there, the others leave partial results in slot 2c (the sequence the block
// starts in) or 2c + 1 (a later one it ends in), and the join adds a
// sequence's slots in order.  The lengths are read on the device only, so one
// captured launch serves every step.
#pragma once

#include "attention.cuh"

namespace hla {

struct DecodeLine {
    const int64_t* lens;
    int n_seqs;
    int64_t cap;  // positions a page table can hold
    int unit;     // keys of a unit
    __device__ __forceinline__ int64_t len(int s) const { return clamp_i64(__ldg(lens + s), 0, cap); }
    __device__ __forceinline__ int64_t units(int s) const {
        return s < n_seqs ? (len(s) + unit - 1) / unit : 0;
    }
};

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Units of all sequences, and those of the sequences before s (full warp).
__device__ __forceinline__ int64_t line_units(const DecodeLine& L, int s, int64_t* before) {
    int64_t all = 0, pre = 0;
    for (int i = threadIdx.x & 31; i < L.n_seqs; i += 32) {
        const int64_t u = L.units(i);
        all += u;
        if (i < s) pre += u;
    }
    if (before) *before = warp_sum64(pre);
    return warp_sum64(all);
}

// The sequence that holds unit x of the line (x < U), and its first unit (full warp).
__device__ __forceinline__ int line_find(const DecodeLine& L, int64_t x, int64_t* first) {
    int64_t base = 0;
    for (int s0 = 0; s0 < L.n_seqs; s0 += 32) {
        const int lane = threadIdx.x & 31;
        const int64_t u = L.units(s0 + lane);
        int64_t incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned m = __ballot_sync(0xffffffffu, base + incl > x);
        if (m) {
            const int src = __ffs(m) - 1;
            *first = base + __shfl_sync(0xffffffffu, incl - u, src);
            return s0 + src;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    *first = base;
    return L.n_seqs;
}

// Partial results of slot i, query head h: the weighted sum of values in units
// of 2^vmax, the sum of weights in units of 2^kmax (base-2 logs).
struct DecodePart {
    float* o;   // [slots][Hq][d]
    float* st;  // [slots][Hq][4]: kmax, sum, vmax
};

}  // namespace hla
