// Shared definitions of the full softmax layers: rotary positions, packed
// attention and its gradient, the paged cache and the decode step.
#pragma once

#include "hla_common.cuh"

namespace hla {

constexpr int kMaxRopePairs = 128;

// Angles per position as 64-bit fractions of a turn: position p's angle is
// p * freq mod 2^64, i.e. mod one turn.
struct RopeDims {
    int Hq, Hkv, d, r;
    int interleaved;
    int sign;  // -1: the gradient (rotate back)
    float gain;
    int64_t total, q_in, k_in, q_out, k_out;  // token strides in elements
    uint64_t freq[kMaxRopePairs];
};
template <typename T>
cudaError_t launch_rope(const RopeDims& R, const T* q, const T* k, const int64_t* pos, T* qo, T* ko,
                        cudaStream_t st);

struct AttnDims {
    int Hq, Hkv, d, G;
    int n_seqs;
    int64_t total_q, total_k;
    int64_t sq, sk, sv;  // token strides in elements
    float scale;         // on the scores
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A block of query (or key) positions of one sequence.
struct AttnBlock {
    int64_t q0, k0;  // first query and key row of the sequence
    int lq, lk;      // its lengths
    int first;       // first position of the block within the sequence
    int found;
};

// The r-th block of `rows` query positions over all sequences, the blocks that
// see the most keys first (a block's cost: its index from the sequence's start
// plus the keys in front, in blocks), so that the longest start first.  Every
// sequence has exactly one block of each cost from off + 1 to off + nblk, so
// the number of blocks that cost c or more is a sum over the sequences, and c
// is found by bisection.  Called by a full warp; the result is uniform.
__device__ __forceinline__ AttnBlock attn_find_block(const AttnDims& A, const int32_t* __restrict__ cu_q,
                                                     const int32_t* __restrict__ cu_k, int rows, int64_t r,
                                                     bool by_key) {
    const int lane = threadIdx.x & 31;
    auto shape = [&](int s, int* nblk, int* top) {
        *nblk = 0;
        *top = 0;
        if (s < A.n_seqs) {
            int64_t a, n, b, m;
            seq_range(cu_q, s, A.total_q, &a, &n);
            seq_range(cu_k, s, A.total_k, &b, &m);
            if (by_key) {  // key blocks: the first ones are seen by the most rows
                *nblk = (int)((m + rows - 1) / rows);
                *top = *nblk;
            } else {
                *nblk = (int)((n + rows - 1) / rows);
                const int64_t off = m > n ? (m - n) / rows : 0;
                *top = *nblk + (int)off;
            }
        }
    };
    int n0, t0;  // the first 32 sequences stay in registers
    shape(lane, &n0, &t0);
    auto count = [&](int c) {  // blocks of cost >= c
        int v = max(0, min(n0, t0 - c + 1));
        for (int s = 32 + lane; s < A.n_seqs; s += 32) {
            int n, t;
            shape(s, &n, &t);
            v += max(0, min(n, t - c + 1));
        }
        return (int64_t)__reduce_add_sync(0xffffffffu, v);
    };
    int hi = t0;
    for (int s = 32 + lane; s < A.n_seqs; s += 32) {
        int n, t;
        shape(s, &n, &t);
        hi = max(hi, t);
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    AttnBlock B = {};
    if (hi == 0 || count(1) <= r) return B;  // past the last block
    int lo = 1;                              // count(lo) > r >= count(hi + 1) = 0
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (count(mid) > r) lo = mid; else hi = mid - 1;
    }
    int64_t left = r - count(lo + 1);  // among the sequences with a block of cost lo
    for (int s0 = 0; s0 < A.n_seqs; s0 += 32) {
        int n, t;
        shape(s0 + lane, &n, &t);
        const unsigned has = __ballot_sync(0xffffffffu, t >= lo && lo > t - n);
        const int here = __popc(has);
        if (left < here) {
            const int src = __fns(has, 0, (int)left + 1);
            const int s = s0 + src;
            int64_t a, lq, b, lk;
            seq_range(cu_q, s, A.total_q, &a, &lq);
            seq_range(cu_k, s, A.total_k, &b, &lk);
            const int nb = __shfl_sync(0xffffffffu, n, src), tb = __shfl_sync(0xffffffffu, t, src);
            B.q0 = a;
            B.k0 = b;
            B.lq = (int)lq;
            B.lk = (int)lk;
            const int idx = lo - 1 - (tb - nb);  // 0-based block, counted from the cheapest
            B.first = (by_key ? nb - 1 - idx : idx) * rows;
            B.found = 1;
            return B;
        }
        left -= here;
    }
    return B;
}

// Flags a malformed sequence table (every thread of the block may call it).
__device__ __forceinline__ void attn_check_table(const int32_t* __restrict__ cu, int n, int64_t total,
                                                 int32_t* err) {
    bool bad = threadIdx.x == 0 && (__ldg(cu) != 0 || __ldg(cu + n) > total);
    for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= __ldg(cu + i) > __ldg(cu + i + 1);
    if (bad) atomicExch(err, kErrSeqlens);
}

// Adds the parts (32 at most) of every row of the sequences, in order; a warp per row and head.
template <int D, typename T>
__global__ void __launch_bounds__(256)
attention_join_kernel(AttnDims A, const int32_t* __restrict__ cu_q, int parts, const float* __restrict__ part_o,
                      const float* __restrict__ part_lse, T* __restrict__ out, float* __restrict__ lse) {
    constexpr int E = D / 32;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), rows = A.total_q * A.Hq;
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    const int64_t t = r / A.Hq;
    int64_t a, n;
    seq_range(cu_q, seq_of_token(cu_q, A.n_seqs, t), A.total_q, &a, &n);
    if (t < a || t >= a + n) return;  // behind the last sequence
    const float l = lane < parts ? __ldg(part_lse + lane * rows + r) : -INFINITY;
    float m = l;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float w = l == -INFINITY ? 0.f : exp2f((l - m) * kLog2e);  // NaN stays NaN
    float sum = w, acc[E];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = 0.f;
    for (int p = 0; p < parts; ++p) {
        const float wp = __shfl_sync(0xffffffffu, w, p);
        if (wp == 0.f) continue;  // no keys
        float o[E];
        load_vec<E>(part_o + (p * rows + r) * D + lane * E, o);
#pragma unroll
        for (int x = 0; x < E; ++x) acc[x] = fmaf(wp, o[x], acc[x]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    struct alignas(E * sizeof(T)) { T x[E]; } y;
#pragma unroll
    for (int x = 0; x < E; ++x) y.x[x] = from_f32<T>(acc[x] * inv);
    *reinterpret_cast<decltype(y)*>(out + r * D + lane * E) = y;
    if (lane == 0) lse[r] = sum == 0.f ? -INFINITY : m + logf(sum);
}

// The most parts, up to `most`, whose results fit into `room` bytes; bytes(parts), 0 for one.
template <class Bytes> int parts_within(int most, size_t room, Bytes bytes) {
    while (most > 1 && bytes(most) > room) --most;
    return most;
}

// fp32 layers (attention_f32.cu).  The bytes of partial results of as many parts as suit the sizes (0: one part; `room`
// bytes are there, and as many parts are taken as they hold), and the floats that the gradient needs: dout . out per row and head, (several
// query heads per kv head) dk and dv of each query head, and (parts) dq of each part.
cudaError_t launch_attention_f32(const AttnDims& A, const float* q, const float* k, const float* v, const int32_t* cu_q,
                                 const int32_t* cu_k, float* out, float* lse, float* part_ws, size_t room, int32_t* err,
                                 cudaStream_t st);
size_t attention_f32_part_bytes(const AttnDims& A);
size_t attention_backward_f32_floats(const AttnDims& A, bool parts);
cudaError_t launch_attention_backward_f32(const AttnDims& A, const float* q, const float* k, const float* v,
                                          const float* out, const float* lse, const float* dout, const int32_t* cu_q,
                                          const int32_t* cu_k, float* dq, float* dk, float* dv, float* ws, size_t room,
                                          int32_t* err, cudaStream_t st);
// What is left without keys, or without queries: rows of the sequences to zero (x, and y if given), lse to -infinity;
// the other side's rows and table are checked only.
template <typename T>
cudaError_t launch_attention_empty(int64_t total, int64_t other, int n_seqs, const int32_t* cu, const int32_t* cu_other,
                                   int heads, int d, T* x, T* y, float* lse, int32_t* err, cudaStream_t st);

struct CacheDims {
    int Hkv, d, page, n_pages, max_pages, n_seqs;
    int64_t total;
};
template <typename T>
cudaError_t launch_cache_write(const CacheDims& C, bool e4m3, const hla_cache& c, const T* k, const T* v,
                               const int32_t* cu, const int64_t* start, cudaStream_t st);
template <typename T>
cudaError_t launch_cache_read(const CacheDims& C, bool e4m3, const hla_cache& c, T* k, T* v, const int32_t* cu,
                              const int64_t* start, cudaStream_t st);

size_t attention_decode_ws_bytes(int Hq, int Hkv, int d);
template <typename T>
cudaError_t launch_attention_decode(const AttnDims& A, const CacheDims& C, bool e4m3, const hla_cache& c, const T* q,
                                    const int64_t* lens, T* out, float* part, cudaStream_t st);

}  // namespace hla
