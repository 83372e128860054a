// Gated linear recurrence over packed sequences, its gradient, and its step: what their kernels share.
//
//   h_t = exp(g_t) h_{t-1} + x_t                    per channel, from h0 (or 0)
//   l_t = dout_t + exp(g_{t+1}) l_{t+1}              (dh_last behind the last row)
//   dx_t = l_t,  dg_t = l_t exp(g_t) h_{t-1},  dh0 = exp(g_1) l_1
//
// Memory bound: gates and inputs are read once, outputs written once.  A row is
// an affine map of the state, so that a run of rows is one too, h -> A h + B.
// A block takes a tile of rows by a slab of 32 x 2 (or 4) channels, a warp a run
// of its rows, which stays in registers: every warp forms its run's (A, B), the
// tile's own is handed to the tiles behind it, the state in front of the tile is
// taken from the tiles before it, and each warp then walks its rows with the
// state in front of them.
//
// A run's A is kept as its root and applied twice, a tile's too where A does not
// fit fp32 (which costs calls of few channels 8 %: 131072 rows of one channel 55
// us, 51 with gates that sum up to less than 80 over a tile).
//
// The state in front of a tile: every tile publishes (A, B) and, once it knows
// it, the state behind it.  A tile looks at the eight tiles before it, then at
// up to 32 (four channels a lane: 16); the nearest with a state is carried
// forward by the (A, B) of those between, tile after tile.  That is what each of
// those tiles does itself, rounding for rounding, so that results do not depend
// on which of them was found.  Tiles are handed out in order of time, so that
// those waited for are running.  Every word carries its own flag: no fences, and
// one trip through L2 per look.
//
// Gates of a run and channel enter as v = exp(g) - 1, with the state added (w =
// 1), where all of them are within [-ln 2, 0]: a state that decays slowly (|g| of
// 1e-3 and less, thousands of rows) keeps its bits, where a rounded exp(g) would
// be off by up to 2^-25 in every row, the same way for the same gate.  Otherwise
// as v = exp(g) (w = 0), so that a closed gate leaves nothing of the state, not
// even a rounding.  Either way a row is w h + (v h + x): two packed FMAs for two
// channels.  Instructions are what these kernels have few of: a row of 64 channels
// takes 34 in the forward pass, a warp's run another 800, and at the copy rate an
// SM has about 55 for a row of bf16 values and gates.
//
// The gradient runs the tiles from the last to the first.  States in front of
// its rows come from those that the forward pass kept every 64 rows.
#pragma once

#include <algorithm>

#include "layer.cuh"

namespace hla {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kPolls = 1 << 20;     // looks at a tile that has nothing yet (about 0.7 us each)
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
// exp(g) - 1 = g q(g) on [-ln 2, 0]: q of degree 5 by Remez' exchange on the relative error (2^-26.7, in fp32 2^-23.2).
__device__ __forceinline__ float2 mild(float2 g) {
    float2 q = splat(0x1.0ed49ep-10f);
    q = ffma2(q, g, splat(0x1.0858e4p-7f));
    q = ffma2(q, g, splat(0x1.548ecap-5f));
    q = ffma2(q, g, splat(0x1.554d38p-3f));
    q = ffma2(q, g, splat(0x1.ffffc2p-2f));
    q = ffma2(q, g, splat(1.f));
    return mul2(g, q);
}
// exp(g) for |g| <= kBig, by the hardware's power of two: off by up to 2^-22 of itself, and by 2^-22 ln 2 where g / ln 2 is
// rounded (below 8), which with the row's own rounding is less than the 2^-21 of its magnitudes that a row may add.
__device__ __forceinline__ float2 strong(float2 g) {
    const float2 t = mul2(g, splat(1.44269504f));
    float2 a;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(t.y));
    return a;
}
constexpr float kLow = -0.69314f, kBig = 5.5f;  // mild: kLow to 0
// exp(g) h + x
__device__ __forceinline__ float2 through(float2 v, float2 w, float2 h, float2 x) { return ffma2(w, h, ffma2(v, h, x)); }
// exp(g) h
__device__ __forceinline__ float2 times(float2 v, float2 w, float2 h) { return ffma2(w, h, mul2(v, h)); }

// The factor exp(s) of a run whose gates add up to s, as its root, which is applied twice and is a normal number as far as a
// state can stay one under it (at most exp(88): a normal state that grows by more than exp(176) passes fp32's range).  So
// that 0 stays 0, and what shrinks or grows by more than fp32 holds comes out as row by row.  The root of a tile's factor is the
// product of its runs', as long as that cannot leave fp32's range (sums up to kFar each: exp(80) in all), else that of the sum
// of their sums; a tile hands on its square where that is within exp(+-80).
constexpr float kFar = 20.f;
__device__ __forceinline__ float2 roots(float2 s) {
    return make_float2(expf(fminf(0.5f * s.x, 88.f)), expf(fminf(0.5f * s.y, 88.f)));
}
__device__ __forceinline__ bool within(float2 s, float most) { return fabsf(s.x) <= most && fabsf(s.y) <= most; }
__device__ __forceinline__ bool squares(float2 root) {
    const float hi = 2.3538527e17f, lo = 4.2483543e-18f;  // exp(+-40)
    return root.x >= lo && root.x <= hi && root.y >= lo && root.y <= hi;
}
__device__ __forceinline__ float2 twice(float2 root, float2 c, float2 b) { return ffma2(root, mul2(root, c), b); }

// Two values, each in a word with its own flags (0 where it has not been written; 1, and 2 for a root).
__device__ __forceinline__ void put_words(uint64_t* p, float2 v, uint32_t flags = 1) {
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"((uint64_t)flags << 32 | __float_as_uint(v.x)),
                 "l"((uint64_t)flags << 32 | __float_as_uint(v.y)) : "memory");
}
__device__ __forceinline__ uint32_t get_words(const uint64_t* p, float2* v) {
    uint64_t x, y;
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "l"(p) : "memory");
    *v = make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)y));
    return (uint32_t)((x & y) >> 32);
}

// Carries between tiles: per tile and channel the state behind it, and its (A, B).
struct Carry {
    uint64_t* state;
    uint64_t* map;  // two words each
    int* ticket;
};

// Two neighbouring values of a row, in fp32.
template <int CPL> __device__ __forceinline__ float2 two(const Piece<float, CPL>& v, int p) {
    return make_float2(v.x[2 * p], v.x[2 * p + 1]);
}
template <int CPL> __device__ __forceinline__ float2 two(const Piece<__nv_bfloat16, CPL>& v, int p) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(v.x)[p];
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T, int CPL> __device__ __forceinline__ Piece<T, CPL> pack(const float2 (&f)[CPL / 2]) {
    Piece<T, CPL> v;
#pragma unroll
    for (int p = 0; p < CPL / 2; ++p) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<__nv_bfloat162*>(&v.x[2 * p]) = __floats2bfloat162_rn(f[p].x, f[p].y);
        } else {
            v.x[2 * p] = f[p].x;
            v.x[2 * p + 1] = f[p].y;
        }
    }
    return v;
}

// The channels of a lane: CPL in a row (VEC), else 32 apart.
template <int CPL, bool VEC>
struct Lane {
    int c0, from;  // (a lane past the last channel reads the first ones, and stores nothing)
    bool on[VEC ? 1 : CPL];
    __device__ __forceinline__ Lane(int slab, int channels) {
        const int lane = threadIdx.x & 31;
        c0 = slab * 32 * CPL + (VEC ? lane * CPL : lane);
#pragma unroll
        for (int j = 0; j < (VEC ? 1 : CPL); ++j) on[j] = c0 + 32 * j < channels;
        from = on[0] ? c0 : 0;
    }
    template <typename U> __device__ __forceinline__ Piece<U, CPL> load(const U* row) const {
        Piece<U, CPL> v;
        if constexpr (VEC) {
            v = *reinterpret_cast<const Piece<U, CPL>*>(row + from);
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j) v.x[j] = on[j] ? row[c0 + 32 * j] : from_f32<U>(0.f);
        }
        return v;
    }
    template <typename U> __device__ __forceinline__ void store(U* row, const float2 (&f)[CPL / 2]) const {
        const Piece<U, CPL> v = pack<U, CPL>(f);
        if constexpr (VEC) {
            if (on[0]) *reinterpret_cast<Piece<U, CPL>*>(row + c0) = v;
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                if (on[j]) row[c0 + 32 * j] = v.x[j];
        }
    }
    __device__ __forceinline__ void load_pairs(const float* row, float2 (&f)[CPL / 2]) const {
        const Piece<float, CPL> v = load(row);
#pragma unroll
        for (int p = 0; p < CPL / 2; ++p) f[p] = two(v, p);
    }
};

// What a warp's rows are: bit i for row t0 + i.  seq: of row t0 + lane.
struct Rows {
    uint32_t valid, first, last;
    int seq;
    __device__ __forceinline__ Rows(const int32_t* __restrict__ cu, const RecDims& R, int64_t t0, int n) {
        const int lane = threadIdx.x & 31;
        const int64_t t = t0 + lane;
        bool v = false, f = false, l = false;
        seq = 0;
        if (lane < n && t < R.total) {
            seq = seq_of_token(cu, R.n_seqs, t);
            int64_t a, m;
            seq_range(cu, seq, R.total, &a, &m);
            v = t >= a && t < a + m;
            f = v && t == a;
            l = v && t == a + m - 1;
        }
        valid = __ballot_sync(kFull, v);
        first = __ballot_sync(kFull, f);
        last = __ballot_sync(kFull, l);
    }
};

// The tile of this block: tickets in order of time where there is more than one tile in time.
__device__ __forceinline__ int take_tile(int* ticket, int n_time) {
    if (n_time == 1) return blockIdx.x;
    __shared__ int tile;
    if (threadIdx.x == 0) tile = atomicAdd(ticket, 1);
    __syncthreads();
    return tile;
}

__device__ __forceinline__ void check_table(const int32_t* __restrict__ cu, const RecDims& R, int32_t* err) {
    bool bad = false;
    for (int i = threadIdx.x; i <= R.n_seqs; i += kThreads) {
        const int64_t v = __ldg(cu + i);
        bad |= v < 0 || v > R.total || (i == 0 ? v != 0 : v < __ldg(cu + i - 1));
    }
    if (bad) atomicExch(err, kErrSeqlens);
}

// The state in front of tile k (of the order in which tiles are handed out), after this tile has published its own
// (A, B), or its state where that does not depend on what is in front.  Called by the whole block.
template <int NP>
__device__ __forceinline__ void look_back(const Carry& S, int k, int n_slabs, int slab, float2 (&c)[NP], int32_t* err) {
    constexpr int kDeep = 4 / NP, kLook = kDeep * kWarps;  // a warp looks at the tile 1 + warp before this one, 9 + warp ...
    __shared__ float2 pa[kLook][NP][32], pb[kLook][NP][32];
    __shared__ int status[kLook];  // 0 nothing yet, 1 (A, B), 2 the state, 3 given up; 5 (A, B), A as its root
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int polls = 0, m, deep = 1;
    bool some;  // A as its root
    for (int i = threadIdx.x; i < kLook; i += kThreads) status[i] = 0;
    __syncthreads();
    for (;;) {
        for (int d = 0; d < deep; ++d) {
            const int i = d * kWarps + warp, pred = k - 1 - i;
            const int had = status[i];  // (written by this warp alone)
            if ((had & 3) >= 2) continue;
            int have = had;
            if (pred < 0) {
#pragma unroll
                for (int p = 0; p < NP; ++p) pb[i][p][lane] = splat(0.f);
                have = 2;
            } else {
                const int64_t at = (((int64_t)pred * n_slabs + slab) * 32 + lane) * 2 * NP;
                do {
                    float2 s[NP], a[NP], b[NP];
                    uint32_t is = 3, has = 3;
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        is &= get_words(S.state + at + 2 * p, &s[p]);
                        if (!have) {
                            has &= get_words(S.map + 2 * at + 4 * p, &a[p]);
                            has &= get_words(S.map + 2 * at + 4 * p + 2, &b[p]);
                        }
                    }
                    if (__all_sync(kFull, is != 0)) {
#pragma unroll
                        for (int p = 0; p < NP; ++p) pb[i][p][lane] = s[p];
                        have = 2;
                    } else if (!have && __all_sync(kFull, has != 0)) {
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            pa[i][p][lane] = a[p];
                            pb[i][p][lane] = b[p];
                        }
                        have = has & 2 ? 5 : 1;  // (the same in all lanes)
                    }
                    if ((have & 3) < 2 && ++polls > kPolls) have = 3;
                } while (!have);
            }
            __syncwarp();
            if (lane == 0) status[i] = have;
        }
        __syncthreads();
        const int got = status[lane % kLook];
        const unsigned ready = __ballot_sync(kFull, got == 2);
        some = __any_sync(kFull, got == 5);
        if (__any_sync(kFull, got == 3)) {
            m = -1;
            break;
        }
        if (ready) {  // (the tiles between have their (A, B))
            m = __ffs(ready) - 1;
            break;
        }
        if (deep < kDeep) ++deep;
        __syncthreads();  // before status is written again
    }
    if (m < 0) {
        if (threadIdx.x == 0) atomicExch(err, kErrTimeout);
        // NaN, so that what depends on the state is not taken for an answer where nobody reads the error word
#pragma unroll
        for (int p = 0; p < NP; ++p) c[p] = splat(__int_as_float(0x7fc00000));
        return;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) c[p] = pb[m][p][lane];
    if (some) {
#pragma unroll 4
        for (int w = m - 1; w >= 0; --w) {
            const bool root = status[w] == 5;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const float2 a = pa[w][p][lane], f = root ? a : splat(1.f);
                c[p] = ffma2(a, mul2(f, c[p]), pb[w][p][lane]);
            }
        }
        return;
    }
#pragma unroll 4
    for (int w = m - 1; w >= 0; --w)
#pragma unroll
        for (int p = 0; p < NP; ++p) c[p] = ffma2(pa[w][p][lane], c[p], pb[w][p][lane]);
}

// The warps' (A, B) of a tile, A as its root, in the order in which the state passes them.
template <int NP>
struct Runs {
    float2 a[kWarps][NP][32], b[kWarps][NP][32];
    int kind[kWarps];  // 1: the state does not pass this run; 2: some sum of gates is past kFar
    __device__ __forceinline__ void put(int w, const float2 (&A)[NP], const float2 (&B)[NP], bool cut, bool far) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            a[w][p][lane] = A[p];
            b[w][p][lane] = B[p];
        }
        if (lane == 0) kind[w] = (cut ? 1 : 0) | (far ? 2 : 0);
    }
    // from run w0 to run w1
    __device__ __forceinline__ void pass(int w0, int w1, float2 (&c)[NP]) const {
        const int lane = threadIdx.x & 31;
        for (int w = w0; w < w1; ++w) {
            const bool is = kind[w] & 1;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const float2 y = b[w][p][lane], z = twice(a[w][p][lane], c[p], y);
                c[p] = is ? y : z;
            }
        }
    }
};
// The sums of the runs' gates.
template <int NP> using Sums = float2[kWarps][NP][32];

// Publishes tile k's map (or state, where a run of it is cut), takes the state in front of it, publishes the one behind.
template <int NP>
__device__ __forceinline__ void tile_carry(const Carry& S, const Runs<NP>& runs, const Sums<NP>& sums, int k,
                                           int n_time, int n_slabs, int slab, float2 (&c)[NP], int32_t* err) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int p = 0; p < NP; ++p) c[p] = splat(0.f);
    if (n_time == 1) return;
    float2 A[NP], B[NP];
    int kinds = 0;
    bool root = false;
    const int64_t at = (((int64_t)k * n_slabs + slab) * 32 + lane) * 2 * NP;
    if (threadIdx.x < 32 && k + 1 < n_time) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            A[p] = splat(1.f);
            B[p] = splat(0.f);
        }
        runs.pass(0, kWarps, B);
        for (int w = 0; w < kWarps; ++w) {
            kinds |= runs.kind[w];
#pragma unroll
            for (int p = 0; p < NP; ++p) A[p] = mul2(A[p], runs.a[w][p][lane]);
        }
        if (kinds == 2)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float2 total = splat(0.f);
                for (int w = 0; w < kWarps; ++w) total = add2(total, sums[w][p][lane]);
                A[p] = roots(total);
            }
        bool fine = true;
#pragma unroll
        for (int p = 0; p < NP; ++p) fine = fine && squares(A[p]);
        root = !__all_sync(kFull, fine);
#pragma unroll
        for (int p = 0; p < NP; ++p)
            if (!root) A[p] = mul2(A[p], A[p]);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (kinds & 1) {
                put_words(S.state + at + 2 * p, B[p]);
            } else {
                put_words(S.map + 2 * at + 4 * p, A[p], root ? 3 : 1);
                put_words(S.map + 2 * at + 4 * p + 2, B[p], root ? 3 : 1);
            }
        }
    }
    look_back<NP>(S, k, n_slabs, slab, c, err);
    if (threadIdx.x < 32 && k + 1 < n_time && !(kinds & 1))
#pragma unroll
        for (int p = 0; p < NP; ++p) put_words(S.state + at + 2 * p, root ? twice(A[p], c[p], B[p]) : ffma2(A[p], c[p], B[p]));
}

// A warp's gates as (v, w): v per row and pair of channels, or (SHARED) row i's in lane i; w per pair.
template <typename G, int CPL, bool SHARED, bool VEC, int ROWS>
struct Gates {
    static constexpr int NP = SHARED ? 1 : CPL / 2;
    Piece<G, CPL> raw[SHARED ? 1 : ROWS];
    float2 v[SHARED ? 1 : ROWS][NP];
    float2 w[NP];
    float2 sum[NP];  // of the run's g

    template <bool FULL> __device__ __forceinline__ void load(const Lane<CPL, VEC>& at, const G* g, int64_t stride, int slab, int n) {
        if constexpr (SHARED) {
            const int lane = threadIdx.x & 31;
            raw[0].x[0] = lane < n ? g[lane * stride + slab] : from_f32<G>(0.f);
        } else {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) raw[i] = FULL || i < n ? at.load(g + i * stride) : Piece<G, CPL>{};
        }
    }
    // valid: the rows that are part of a sequence (the others let the state pass)
    template <bool EDGE> __device__ __forceinline__ void form(uint32_t valid) {
#pragma unroll
        for (int p = 0; p < NP; ++p) sum[p] = splat(0.f);
        if constexpr (SHARED) {
            const int lane = threadIdx.x & 31;
            float g = to_f32(raw[0].x[0]);
            if (lane >= ROWS || (EDGE && !(valid >> lane & 1))) g = 0.f;
            float s = g;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            sum[0] = splat(s);
            const bool far = __any_sync(kFull, !(g <= 0.f && g >= kLow));
            w[0] = splat(far ? 0.f : 1.f);
            v[0][0] = far ? splat(expf(g)) : mild(splat(g));
        } else {
            float2 least[NP], most[NP];  // of the run's gates, and 0 (NaN passes as mild, and stays NaN)
            if constexpr (EDGE) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
                    if (!(valid >> i & 1)) raw[i] = Piece<G, CPL>{};
            }
            if constexpr (sizeof(G) == 2) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    __nv_bfloat162 lo = __float2bfloat162_rn(0.f), hi = lo;
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const __nv_bfloat162 y = reinterpret_cast<const __nv_bfloat162*>(raw[i].x)[p];
                        lo = __hmin2(lo, y);
                        hi = __hmax2(hi, y);
                    }
                    least[p] = __bfloat1622float2(lo);
                    most[p] = __bfloat1622float2(hi);
                }
            } else {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    least[p] = most[p] = splat(0.f);
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const float2 y = two(raw[i], p);
                        least[p] = make_float2(fminf(least[p].x, y.x), fminf(least[p].y, y.y));
                        most[p] = make_float2(fmaxf(most[p].x, y.x), fmaxf(most[p].y, y.y));
                    }
                }
            }
            bool far = false, big = false, fx[NP], fy[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                fx[p] = least[p].x < kLow || most[p].x > 0.f;
                fy[p] = least[p].y < kLow || most[p].y > 0.f;
                w[p] = make_float2(fx[p] ? 0.f : 1.f, fy[p] ? 0.f : 1.f);
                far |= fx[p] || fy[p];
                big |= fminf(least[p].x, least[p].y) < -kBig || fmaxf(most[p].x, most[p].y) > kBig;
            }
            auto all = [&](auto f) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const float2 g = two(raw[i], p);
                        sum[p] = add2(sum[p], g);
                        v[i][p] = f(p, g);
                    }
            };
            auto either = [&](int p, float2 y, float2 a) { return make_float2(fx[p] ? a.x : y.x, fy[p] ? a.y : y.y); };
            if (!__any_sync(kFull, far)) all([&](int p, float2 g) { return mild(g); });
            else if (!__any_sync(kFull, big)) all([&](int p, float2 g) { return either(p, mild(g), strong(g)); });
            else all([&](int p, float2 g) { return either(p, mild(g), make_float2(expf(g.x), expf(g.y))); });
        }
    }
    __device__ __forceinline__ float2 at(int i, int p) const {
        if constexpr (SHARED) return splat(__shfl_sync(kFull, v[0][0].x, i));
        else return v[i][p];
    }
    __device__ __forceinline__ float2 keep(int p) const { return w[SHARED ? 0 : p]; }
    __device__ __forceinline__ float2 total(int p) const { return sum[SHARED ? 0 : p]; }
};

struct Tiles {
    int cpl, rows, n_slabs, n_time;
};
// Runs of `most` rows where that makes two tiles for every SM (152), else of 8 rows, so that small calls spread (us, forward and
// gradient, 1024 channels: 640 rows 8.5 and 9.0 in runs of 8, 9.1 and 10.5 in runs of 16; 2432 rows 14.2 and 16.3, 12.7 and 13.7).
inline Tiles tiles(const RecDims& R, int most) {
    Tiles t;
    t.cpl = R.gate_dim == 128 ? 4 : 2;
    t.n_slabs = (R.channels + 32 * t.cpl - 1) / (32 * t.cpl);
    auto times = [&](int rows) { return std::max<int64_t>(1, (R.total + (int64_t)rows * kWarps - 1) / (rows * kWarps)); };
    t.rows = times(most) * t.n_slabs >= 304 ? most : 8;
    t.n_time = (int)times(t.rows);
    return t;
}
inline int most_rows(const RecDims& R, bool f32, bool backward) {
    if (R.gate_dim == 128) return backward ? 8 : 16;
    if (R.gate_dim == 64) return f32 || backward ? 16 : 32;
    return f32 && backward ? 8 : 16;
}
inline size_t tile_bytes(const Tiles& t) { return t.n_time == 1 ? 0 : (size_t)t.n_time * t.n_slabs * 32 * t.cpl * 24; }

inline Carry carry_of(char* ws, const Tiles& t) {
    Carry c;
    c.ticket = reinterpret_cast<int*>(ws);
    c.state = reinterpret_cast<uint64_t*>(ws + 256);
    c.map = c.state + (size_t)t.n_time * t.n_slabs * 32 * t.cpl;
    return c;
}
inline cudaError_t clear(char* ws, const Tiles& t, cudaStream_t st) {
    return t.n_time == 1 ? cudaSuccess : cudaMemsetAsync(ws, 0, 256 + tile_bytes(t), st);
}
// Pairs (fours) of channels at once where every row starts on their boundary.
template <typename T, typename G>
bool pairs(const RecDims& R, const T* x, const G* g, const T* y, const T* z, const G* w, int cpl) {
    const uintptr_t a = (uintptr_t)x | (uintptr_t)y | (uintptr_t)z;
    if (R.channels % cpl || R.sx % cpl || a % (cpl * sizeof(T))) return false;
    return R.gate_dim > 1 || !(R.sg % cpl || ((uintptr_t)g | (uintptr_t)w) % (cpl * sizeof(G)));
}
template <template <typename, typename, int, bool, bool, int> class K, typename T, typename G, int MOST1, int MOST, int MOST4, typename... A>
cudaError_t choose(const RecDims& R, const Tiles& t, bool vec, cudaStream_t st, A... a) {
    if (R.gate_dim == 128)
        return t.rows == 8 ? (vec ? K<T, G, 4, true, true, 8>::run(t, st, a...) : K<T, G, 4, true, false, 8>::run(t, st, a...))
                           : (vec ? K<T, G, 4, true, true, MOST4>::run(t, st, a...) : K<T, G, 4, true, false, MOST4>::run(t, st, a...));
    if (R.gate_dim == 64)
        return t.rows == 8 ? (vec ? K<T, G, 2, true, true, 8>::run(t, st, a...) : K<T, G, 2, true, false, 8>::run(t, st, a...))
                           : (vec ? K<T, G, 2, true, true, MOST>::run(t, st, a...) : K<T, G, 2, true, false, MOST>::run(t, st, a...));
    return t.rows == 8 ? (vec ? K<T, G, 2, false, true, 8>::run(t, st, a...) : K<T, G, 2, false, false, 8>::run(t, st, a...))
                       : (vec ? K<T, G, 2, false, true, MOST1>::run(t, st, a...) : K<T, G, 2, false, false, MOST1>::run(t, st, a...));
}

}  // namespace

}  // namespace hla
