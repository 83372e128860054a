// Gated linear recurrence over packed sequences, its gradient, and its step.
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
// The state in front of a tile: every tile publishes (A, B) and, once it knows
// it, the state behind it.  A tile looks at up to eight tiles before it; the
// nearest with a state is carried forward by the (A, B) of those between, tile
// after tile.  That is what each of those tiles does itself, rounding for
// rounding, so that results do not depend on which of them was found.  Tiles
// are handed out in order of time, so that those waited for are running.  Every
// word carries its own flag: no fences, and one trip through L2 per look.
//
// A gate near 1 enters as exp(g) - 1: a state that decays slowly (|g| of 1e-3
// and less, thousands of rows) keeps its bits, where a rounded exp(g) would be
// off by up to 2^-25 in every row, the same way for the same gate.  Below 1/2 it
// enters as exp(g), so that a closed gate leaves nothing of the state, not even
// a rounding.
//
// The gradient runs the tiles from the last to the first.  States in front of
// its rows come from those that the forward pass kept every 64 rows.
#include <algorithm>

#include "layer.cuh"

namespace hla {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kLook = kWarps;       // tiles before a tile that it looks at, one per warp
constexpr int kPolls = 1 << 20;     // looks at a tile that has nothing yet (about 0.7 us each)
constexpr unsigned kFull = 0xffffffffu;

// A gate as v: exp(g) - 1 (negative) for -0.69 < g < 0, else exp(g).  g = k ln 2 + r, |r| <= ln 2 / 2, and the exponential
// series of r to r^7 (the rest is below 2^-25 of it).
__device__ __forceinline__ float gate(float g) {
    float k = rintf(g * 1.44269504f);
    float r = fmaf(k, -0.693145752f, g);   // ln 2 in two parts, the first with 16 bits: k times it is exact
    r = fmaf(k, -1.42860677e-6f, r);
    float p = 1.f / 5040.f;
    p = fmaf(p, r, 1.f / 720.f);
    p = fmaf(p, r, 1.f / 120.f);
    p = fmaf(p, r, 1.f / 24.f);
    p = fmaf(p, r, 1.f / 6.f);
    p = fmaf(p, r, 0.5f);
    p = fmaf(p, r * r, r);
    const bool big = k > 127.f;
    const float s = __int_as_float(((int)(big ? 127.f : k) + 127) << 23);
    const float e = fmaf(s, p, s - 1.f);
    float a = fmaf(s, p, s);
    a = big ? (g > 88.8f ? __int_as_float(0x7f800000) : a * 2.f) : a;
    a = g < -87.f ? 0.f : a;  // below the smallest normal number
    return e < 0.f && e > -0.5f ? e : a;
}
// exp(g) h + x
__device__ __forceinline__ float through(float v, float h, float x) { return fmaf(v, h, x) + (v < 0.f ? h : 0.f); }
// exp(g) h
__device__ __forceinline__ float times(float v, float h) { return fmaf(v, h, v < 0.f ? h : 0.f); }

__device__ __forceinline__ void put_word(uint64_t* p, float v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"((uint64_t)1 << 32 | __float_as_uint(v)) : "memory");
}
__device__ __forceinline__ bool get_word(const uint64_t* p, float* v) {
    uint64_t w;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
    *v = __uint_as_float((uint32_t)w);
    return w >> 32;
}

// Carries between tiles: per tile and channel the state behind it, and its (A, B).
struct Carry {
    uint64_t* state;
    uint64_t* map;  // two words each
    int* ticket;
};

// A tile of rows by channels, as one lane sees it.
template <typename T, int CPL, bool VEC>
struct Lane {
    int c[CPL];   // channels
    bool on[CPL];
    __device__ __forceinline__ Lane(int slab, int channels) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            c[j] = slab * 32 * CPL + (VEC ? lane * CPL + j : j * 32 + lane);
            on[j] = c[j] < channels;
        }
    }
    template <typename U>
    __device__ __forceinline__ void load(const U* row, U (&v)[CPL]) const {
        if constexpr (VEC) {
            if (on[0]) *reinterpret_cast<Piece<U, CPL>*>(v) = *reinterpret_cast<const Piece<U, CPL>*>(row + c[0]);
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                if (on[j]) v[j] = row[c[j]];
        }
    }
    template <typename U>
    __device__ __forceinline__ void store(U* row, const float (&f)[CPL]) const {
        Piece<U, CPL> v;
#pragma unroll
        for (int j = 0; j < CPL; ++j) v.x[j] = from_f32<U>(f[j]);
        if constexpr (VEC) {
            if (on[0]) *reinterpret_cast<Piece<U, CPL>*>(row + c[0]) = v;
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                if (on[j]) row[c[j]] = v.x[j];
        }
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
template <int CPL>
__device__ __forceinline__ void look_back(const Carry& S, int k, int n_slabs, int slab, float (&c)[CPL], int32_t* err) {
    __shared__ float pa[kLook][32 * CPL], pb[kLook][32 * CPL];
    __shared__ int status[kLook];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pred = k - 1 - warp;
    int have = 0, polls = 0, m;
    bool late = false;
    for (;;) {
        if (pred < 0) {
            if (!have)
#pragma unroll
                for (int j = 0; j < CPL; ++j) pb[warp][lane * CPL + j] = 0.f;
            have = 2;
        } else if (have < 2 && !late) {
            const int64_t at = ((int64_t)pred * n_slabs + slab) * 32 * CPL + lane * CPL;
            do {
                float s[CPL], a[CPL], b[CPL];
                bool is = true, has = true;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    is &= get_word(S.state + at + j, &s[j]);
                    if (!have) {
                        has &= get_word(S.map + 2 * (at + j), &a[j]);
                        has &= get_word(S.map + 2 * (at + j) + 1, &b[j]);
                    }
                }
                if (__all_sync(kFull, is)) {
#pragma unroll
                    for (int j = 0; j < CPL; ++j) pb[warp][lane * CPL + j] = s[j];
                    have = 2;
                } else if (!have && __all_sync(kFull, has)) {
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        pa[warp][lane * CPL + j] = a[j];
                        pb[warp][lane * CPL + j] = b[j];
                    }
                    have = 1;
                }
                late = ++polls > kPolls;
            } while (!have && !late);
        }
        if (lane == 0) status[warp] = late && have < 2 ? 3 : have;
        __syncthreads();
        bool gone = false;
        m = kLook;
#pragma unroll
        for (int w = kLook - 1; w >= 0; --w) {
            const int s = status[w];
            gone |= s == 3;
            m = s == 2 ? w : m;
        }
        if (m < kLook) {
            bool fit = true;  // every tile between has its (A, B), unless a wait ran out
            for (int w = 0; w < m; ++w) fit &= status[w] == 1;
            if (fit) break;
        }
        if (gone) {
            m = -1;
            break;
        }
        __syncthreads();  // before status is written again
    }
    if (m < 0) {
        if (threadIdx.x == 0) atomicExch(err, kErrTimeout);
#pragma unroll
        for (int j = 0; j < CPL; ++j) c[j] = 0.f;
        return;
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j) c[j] = pb[m][lane * CPL + j];
    for (int w = m - 1; w >= 0; --w)
#pragma unroll
        for (int j = 0; j < CPL; ++j) c[j] = fmaf(pa[w][lane * CPL + j], c[j], pb[w][lane * CPL + j]);
}

// The warps' (A, B) of a tile, in the order in which the state passes them.
template <int CPL>
struct Runs {
    float a[kWarps][32 * CPL], b[kWarps][32 * CPL];
    int cut[kWarps];  // the state does not pass this run
    __device__ __forceinline__ void put(int w, const float (&A)[CPL], const float (&B)[CPL], bool is_cut) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            a[w][lane * CPL + j] = A[j];
            b[w][lane * CPL + j] = B[j];
        }
        if (lane == 0) cut[w] = is_cut;
    }
    __device__ __forceinline__ void pass(int w, float (&c)[CPL]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float y = b[w][lane * CPL + j];
            c[j] = cut[w] ? y : fmaf(a[w][lane * CPL + j], c[j], y);
        }
    }
};

// Publishes tile k's map (or state, where a run of it is cut), takes the state in front of it, publishes the one behind.
template <int CPL>
__device__ __forceinline__ void tile_carry(const Carry& S, const Runs<CPL>& runs, int k, int n_time, int n_slabs, int slab,
                                           float (&c)[CPL], int32_t* err) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < CPL; ++j) c[j] = 0.f;
    if (n_time == 1) return;
    float A[CPL], B[CPL];
    bool cut = false;
    const int64_t at = ((int64_t)k * n_slabs + slab) * 32 * CPL + lane * CPL;
    if (threadIdx.x < 32 && k + 1 < n_time) {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            A[j] = 1.f;
            B[j] = 0.f;
        }
        for (int w = 0; w < kWarps; ++w) {
            runs.pass(w, B);
            cut |= runs.cut[w];
#pragma unroll
            for (int j = 0; j < CPL; ++j) A[j] *= runs.a[w][lane * CPL + j];
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            if (cut) {
                put_word(S.state + at + j, B[j]);
            } else {
                put_word(S.map + 2 * (at + j), A[j]);
                put_word(S.map + 2 * (at + j) + 1, B[j]);
            }
        }
    }
    look_back<CPL>(S, k, n_slabs, slab, c, err);
    if (threadIdx.x < 32 && k + 1 < n_time && !cut)
#pragma unroll
        for (int j = 0; j < CPL; ++j) put_word(S.state + at + j, fmaf(A[j], c[j], B[j]));
}

// A warp's gates (as gate() gives them): per row and channel, or (SHARED) row i's in lane i.
template <typename G, int CPL, bool SHARED, int ROWS>
struct Gates {
    float e[SHARED ? 1 : ROWS][SHARED ? 1 : CPL];
    __device__ __forceinline__ float at(int i, int j) const {
        if constexpr (SHARED) return __shfl_sync(kFull, e[0][0], i);
        else return e[i][j];
    }
};

template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
recurrence_kernel(const RecDims R, const G* __restrict__ g, const T* __restrict__ x, const float* h0,
                  const int32_t* __restrict__ cu, T* __restrict__ out, float* h_last, float* __restrict__ states,
                  const Carry S, int n_time, int n_slabs, int32_t* err) {
    __shared__ Runs<CPL> runs;
    const int tile = take_tile(S.ticket, n_time), k = tile / n_slabs, slab = tile - k * n_slabs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)k * kWarps + warp) * ROWS;
    const int n = (int)clamp_i64(R.total - t0, 0, ROWS);
    const Lane<T, CPL, VEC> at(slab, R.channels);
    T xs[ROWS][CPL];
    G gs[SHARED ? 1 : ROWS][SHARED ? 1 : CPL];
    const T* xr = x + t0 * R.sx;
    const G* gr = g + t0 * R.sg;
    if constexpr (SHARED) {
        if (lane < n) gs[0][0] = gr[(int64_t)lane * R.sg + slab];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (i < n) {
            at.load(xr + (int64_t)i * R.sx, xs[i]);
            if constexpr (!SHARED) at.load(gr + (int64_t)i * R.sg, gs[i]);
        }
    const Rows rows(cu, R, t0, ROWS);
    if (tile == 0) check_table(cu, R, err);
    Gates<G, CPL, SHARED, ROWS> e;
    if constexpr (SHARED) {
        e.e[0][0] = rows.valid >> lane & 1 ? gate(to_f32(gs[0][0])) : 1.f;
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < CPL; ++j) e.e[i][j] = rows.valid >> i & 1 && at.on[j] ? gate(to_f32(gs[i][j])) : 1.f;
    }
    auto in = [&](int i, int j) { return rows.valid >> i & 1 && at.on[j] ? to_f32(xs[i][j]) : 0.f; };
    auto start = [&](int i, float (&h)[CPL]) {  // the state in front of a sequence's first row
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int j = 0; j < CPL; ++j) h[j] = h0 && at.on[j] ? h0[(int64_t)s * R.channels + at.c[j]] : 0.f;
    };
    float A[CPL], B[CPL], kept[CPL];  // kept: h0 of the run's last sequence (another tile may end it, in h0's place)
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        A[j] = 1.f;
        B[j] = kept[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (rows.first >> i & 1) {
            start(i, kept);
#pragma unroll
            for (int j = 0; j < CPL; ++j) B[j] = kept[j];
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float y = e.at(i, j);
            B[j] = through(y, B[j], in(i, j));
            A[j] = times(y, A[j]);
        }
    }
    runs.put(warp, A, B, rows.first != 0);
    __syncthreads();
    float h[CPL];
    tile_carry<CPL>(S, runs, k, n_time, n_slabs, slab, h, err);
    for (int w = 0; w < warp; ++w) runs.pass(w, h);
    if (states && t0 % kStateRows == 0 && t0 < R.total) at.store(states + t0 / kStateRows * R.channels, h);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (rows.first >> i & 1) {
            if (rows.first >> i == 1) {
#pragma unroll
                for (int j = 0; j < CPL; ++j) h[j] = kept[j];
            } else {
                start(i, h);
            }
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) h[j] = through(e.at(i, j), h[j], in(i, j));
        if (rows.valid >> i & 1) at.store(out + (t0 + i) * R.channels, h);
        if (rows.last >> i & 1 && h_last) {
            const int s = __shfl_sync(kFull, rows.seq, i);
            at.store(h_last + (int64_t)s * R.channels, h);
        }
    }
    if (!h_last) return;
    for (int s = k * kWarps + warp; s < R.n_seqs; s += n_time * kWarps) {  // sequences without rows
        int64_t a, m;
        seq_range(cu, s, R.total, &a, &m);
        if (m > 0) continue;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            if (!at.on[j]) continue;
            const int64_t p = (int64_t)s * R.channels + at.c[j];
            h_last[p] = h0 ? h0[p] : 0.f;
        }
    }
}

// Sum over the warp's 32 lanes of v[i], for every i: row i's sum comes back in lane i of the result.
template <int ROWS>
__device__ __forceinline__ float sums_to_lanes(float (&v)[ROWS]) {
    const int lane = threadIdx.x & 31;
    // halves: a lane gives away the rows of its other half and keeps the sums of its own
#pragma unroll
    for (int n = ROWS / 2; n; n >>= 1) {
        const bool hi = lane & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(kFull, give, n);
        }
    }
#pragma unroll
    for (int o = ROWS; o < 32; o <<= 1) v[0] += __shfl_xor_sync(kFull, v[0], o);
    return v[0];
}

template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
recurrence_backward_kernel(const RecDims R, const G* __restrict__ g, const T* __restrict__ x, const float* h0,
                           const float* __restrict__ states, const int32_t* __restrict__ cu, const T* __restrict__ dout,
                           const float* dh_last, G* __restrict__ dg, T* __restrict__ dx, float* dh0, const Carry S,
                           int n_time, int n_slabs, int32_t* err) {
    __shared__ Runs<CPL> ahead, back;  // forward in time; backward, in the order in which tiles are handed out
    const int tile = take_tile(S.ticket, n_time), k = tile / n_slabs, slab = tile - k * n_slabs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)(n_time - 1 - k) * kWarps + warp) * ROWS;
    const int n = (int)clamp_i64(R.total - t0, 0, ROWS);
    const Lane<T, CPL, VEC> at(slab, R.channels);
    T xs[ROWS][CPL], ds[ROWS][CPL];
    G gs[SHARED ? 1 : ROWS][SHARED ? 1 : CPL];
    const T* xr = x + t0 * R.sx;
    const T* dr = dout + t0 * R.channels;
    const G* gr = g + t0 * R.sg;
    if constexpr (SHARED) {
        if (lane < n) gs[0][0] = gr[(int64_t)lane * R.sg + slab];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (i < n) {
            at.load(xr + (int64_t)i * R.sx, xs[i]);
            at.load(dr + (int64_t)i * R.channels, ds[i]);
            if constexpr (!SHARED) at.load(gr + (int64_t)i * R.sg, gs[i]);
        }
    constexpr int kPer = kStateRows / ROWS;  // runs between kept states
    float h[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) h[j] = n > 0 && at.on[j] ? states[t0 / kStateRows * R.channels + at.c[j]] : 0.f;
    const Rows rows(cu, R, t0, ROWS);
    if (tile == 0) check_table(cu, R, err);
    Gates<G, CPL, SHARED, ROWS> e;
    if constexpr (SHARED) {
        e.e[0][0] = rows.valid >> lane & 1 ? gate(to_f32(gs[0][0])) : 1.f;
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < CPL; ++j) e.e[i][j] = rows.valid >> i & 1 && at.on[j] ? gate(to_f32(gs[i][j])) : 1.f;
    }
    auto in = [&](int i, int j) { return rows.valid >> i & 1 && at.on[j] ? to_f32(xs[i][j]) : 0.f; };
    auto grad = [&](int i, int j) { return rows.valid >> i & 1 && at.on[j] ? to_f32(ds[i][j]) : 0.f; };
    auto start = [&](int i, float (&v)[CPL]) {
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int j = 0; j < CPL; ++j) v[j] = h0 && at.on[j] ? h0[(int64_t)s * R.channels + at.c[j]] : 0.f;
    };
    auto end = [&](int i, float (&v)[CPL]) {  // what comes from behind a sequence's last row
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int j = 0; j < CPL; ++j) v[j] = dh_last && at.on[j] ? dh_last[(int64_t)s * R.channels + at.c[j]] : 0.f;
    };
    float A[CPL], B[CPL], M[CPL], kept[CPL];  // kept: dh_last of the run's first sequence (another tile may write dh0 there)
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        A[j] = 1.f;
        B[j] = M[j] = kept[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (rows.first >> i & 1) start(i, B);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float y = e.at(i, j);
            B[j] = through(y, B[j], in(i, j));
            A[j] = times(y, A[j]);
        }
    }
#pragma unroll
    for (int i = ROWS - 1; i >= 0; --i) {  // m_t = exp(g_t) l_t, l_t = dout_t + m_{t+1}
        if (rows.last >> i & 1) {
            end(i, kept);
#pragma unroll
            for (int j = 0; j < CPL; ++j) M[j] = kept[j];
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float l = grad(i, j) + M[j];
            M[j] = times(e.at(i, j), l);
        }
    }
    ahead.put(warp, A, B, rows.first != 0);
    back.put(kWarps - 1 - warp, A, M, rows.last != 0);
    __syncthreads();
    for (int w = warp / kPer * kPer; w < warp; ++w) ahead.pass(w, h);
    float u[ROWS][CPL];  // exp(g_t) h_{t-1}
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (rows.first >> i & 1) start(i, h);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float y = e.at(i, j);
            u[i][j] = times(y, h[j]);
            h[j] = through(y, h[j], in(i, j));
        }
    }
    float m[CPL];
    tile_carry<CPL>(S, back, k, n_time, n_slabs, slab, m, err);
    for (int w = 0; w < kWarps - 1 - warp; ++w) back.pass(w, m);
#pragma unroll
    for (int i = ROWS - 1; i >= 0; --i) {
        if (rows.last >> i & 1) {
            if ((rows.last & ((1u << i) - 1)) == 0) {
#pragma unroll
                for (int j = 0; j < CPL; ++j) m[j] = kept[j];
            } else {
                end(i, m);
            }
        }
        float l[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            l[j] = grad(i, j) + m[j];
            m[j] = times(e.at(i, j), l[j]);
            u[i][j] *= l[j];
        }
        if (rows.valid >> i & 1) {
            at.store(dx + (t0 + i) * R.channels, l);
            if constexpr (!SHARED) at.store(dg + (t0 + i) * R.channels, u[i]);
        }
        if (rows.first >> i & 1 && dh0) {
            const int s = __shfl_sync(kFull, rows.seq, i);
            at.store(dh0 + (int64_t)s * R.channels, m);
        }
    }
    if constexpr (SHARED) {
        float v[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            v[i] = u[i][0];
#pragma unroll
            for (int j = 1; j < CPL; ++j) v[i] += u[i][j];
        }
        const float y = sums_to_lanes(v);
        if (lane < ROWS && rows.valid >> lane & 1)
            dg[(t0 + lane) * (R.channels / R.gate_dim) + slab] = from_f32<G>(y);
    }
    if (!dh0) return;
    for (int s = k * kWarps + warp; s < R.n_seqs; s += n_time * kWarps) {
        int64_t a, len;
        seq_range(cu, s, R.total, &a, &len);
        if (len > 0) continue;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            if (!at.on[j]) continue;
            const int64_t p = (int64_t)s * R.channels + at.c[j];
            dh0[p] = dh_last ? dh_last[p] : 0.f;
        }
    }
}

// One row per sequence: the state in place.  A thread takes V channels of a row.
template <typename T, typename G, int V>
__global__ void __launch_bounds__(256)
recurrence_step_kernel(const RecDims R, const G* __restrict__ g, const T* __restrict__ x, float* h, T* __restrict__ out) {
    const int per = R.channels / V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= R.total * per) return;
    const int64_t row = i / per;
    const int c = (int)(i - row * per) * V;
    using P = Piece<T, V>;
    using H = Piece<float, V>;
    const P a = *reinterpret_cast<const P*>(x + row * R.sx + c);
    H s = *reinterpret_cast<const H*>(h + row * R.channels + c);
    P o;
    float e[V];
    if (R.gate_dim > 1) {
        e[0] = gate(to_f32(g[row * R.sg + c / R.gate_dim]));
#pragma unroll
        for (int j = 1; j < V; ++j) e[j] = e[0];
    } else {
        const Piece<G, V> y = *reinterpret_cast<const Piece<G, V>*>(g + row * R.sg + c);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = gate(to_f32(y.x[j]));
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s.x[j] = through(e[j], s.x[j], to_f32(a.x[j]));
        o.x[j] = from_f32<T>(s.x[j]);
    }
    *reinterpret_cast<H*>(h + row * R.channels + c) = s;
    *reinterpret_cast<P*>(out + row * R.channels + c) = o;
}

struct Tiles {
    int cpl, rows, n_slabs, n_time;
};
// Runs of `most` rows where that makes two tiles for every SM (152), else of 8 rows, so that small calls spread.
Tiles tiles(const RecDims& R, int most) {
    Tiles t;
    t.cpl = R.gate_dim == 128 ? 4 : 2;
    t.n_slabs = (R.channels + 32 * t.cpl - 1) / (32 * t.cpl);
    auto times = [&](int rows) { return std::max<int64_t>(1, (R.total + (int64_t)rows * kWarps - 1) / (rows * kWarps)); };
    t.rows = times(most) * t.n_slabs >= 304 ? most : 8;
    t.n_time = (int)times(t.rows);
    return t;
}
int most_rows(const RecDims& R, bool f32, bool backward) {
    if (R.gate_dim == 128) return backward ? 8 : 16;
    return f32 || backward ? 16 : 32;
}
size_t tile_bytes(const Tiles& t) { return t.n_time == 1 ? 0 : (size_t)t.n_time * t.n_slabs * 32 * t.cpl * 24; }

Carry carry_of(char* ws, const Tiles& t) {
    Carry c;
    c.ticket = reinterpret_cast<int*>(ws);
    c.state = reinterpret_cast<uint64_t*>(ws + 256);
    c.map = c.state + (size_t)t.n_time * t.n_slabs * 32 * t.cpl;
    return c;
}
cudaError_t clear(char* ws, const Tiles& t, cudaStream_t st) {
    return t.n_time == 1 ? cudaSuccess : cudaMemsetAsync(ws, 0, 256 + tile_bytes(t), st);
}

}  // namespace

size_t recurrence_carry_bytes(const RecDims& R, bool f32) {
    size_t most = 0;
    for (int back = 0; back < 2; ++back) {
        // the tiles of this size, and the most that a smaller one can have (fewer than 304 of the larger runs, in runs of 8)
        const Tiles t = tiles(R, most_rows(R, f32, back));
        RecDims s = R;
        s.total = std::min<int64_t>(R.total, (int64_t)(304 / t.n_slabs + 1) * most_rows(R, f32, back) * kWarps);
        Tiles u = t;
        u.n_time = (int)((s.total + 8 * kWarps - 1) / (8 * kWarps));
        most = std::max({most, tile_bytes(t), tile_bytes(u)});
    }
    return most ? 256 + most : 0;
}

namespace {
template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
struct Forward {
    template <typename... A> static cudaError_t run(const Tiles& t, cudaStream_t st, A... a) {
        recurrence_kernel<T, G, CPL, SHARED, VEC, ROWS><<<(unsigned)(t.n_time * t.n_slabs), kThreads, 0, st>>>(a...);
        return cudaGetLastError();
    }
};
template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
struct Backward {
    template <typename... A> static cudaError_t run(const Tiles& t, cudaStream_t st, A... a) {
        recurrence_backward_kernel<T, G, CPL, SHARED, VEC, ROWS><<<(unsigned)(t.n_time * t.n_slabs), kThreads, 0, st>>>(a...);
        return cudaGetLastError();
    }
};
// Pairs (fours) of channels at once where every row starts on their boundary, for the state's fp32 as well.
template <typename T, typename G>
bool pairs(const RecDims& R, const T* x, const G* g, const T* y, const T* z, const G* w, int cpl) {
    const uintptr_t a = (uintptr_t)x | (uintptr_t)y | (uintptr_t)z;
    if (R.channels % cpl || R.sx % cpl || a % (cpl * sizeof(T))) return false;
    return R.gate_dim > 1 || !(R.sg % cpl || ((uintptr_t)g | (uintptr_t)w) % (cpl * sizeof(G)));
}
template <template <typename, typename, int, bool, bool, int> class K, typename T, typename G, int MOST, int MOST4, typename... A>
cudaError_t choose(const RecDims& R, const Tiles& t, bool vec, cudaStream_t st, A... a) {
    if (R.gate_dim == 128)
        return t.rows == 8 ? (vec ? K<T, G, 4, true, true, 8>::run(t, st, a...) : K<T, G, 4, true, false, 8>::run(t, st, a...))
                           : (vec ? K<T, G, 4, true, true, MOST4>::run(t, st, a...) : K<T, G, 4, true, false, MOST4>::run(t, st, a...));
    if (R.gate_dim == 64)
        return t.rows == 8 ? (vec ? K<T, G, 2, true, true, 8>::run(t, st, a...) : K<T, G, 2, true, false, 8>::run(t, st, a...))
                           : (vec ? K<T, G, 2, true, true, MOST>::run(t, st, a...) : K<T, G, 2, true, false, MOST>::run(t, st, a...));
    return t.rows == 8 ? (vec ? K<T, G, 2, false, true, 8>::run(t, st, a...) : K<T, G, 2, false, false, 8>::run(t, st, a...))
                       : (vec ? K<T, G, 2, false, true, MOST>::run(t, st, a...) : K<T, G, 2, false, false, MOST>::run(t, st, a...));
}
}  // namespace

template <typename T, typename G>
cudaError_t launch_recurrence(const RecDims& R, const G* g, const T* x, const float* h0, const int32_t* cu, T* out,
                              float* h_last, float* states, char* carry, int32_t* err, cudaStream_t st) {
    constexpr bool f32 = sizeof(T) == 4;
    const Tiles t = tiles(R, most_rows(R, f32, false));
    cudaError_t e = clear(carry, t, st);
    if (e != cudaSuccess) return e;
    return choose<Forward, T, G, f32 ? 16 : 32, 16>(R, t, pairs<T, G>(R, x, g, out, out, g, t.cpl), st, R, g, x, h0, cu,
                                                    out, h_last, states, carry_of(carry, t), t.n_time, t.n_slabs, err);
}

template <typename T, typename G>
cudaError_t launch_recurrence_backward(const RecDims& R, const G* g, const T* x, const float* h0, const float* states,
                                       const int32_t* cu, const T* dout, const float* dh_last, G* dg, T* dx,
                                       float* dh0, char* carry, int32_t* err, cudaStream_t st) {
    constexpr bool f32 = sizeof(T) == 4;
    const Tiles t = tiles(R, most_rows(R, f32, true));
    cudaError_t e = clear(carry, t, st);
    if (e != cudaSuccess) return e;
    return choose<Backward, T, G, 16, 8>(R, t, pairs<T, G>(R, x, g, dout, dx, dg, t.cpl), st, R, g, x, h0, states, cu,
                                         dout, dh_last, dg, dx, dh0, carry_of(carry, t), t.n_time, t.n_slabs, err);
}

template <typename T, typename G>
cudaError_t launch_recurrence_step(const RecDims& R, const G* g, const T* x, float* h, T* out, cudaStream_t st) {
    if (R.total == 0) return cudaSuccess;
    const bool vec = R.channels % 4 == 0 && R.sx % 4 == 0 && (uintptr_t)h % 16 == 0 &&
                     ((uintptr_t)x | (uintptr_t)out) % (4 * sizeof(T)) == 0 &&
                     (R.gate_dim > 1 || (R.sg % 4 == 0 && (uintptr_t)g % (4 * sizeof(G)) == 0));
    const int64_t n = R.total * (R.channels / (vec ? 4 : 1)), blocks = (n + 255) / 256;
    if (vec) recurrence_step_kernel<T, G, 4><<<(unsigned)blocks, 256, 0, st>>>(R, g, x, h, out);
    else recurrence_step_kernel<T, G, 1><<<(unsigned)blocks, 256, 0, st>>>(R, g, x, h, out);
    return cudaGetLastError();
}

#define HLA_RECURRENCE(T, G)                                                                                          \
    template cudaError_t launch_recurrence<T, G>(const RecDims&, const G*, const T*, const float*, const int32_t*, T*, \
                                                 float*, float*, char*, int32_t*, cudaStream_t);                      \
    template cudaError_t launch_recurrence_backward<T, G>(const RecDims&, const G*, const T*, const float*,           \
                                                          const float*, const int32_t*, const T*, const float*, G*,   \
                                                          T*, float*, char*, int32_t*, cudaStream_t);                 \
    template cudaError_t launch_recurrence_step<T, G>(const RecDims&, const G*, const T*, float*, T*, cudaStream_t);
HLA_RECURRENCE(float, float)
HLA_RECURRENCE(float, __nv_bfloat16)
HLA_RECURRENCE(__nv_bfloat16, float)
HLA_RECURRENCE(__nv_bfloat16, __nv_bfloat16)

}  // namespace hla
