// Gradient of the gated linear recurrence.
//
// Measured: 16309 rows of 4096 bf16 channels, a gate per channel, 192 us (4.7 TB/s); 16384 rows of 2048, a gate per 64, 76 us
// (2.7 TB/s; 83 with two blocks an SM, 87 with runs of 8 rows): a row's gate goes from its lane to all four times, and the
// gate's gradient is summed over the warp; and at the 80 registers of three blocks an SM 108 to 164 bytes a thread are
// spilled (a gate per 128: 224 to 360), which costs less than the third block gives.
#include "recurrence.cuh"

namespace hla {

namespace {

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
__global__ void __launch_bounds__(kThreads, SHARED && sizeof(T) == 2 ? 3 : 2)
recurrence_backward_kernel(const RecDims R, const G* __restrict__ g, const T* __restrict__ x, const float* h0,
                           const float* __restrict__ states, const int32_t* __restrict__ cu, const T* __restrict__ dout,
                           const float* dh_last, G* __restrict__ dg, T* __restrict__ dx, float* dh0, const Carry S,
                           int n_time, int n_slabs, int32_t* err) {
    constexpr int NP = CPL / 2;
    __shared__ Sums<NP> sums;
    __shared__ Runs<NP> ahead, back;  // forward in time; backward, in the order in which tiles are handed out
    const int tile = take_tile(S.ticket, n_time), k = tile / n_slabs, slab = tile - k * n_slabs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)(n_time - 1 - k) * kWarps + warp) * ROWS;
    const int n = (int)clamp_i64(R.total - t0, 0, ROWS);
    const Lane<CPL, VEC> at(slab, R.channels);
    Piece<T, CPL> xs[ROWS], ds[ROWS];
    Gates<G, CPL, SHARED, VEC, ROWS> e;
    const T* xr = x + t0 * R.sx;
    const T* dr = dout + t0 * R.channels;
    const uint32_t sx = (uint32_t)R.sx, sg = (uint32_t)R.sg, so = (uint32_t)R.channels;
    if (n == ROWS) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            xs[i] = at.load(xr + (uint64_t)i * sx);
            ds[i] = at.load(dr + (uint64_t)i * so);
        }
        e.template load<true>(at, g + t0 * R.sg, sg, slab, n);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            xs[i] = i < n ? at.load(xr + (uint64_t)i * sx) : Piece<T, CPL>{};
            ds[i] = i < n ? at.load(dr + (uint64_t)i * so) : Piece<T, CPL>{};
        }
        e.template load<false>(at, g + t0 * R.sg, sg, slab, n);
    }
    constexpr int kPer = kStateRows / ROWS;  // runs between kept states
    float2 h[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) h[p] = splat(0.f);
    if (n > 0) at.load_pairs(states + t0 / kStateRows * R.channels, h);
    const Rows rows(cu, R, t0, ROWS);
    if (tile == 0) check_table(cu, R, err);
    const bool edge = (rows.first | rows.last) != 0 || rows.valid != (1u << ROWS) - 1;
    auto start = [&](int i, float2 (&v)[NP]) {
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int p = 0; p < NP; ++p) v[p] = splat(0.f);
        if (h0) at.load_pairs(h0 + (int64_t)s * R.channels, v);
    };
    auto end = [&](int i, float2 (&v)[NP]) {  // what comes from behind a sequence's last row
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int p = 0; p < NP; ++p) v[p] = splat(0.f);
        if (dh_last) at.load_pairs(dh_last + (int64_t)s * R.channels, v);
    };
    // m_t = exp(g_t) l_t, l_t = dout_t + m_{t+1}
    float2 B[NP], M[NP], kept[NP];  // kept: dh_last of the run's first sequence (another tile may write dh0 there)
#pragma unroll
    for (int p = 0; p < NP; ++p) B[p] = M[p] = kept[p] = splat(0.f);
    if (!edge) {
        e.template form<false>(0);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int p = 0; p < NP; ++p) B[p] = through(e.at(i, p), e.keep(p), B[p], two(xs[i], p));
#pragma unroll
        for (int i = ROWS - 1; i >= 0; --i)
#pragma unroll
            for (int p = 0; p < NP; ++p) M[p] = times(e.at(i, p), e.keep(p), add2(two(ds[i], p), M[p]));
    } else {
        e.template form<true>(rows.valid);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (!(rows.valid >> i & 1)) xs[i] = ds[i] = Piece<T, CPL>{};
            if (rows.first >> i & 1) start(i, B);
#pragma unroll
            for (int p = 0; p < NP; ++p) B[p] = through(e.at(i, p), e.keep(p), B[p], two(xs[i], p));
        }
#pragma unroll
        for (int i = ROWS - 1; i >= 0; --i) {
            if (rows.last >> i & 1) {
                end(i, kept);
#pragma unroll
                for (int p = 0; p < NP; ++p) M[p] = kept[p];
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) M[p] = times(e.at(i, p), e.keep(p), add2(two(ds[i], p), M[p]));
        }
    }
    float2 A[NP];
    bool far = false;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float2 total = e.total(p);
        sums[kWarps - 1 - warp][p][threadIdx.x & 31] = total;
        A[p] = roots(total);
        far = far || !within(total, kFar);
    }
    far = __any_sync(kFull, far);
    ahead.put(warp, A, B, rows.first != 0, far);
    back.put(kWarps - 1 - warp, A, M, rows.last != 0, far);
    __syncthreads();
    ahead.pass(warp / kPer * kPer, warp, h);
    float2 u[ROWS][NP];  // exp(g_t) h_{t-1}
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (edge && rows.first >> i & 1) start(i, h);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float2 v = e.at(i, p);
            u[i][p] = times(v, e.keep(p), h[p]);
            h[p] = through(v, e.keep(p), h[p], two(xs[i], p));
        }
    }
    float2 m[NP];
    tile_carry<NP>(S, back, sums, k, n_time, n_slabs, slab, m, err);
    back.pass(0, kWarps - 1 - warp, m);
    T* px = dx + t0 * R.channels;
    G* pg = dg + t0 * R.channels;
    if (!edge) {
#pragma unroll
        for (int i = ROWS - 1; i >= 0; --i) {
            float2 l[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                l[p] = add2(two(ds[i], p), m[p]);
                m[p] = times(e.at(i, p), e.keep(p), l[p]);
                u[i][p] = mul2(u[i][p], l[p]);
            }
            at.store(px + (uint64_t)i * so, l);
            if constexpr (!SHARED) at.store(pg + (uint64_t)i * so, u[i]);
        }
    } else {
#pragma unroll
        for (int i = ROWS - 1; i >= 0; --i) {
            if (rows.last >> i & 1) {
                if ((rows.last & ((1u << i) - 1)) == 0) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) m[p] = kept[p];
                } else {
                    end(i, m);
                }
            }
            float2 l[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                l[p] = add2(two(ds[i], p), m[p]);
                m[p] = times(e.at(i, p), e.keep(p), l[p]);
                u[i][p] = mul2(u[i][p], l[p]);
            }
            if (rows.valid >> i & 1) {
                at.store(px + (uint64_t)i * so, l);
                if constexpr (!SHARED) at.store(pg + (uint64_t)i * so, u[i]);
            }
            if (rows.first >> i & 1 && dh0) {
                const int s = __shfl_sync(kFull, rows.seq, i);
                at.store(dh0 + (int64_t)s * R.channels, m);
            }
        }
    }
    if constexpr (SHARED) {
        float v[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            v[i] = u[i][0].x + u[i][0].y;
#pragma unroll
            for (int p = 1; p < NP; ++p) v[i] += u[i][p].x + u[i][p].y;
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
        float2 f[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) f[p] = splat(0.f);
        if (dh_last) at.load_pairs(dh_last + (int64_t)s * R.channels, f);
        at.store(dh0 + (int64_t)s * R.channels, f);
    }
}

template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
struct Backward {
    template <typename... A> static cudaError_t run(const Tiles& t, cudaStream_t st, A... a) {
        recurrence_backward_kernel<T, G, CPL, SHARED, VEC, ROWS><<<(unsigned)(t.n_time * t.n_slabs), kThreads, 0, st>>>(a...);
        return cudaGetLastError();
    }
};

}  // namespace

template <typename T, typename G>
cudaError_t launch_recurrence_backward(const RecDims& R, const G* g, const T* x, const float* h0, const float* states,
                                       const int32_t* cu, const T* dout, const float* dh_last, G* dg, T* dx,
                                       float* dh0, char* carry, int32_t* err, cudaStream_t st) {
    constexpr bool f32 = sizeof(T) == 4;
    const Tiles t = tiles(R, most_rows(R, f32, true));
    cudaError_t e = clear(carry, t, st);
    if (e != cudaSuccess) return e;
    return choose<Backward, T, G, f32 ? 8 : 16, 16, 8>(R, t, pairs<T, G>(R, x, g, dout, dx, dg, t.cpl), st, R, g, x, h0, states, cu,
                                         dout, dh_last, dg, dx, dh0, carry_of(carry, t), t.n_time, t.n_slabs, err);
}

#define HLA_RECURRENCE(T, G)                                                                                          \
    template cudaError_t launch_recurrence_backward<T, G>(const RecDims&, const G*, const T*, const float*,           \
                                                          const float*, const int32_t*, const T*, const float*, G*,   \
                                                          T*, float*, char*, int32_t*, cudaStream_t);
HLA_RECURRENCE(float, float)
HLA_RECURRENCE(float, __nv_bfloat16)
HLA_RECURRENCE(__nv_bfloat16, float)
HLA_RECURRENCE(__nv_bfloat16, __nv_bfloat16)

}  // namespace hla
