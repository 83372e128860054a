// Gated linear recurrence, forward, and its step.
//
// Measured: 131071 rows of 1024 bf16 channels and gates 245 us (3.3 TB/s, 2.1 instructions a cycle; a third of the time is the
// tiles' waiting for one another: 32767 rows took 72 us, 53 without looking at other tiles); 16309 rows of 4096, gates in
// fp32, 123 us (4.3 TB/s); the step of 64 x 4096 states 3 us.  At the 80 registers that three blocks an SM leave, these two
// spill 24 and 28 bytes a thread, the others 8 to 32.
#include "recurrence.cuh"

namespace hla {

namespace {

template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS == 8 ? (CPL == 4 ? 3 : 4) : VEC && sizeof(T) == 2 ? 3 : 2)
recurrence_kernel(const RecDims R, const G* __restrict__ g, const T* __restrict__ x, const float* h0,
                  const int32_t* __restrict__ cu, T* __restrict__ out, float* h_last, float* __restrict__ states,
                  const Carry S, int n_time, int n_slabs, int32_t* err) {
    constexpr int NP = CPL / 2;
    __shared__ Runs<NP> runs;
    __shared__ Sums<NP> sums;
    const int tile = take_tile(S.ticket, n_time), k = tile / n_slabs, slab = tile - k * n_slabs;
    const int warp = threadIdx.x >> 5;
    const int64_t t0 = ((int64_t)k * kWarps + warp) * ROWS;
    const int n = (int)clamp_i64(R.total - t0, 0, ROWS);
    const Lane<CPL, VEC> at(slab, R.channels);
    Piece<T, CPL> xs[ROWS];
    Gates<G, CPL, SHARED, VEC, ROWS> e;
    const T* xr = x + t0 * R.sx;
    const uint32_t sx = (uint32_t)R.sx, sg = (uint32_t)R.sg;
    if (n == ROWS) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) xs[i] = at.load(xr + (uint64_t)i * sx);
        e.template load<true>(at, g + t0 * R.sg, sg, slab, n);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) xs[i] = i < n ? at.load(xr + (uint64_t)i * sx) : Piece<T, CPL>{};
        e.template load<false>(at, g + t0 * R.sg, sg, slab, n);
    }
    const Rows rows(cu, R, t0, ROWS);
    if (tile == 0) check_table(cu, R, err);
    const bool edge = (rows.first | rows.last) != 0 || rows.valid != (ROWS == 32 ? kFull : (1u << ROWS % 32) - 1);
    auto start = [&](int i, float2 (&h)[NP]) {  // the state in front of a sequence's first row
        const int s = __shfl_sync(kFull, rows.seq, i);
#pragma unroll
        for (int p = 0; p < NP; ++p) h[p] = splat(0.f);
        if (h0) at.load_pairs(h0 + (int64_t)s * R.channels, h);
    };
    float2 B[NP], kept[NP];  // kept: h0 of the run's last sequence (another tile may end it, in h0's place)
#pragma unroll
    for (int p = 0; p < NP; ++p) B[p] = kept[p] = splat(0.f);
    if (!edge) {
        e.template form<false>(0);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int p = 0; p < NP; ++p) B[p] = through(e.at(i, p), e.keep(p), B[p], two(xs[i], p));
    } else {
        e.template form<true>(rows.valid);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (!(rows.valid >> i & 1)) xs[i] = Piece<T, CPL>{};
            if (rows.first >> i & 1) {
                start(i, kept);
#pragma unroll
                for (int p = 0; p < NP; ++p) B[p] = kept[p];
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) B[p] = through(e.at(i, p), e.keep(p), B[p], two(xs[i], p));
        }
    }
    float2 A[NP];
    bool far = false;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float2 total = e.total(p);
        sums[warp][p][threadIdx.x & 31] = total;
        A[p] = roots(total);
        far = far || !within(total, kFar);
    }
    far = __any_sync(kFull, far);
    runs.put(warp, A, B, rows.first != 0, far);
    __syncthreads();
    float2 h[NP];
    tile_carry<NP>(S, runs, sums, k, n_time, n_slabs, slab, h, err);
    runs.pass(0, warp, h);
    if (states && t0 % kStateRows == 0 && t0 < R.total) at.store(states + t0 / kStateRows * R.channels, h);
    T* o = out + t0 * R.channels;
    const uint32_t so = (uint32_t)R.channels;
    if (!edge) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
#pragma unroll
            for (int p = 0; p < NP; ++p) h[p] = through(e.at(i, p), e.keep(p), h[p], two(xs[i], p));
            at.store(o + (uint64_t)i * so, h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (rows.first >> i & 1) {
                if (rows.first >> i == 1) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) h[p] = kept[p];
                } else {
                    start(i, h);
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) h[p] = through(e.at(i, p), e.keep(p), h[p], two(xs[i], p));
            if (rows.valid >> i & 1) at.store(o + (uint64_t)i * so, h);
            if (rows.last >> i & 1 && h_last) {
                const int s = __shfl_sync(kFull, rows.seq, i);
                at.store(h_last + (int64_t)s * R.channels, h);
            }
        }
    }
    if (!h_last) return;
    for (int s = k * kWarps + warp; s < R.n_seqs; s += n_time * kWarps) {  // sequences without rows
        int64_t a, m;
        seq_range(cu, s, R.total, &a, &m);
        if (m > 0) continue;
        float2 f[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) f[p] = splat(0.f);
        if (h0) at.load_pairs(h0 + (int64_t)s * R.channels, f);
        at.store(h_last + (int64_t)s * R.channels, f);
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
    float y[V];
    if (R.gate_dim > 1) {
        y[0] = to_f32(g[row * R.sg + c / R.gate_dim]);
#pragma unroll
        for (int j = 1; j < V; ++j) y[j] = y[0];
    } else {
        const Piece<G, V> q = *reinterpret_cast<const Piece<G, V>*>(g + row * R.sg + c);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = to_f32(q.x[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool near = y[j] >= kLow && y[j] <= 2.f;
        const float v = near ? expm1f(y[j]) : expf(y[j]);
        s.x[j] = fmaf(v, s.x[j], to_f32(a.x[j])) + (near ? s.x[j] : 0.f);
        o.x[j] = from_f32<T>(s.x[j]);
    }
    *reinterpret_cast<H*>(h + row * R.channels + c) = s;
    *reinterpret_cast<P*>(out + row * R.channels + c) = o;
}

template <typename T, typename G, int CPL, bool SHARED, bool VEC, int ROWS>
struct Forward {
    template <typename... A> static cudaError_t run(const Tiles& t, cudaStream_t st, A... a) {
        recurrence_kernel<T, G, CPL, SHARED, VEC, ROWS><<<(unsigned)(t.n_time * t.n_slabs), kThreads, 0, st>>>(a...);
        return cudaGetLastError();
    }
};

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

template <typename T, typename G>
cudaError_t launch_recurrence(const RecDims& R, const G* g, const T* x, const float* h0, const int32_t* cu, T* out,
                              float* h_last, float* states, char* carry, int32_t* err, cudaStream_t st) {
    constexpr bool f32 = sizeof(T) == 4;
    const Tiles t = tiles(R, most_rows(R, f32, false));
    cudaError_t e = clear(carry, t, st);
    if (e != cudaSuccess) return e;
    return choose<Forward, T, G, 16, f32 ? 16 : 32, 16>(R, t, pairs<T, G>(R, x, g, out, out, g, t.cpl), st, R, g, x, h0, cu,
                                                    out, h_last, states, carry_of(carry, t), t.n_time, t.n_slabs, err);
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
    template cudaError_t launch_recurrence_step<T, G>(const RecDims&, const G*, const T*, float*, T*, cudaStream_t);
HLA_RECURRENCE(float, float)
HLA_RECURRENCE(float, __nv_bfloat16)
HLA_RECURRENCE(__nv_bfloat16, float)
HLA_RECURRENCE(__nv_bfloat16, __nv_bfloat16)

}  // namespace hla
