// Rotary positions of q and k, forward and gradient, one launch.
//
// A pair (a, b) at position p becomes gain (a cos t - b sin t, b cos t +
// a sin t), t = p w_i; the gradient rotates back.  The angle is formed as a
// fraction of a turn in 64-bit fixed point, p * freq mod 2^64: the product is
// exact at any position and needs no range reduction and no fp64 unit.  (freq is
// w_i / 2 pi with a double's precision, so an angle is off by about 2^-53 of
// itself before whole turns are taken off.)  The nearest quarter of a turn is
// taken off before the rest is rounded to fp32 for sincospif: rounded as a whole
// the angle is off by up to 9e-8 wherever it lies, sines near their zeros too.
//
// Memory bound: every element is read and written once.  A block takes a few
// tokens: it forms their r/2 sines and cosines once in shared memory, for all
// heads; then a thread keeps one 16-byte place of the head and walks the
// (token, head) pairs, a few in flight.  (32768 tokens, 40 heads of 128, bf16:
// finding token and head by division and holding both layouts' code, 221 us;
// so 116 us, 5.4 TB/s.  64 tokens: 2.9 us, the length of a launch.)
#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kThreads = 256;

template <typename T, int V> struct alignas(V * sizeof(T)) Piece { T x[V]; };

// Sines of pair i V + j: cs[(token V + j) (r / 2 / V) + i], so that neighbouring threads read neighbouring words.
// IL: interleaved pairs; a thread's V pairs are 2 V elements in a row, else V elements of each half.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeDims R, const T* q, const T* k, const int64_t* __restrict__ pos, T* qo,
            T* ko, int tokens, int heads_per_block) {
    constexpr int kBatch = V == 8 ? 2 : 4;  // pairs of pieces in flight
    extern __shared__ float2 cs[];
    const int half = R.r / 2, places = half / V;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, R.total - t0);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const uint64_t turn = (uint64_t)__ldg(pos + t0 + t) * R.freq[j];
        const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);  // 0 .. 3
        float x, y;
        sincospif((float)(int64_t)(turn - ((uint64_t)quarter << 62)) * 0x1p-63f, &x, &y);  // half turns, within a quarter
        const float c = quarter & 1 ? (quarter & 2 ? x : -x) : (quarter & 2 ? -y : y);
        const float s = quarter & 1 ? (quarter & 2 ? -y : y) : (quarter & 2 ? -x : x);
        cs[(t * V + j % V) * places + j / V] = make_float2(c * R.gain, s * R.gain * (float)R.sign);
    }
    __syncthreads();
    using P = Piece<T, V>;
    const int h0 = blockIdx.y * heads_per_block, nh = min(heads_per_block, R.Hq + R.Hkv - h0);
    auto source = [&](int t, int h) {
        return h < R.Hq ? q + (t0 + t) * R.q_in + (int64_t)h * R.d : k + (t0 + t) * R.k_in + (int64_t)(h - R.Hq) * R.d;
    };
    auto target = [&](int t, int h) {
        return h < R.Hq ? qo + (t0 + t) * R.q_out + (int64_t)h * R.d : ko + (t0 + t) * R.k_out + (int64_t)(h - R.Hq) * R.d;
    };
    {
        const int step = kThreads / places, i = threadIdx.x % places;  // heads a block takes at once; this thread's place
        const int e = IL ? 2 * i * V : i * V, gap = IL ? V : half;
        int h = threadIdx.x / places, t = h < step ? h / nh : nt;
        h -= t * nh;
        while (t < nt) {
            P a[kBatch], b[kBatch];
            T* dst[kBatch];
            int tt[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                tt[x] = t;
                if (t < nt) {
                    const T* src = source(t, h0 + h) + e;
                    dst[x] = target(t, h0 + h) + e;
                    a[x] = *reinterpret_cast<const P*>(src);
                    b[x] = *reinterpret_cast<const P*>(src + gap);
                }
                h += step;
                while (h >= nh && t < nt) {
                    h -= nh;
                    ++t;
                }
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                if (tt[x] >= nt) continue;
                P lo, hi;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 w = cs[(tt[x] * V + j) * places + i];
                    // interleaved: elements a[0..V) b[0..V) are V pairs in a row
                    const T ea = IL ? (2 * j < V ? a[x].x[(2 * j) % V] : b[x].x[(2 * j) % V]) : a[x].x[j];
                    const T eb = IL ? (2 * j + 1 < V ? a[x].x[(2 * j + 1) % V] : b[x].x[(2 * j + 1) % V]) : b[x].x[j];
                    const float fa = to_f32(ea), fb = to_f32(eb);
                    const T ra = from_f32<T>(fa * w.x - fb * w.y), rb = from_f32<T>(fb * w.x + fa * w.y);
                    if (IL) {
                        if (2 * j < V) lo.x[(2 * j) % V] = ra; else hi.x[(2 * j) % V] = ra;
                        if (2 * j + 1 < V) lo.x[(2 * j + 1) % V] = rb; else hi.x[(2 * j + 1) % V] = rb;
                    } else {
                        lo.x[j] = ra;
                        hi.x[j] = rb;
                    }
                }
                *reinterpret_cast<P*>(dst[x]) = lo;
                *reinterpret_cast<P*>(dst[x] + gap) = hi;
            }
        }
    }
    // the elements past the rotated ones, unless they are in place already
    const int copies = (R.d - R.r) / V;
    if (copies == 0 || (qo == q && ko == k)) return;
    for (int u = threadIdx.x; u < nt * nh * copies; u += kThreads) {
        const int th = u / copies, t = th / nh, h = h0 + th - t * nh, e = R.r + (u - th * copies) * V;
        const T* src = source(t, h) + e;
        T* dst = target(t, h) + e;
        if (dst != src) *reinterpret_cast<P*>(dst) = *reinterpret_cast<const P*>(src);
    }
}

template <typename T, int V, bool IL>
cudaError_t launch(const RopeDims& R, const T* q, const T* k, const int64_t* pos, T* qo, T* ko, cudaStream_t st) {
    static DeviceCache cache;
    int n_sm = 0;
    cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
    if (e != cudaSuccess) return e;
    const int heads = R.Hq + R.Hkv, half = R.r / 2, at_once = kThreads / (half / V);
    // Tokens per block: eight (token, head) pairs for every thread, at most 32 KB of sines, and two blocks per SM.
    // With fewer tokens than that, a token's heads are spread over blocks instead (each forms the sines again, which
    // costs less than idle SMs).
    const int64_t want = std::max(1, 8 * at_once / heads);
    int tokens = (int)std::max<int64_t>(1, std::min<int64_t>({want, 4096 / half, R.total / (2 * n_sm)}));
    int split = 1;
    if (R.total < 2 * n_sm)
        split = (int)std::max<int64_t>(1, std::min<int64_t>(2 * n_sm / R.total, (heads + at_once - 1) / at_once));
    const int hpb = (heads + split - 1) / split;
    const int64_t blocks = (R.total + tokens - 1) / tokens;
    rope_kernel<T, V, IL><<<dim3((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb)), kThreads,
                            (size_t)tokens * half * sizeof(float2), st>>>(R, q, k, pos, qo, ko, tokens, hpb);
    return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_rope(const RopeDims& R, const T* q, const T* k, const int64_t* pos, T* qo, T* ko,
                        cudaStream_t st) {
    if (R.total <= 0 || R.Hq + R.Hkv == 0) return cudaSuccess;
    constexpr int V = 16 / (int)sizeof(T);
    // 16-byte pieces where every piece of every head starts on a 16-byte boundary, else single elements
    const uintptr_t p = (uintptr_t)q | (uintptr_t)k | (uintptr_t)qo | (uintptr_t)ko;
    const int64_t s = R.q_in | R.k_in | R.q_out | R.k_out | R.d | (R.r / 2);
    if (p % 16 == 0 && s % V == 0)
        return R.interleaved ? launch<T, V, true>(R, q, k, pos, qo, ko, st) : launch<T, V, false>(R, q, k, pos, qo, ko, st);
    return R.interleaved ? launch<T, 1, true>(R, q, k, pos, qo, ko, st) : launch<T, 1, false>(R, q, k, pos, qo, ko, st);
}
template cudaError_t launch_rope<float>(const RopeDims&, const float*, const float*, const int64_t*, float*, float*,
                                        cudaStream_t);
template cudaError_t launch_rope<__nv_bfloat16>(const RopeDims&, const __nv_bfloat16*, const __nv_bfloat16*,
                                                const int64_t*, __nv_bfloat16*, __nv_bfloat16*, cudaStream_t);

}  // namespace hla
