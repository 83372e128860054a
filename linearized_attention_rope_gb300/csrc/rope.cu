// Rotary positions of q and k, forward and gradient, one launch.
//
// A pair (a, b) at position p becomes gain (a cos t - b sin t, b cos t +
// a sin t), t = p w_i; the gradient rotates back.  The angle is formed as a
// fraction of a turn in 64-bit fixed point, p * freq mod 2^64, which keeps
// 2^-64 of a turn per position at any distance and needs no range reduction
// and no fp64 unit; its top 32 bits go to sincospif.
//
// Memory bound: every element is read and written once.  A block takes a few
// tokens: it forms their r/2 sines and cosines once in shared memory, for all
// heads, then streams 16-byte pieces, four in flight per thread.
#include <algorithm>

#include "attention.cuh"

namespace hla {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // pieces in flight per thread

template <typename T, int V> struct alignas(V * sizeof(T)) PieceV { T x[V]; };

// One unit: V pairs (half layout: V elements of each side; interleaved: 2 V
// consecutive elements), or V or 2 V elements that pass through.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeDims R, const T* q, const T* k, const int64_t* __restrict__ pos, T* qo,
            T* ko, int tokens, int heads_per_block) {
    extern __shared__ float2 cs[];  // [tokens][r / 2]
    const int half = R.r / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, R.total - t0);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const uint64_t turn = (uint64_t)__ldg(pos + t0 + t) * R.freq[j];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
        cs[i] = make_float2(c * R.gain, s * R.gain * (float)R.sign);
    }
    __syncthreads();
    // units of a head: half / V rotated, then the copied rest
    using P = PieceV<T, V>;
    const int h0 = blockIdx.y * heads_per_block, nh = min(heads_per_block, R.Hq + R.Hkv - h0);
    const int ur = half / V, uc = (R.d - R.r) / V, per_head = ur + uc;
    const int units = nt * nh * per_head;
    for (int u0 = threadIdx.x; u0 < units; u0 += kThreads * kBatch) {
        P a[kBatch], b[kBatch];
        T* dst[kBatch];
        int at[kBatch], gap[kBatch];  // cos/sin index (-1: copied); distance of the second piece (0: none)
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int u = u0 + x * kThreads;
            gap[x] = -1;
            if (u >= units) continue;
            const int th = u / per_head, i = u - th * per_head, t = th / nh, h = h0 + th - t * nh;
            const bool isq = h < R.Hq;
            const int64_t row = t0 + t;
            const T* src = isq ? q + row * R.q_in + (int64_t)h * R.d : k + row * R.k_in + (int64_t)(h - R.Hq) * R.d;
            dst[x] = isq ? qo + row * R.q_out + (int64_t)h * R.d : ko + row * R.k_out + (int64_t)(h - R.Hq) * R.d;
            const bool rot = i < ur;
            const int e = rot ? (R.interleaved ? 2 * i * V : i * V) : R.r + (i - ur) * V;
            at[x] = rot ? t * half + i * V : -1;
            gap[x] = rot ? (R.interleaved ? V : half) : 0;
            dst[x] += e;
            a[x] = *reinterpret_cast<const P*>(src + e);
            if (rot) b[x] = *reinterpret_cast<const P*>(src + e + gap[x]);
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            if (gap[x] < 0) continue;
            if (at[x] >= 0) {
                T lo[V], hi[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 w = cs[at[x] + j];
                    const bool il = R.interleaved != 0;
                    // interleaved: the 2 V elements a[0..V) b[0..V) are V pairs in a row
                    const T ea = il ? (2 * j < V ? a[x].x[(2 * j) % V] : b[x].x[(2 * j) % V]) : a[x].x[j];
                    const T eb = il ? (2 * j + 1 < V ? a[x].x[(2 * j + 1) % V] : b[x].x[(2 * j + 1) % V]) : b[x].x[j];
                    const float fa = to_f32(ea), fb = to_f32(eb);
                    lo[j] = from_f32<T>(fa * w.x - fb * w.y);
                    hi[j] = from_f32<T>(fb * w.x + fa * w.y);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (R.interleaved) {
                        a[x].x[j] = j & 1 ? hi[j / 2] : lo[j / 2];
                        b[x].x[j] = (V + j) & 1 ? hi[(V + j) / 2] : lo[(V + j) / 2];
                    } else {
                        a[x].x[j] = lo[j];
                        b[x].x[j] = hi[j];
                    }
                }
                *reinterpret_cast<P*>(dst[x] + gap[x]) = b[x];
            }
            *reinterpret_cast<P*>(dst[x]) = a[x];
        }
    }
}

template <typename T, int V>
cudaError_t launch(const RopeDims& R, const T* q, const T* k, const int64_t* pos, T* qo, T* ko, cudaStream_t st) {
    static DeviceCache cache;
    int n_sm = 0;
    cudaError_t e = device_cached(cache, &n_sm, [](int dev, int* v) { return sm_count(dev, v); });
    if (e != cudaSuccess) return e;
    const int heads = R.Hq + R.Hkv, half = R.r / 2;
    const int64_t per_token = (int64_t)heads * (half / V + (R.d - R.r) / V);
    // Tokens per block: enough units for one full batch of every thread, at most 32 KB of sines.  With fewer
    // tokens than two blocks per SM, a token's heads are spread over blocks instead (each forms the sines again,
    // which costs less than the idle SMs).
    int tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kThreads * kBatch / std::max<int64_t>(1, per_token), 4096 / half));
    int split = 1;
    if (R.total < 2 * n_sm) {
        tokens = 1;
        split = (int)std::max<int64_t>(1, std::min<int64_t>(heads, std::min<int64_t>(2 * n_sm / R.total, per_token / 128)));
    }
    const int hpb = (heads + split - 1) / split;
    const int64_t blocks = (R.total + tokens - 1) / tokens;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    rope_kernel<T, V><<<dim3((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb)), kThreads,
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
    if (p % 16 == 0 && s % V == 0) return launch<T, V>(R, q, k, pos, qo, ko, st);
    return launch<T, 1>(R, q, k, pos, qo, ko, st);
}
template cudaError_t launch_rope<float>(const RopeDims&, const float*, const float*, const int64_t*, float*, float*,
                                        cudaStream_t);
template cudaError_t launch_rope<__nv_bfloat16>(const RopeDims&, const __nv_bfloat16*, const __nv_bfloat16*,
                                                const int64_t*, __nv_bfloat16*, __nv_bfloat16*, cudaStream_t);

}  // namespace hla
