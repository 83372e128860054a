// Products of up to sixteen rows with 4-bit weights: y = x W^T, W[n][k] = scale (q - 8) + offset, a scale (and offset)
// per row n and group of 32, 64 or 128 inputs k.  (More rows: linear4_tc.cu, for which rows are laid out here.)
//
// Bound by the weights' bytes, half a byte each.  Products on the warp-level tensor instruction (m16n8k16, bf16 in,
// fp32 sums): the 16 rows are rows of W, the 8 columns tokens; a weight goes from memory to its one lane's registers,
// which tensor memory would have it leave again.  q - 8 is exact in bf16 and so is every product; a group's sum is scaled
// in fp32 as it is added to the row's.  (Scaled weights would have to be rounded to bf16 each.)  Which k a lane's
// operands stand for is free, as long as both agree: a lane takes words of a weight row as they lie.
//
// A block takes 128 rows, 16 a warp, and, in a cluster of C, a C-th of the inputs; the tokens' inputs and the
// rows' scales come into shared memory 1024 inputs at a time, in the order in which lanes read them: fp32 rows as three
// bf16 parts, cut off 8 bits at a time (nothing is lost), 8-bit rows as bf16 (exact, too).  Offsets are multiplied by the
// group's sum of x, formed on that way.  Weights are two steps (of 128 inputs) ahead of the products.  The cluster's
// sums are added through distributed shared memory, in order of its blocks.
//
// Measured: 16 8-bit rows through 8192 x 28672 with offsets 63 us (1.9 TB/s; 69 on tcgen05, whose 128-row tiles are read
// back for 16 tokens), one row through 4096 x 4096 8 us.  A pair of weights takes a shift, a merge and a difference, the first
// two at half rate: the ALU pipe is busy half of the time, the load/store pipe as much, and neither 32 rows a warp (64), sixteen
// warps a block (63 to 67) nor more weights under way changed that.
#include <algorithm>

#include "layer.cuh"

namespace hla {

namespace {

constexpr int kWarps4 = 8, kThreads4 = 32 * kWarps4;
constexpr int kAhead = 2;  // steps of weights under way

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Nibbles s / 4 and s / 4 + 4 of w, less 8, as two bf16: 0x4300 | q is 128 + q.
__device__ __forceinline__ uint32_t nibbles(uint32_t w, int s) {
    const uint32_t y = ((w >> s) & 0x000f000fu) | 0x43004300u, off = 0x43084308u;
    const __nv_bfloat162 d = __hsub2(reinterpret_cast<const __nv_bfloat162&>(y), reinterpret_cast<const __nv_bfloat162&>(off));
    return reinterpret_cast<const uint32_t&>(d);
}

__device__ __forceinline__ uint4 load_far(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// fp32 as three bf16 parts; an infinity or NaN is in the first alone.
__device__ __forceinline__ void three_parts(float v, __nv_bfloat16 (&o)[3]) {
    const bool fine = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
    if (v != v) v = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        const float top = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
        o[s] = from_f32<__nv_bfloat16>(top);
        v = fine ? v - top : 0.f;
    }
}

template <typename T, typename X, int MT, int GROUP, bool OFFS>
struct Plan {
    static constexpr int kParts = sizeof(X) == 4 ? 3 : 1;
    static constexpr int kSteps = sizeof(X) == 4 ? 4 : 8;  // of 128 inputs, in shared memory
    static constexpr int kRows = 16 * kWarps4, kTok = 8 * MT;
    static constexpr int kPitch = kSteps * 256 + 64;  // bytes of a token: two rows' 64 bytes lie in different banks
    static constexpr int kGroups = kSteps * (128 / GROUP);
    static constexpr int kScalePitch = kRows + 2;
    static constexpr size_t kX = (size_t)kParts * kTok * kPitch, kScale = (size_t)kGroups * kScalePitch * sizeof(T);
    static constexpr size_t kIn = kX + kScale * (OFFS ? 2 : 1) + (OFFS ? (size_t)kGroups * kTok * 4 : 0);
    static constexpr size_t kSmem = std::max<size_t>(kIn, (size_t)kTok * kRows * 4);
};

template <typename T, typename X, int MT, int GROUP, bool OFFS>
__global__ void __launch_bounds__(kThreads4, 3)
linear4_kernel(const Linear4Dims L, const X* __restrict__ x, const uint8_t* __restrict__ exps, const uint8_t* __restrict__ w,
               const T* __restrict__ scales, const T* __restrict__ offsets, T* __restrict__ out, int n_split, bool vec) {
    using S = Plan<T, X, MT, GROUP, OFFS>;
    constexpr int kWords = GROUP / 32, kSub = 128 / GROUP;  // words of a lane per group, groups of a step
    extern __shared__ __align__(16) uint8_t sm[];
    T* const sm_scale = reinterpret_cast<T*>(sm + S::kX);                // [group][row]
    T* const sm_off = sm_scale + S::kScale / sizeof(T);
    float* const sm_sum = reinterpret_cast<float*>(sm + S::kX + 2 * S::kScale);  // [group][token]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const uint32_t rank = n_split > 1 ? cluster_rank() : 0;
    const int n0 = blockIdx.x / n_split * S::kRows, n_groups = L.n_in / GROUP, stages = (L.n_in + 127) / 128;
    const int s0 = (int)((int64_t)stages * rank / n_split), s1 = (int)((int64_t)stages * (rank + 1) / n_split);
    const uint8_t* wr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        wr[h] = w + (int64_t)min(n0 + warp * 16 + h * 8 + gq, L.n_out - 1) * (L.n_in / 2) + tq * (kWords * 4);
    const int x_shift = L.x_group == 32 ? 5 : 7, x_groups = L.x_group ? L.n_in >> x_shift : 1;  // of a row's exponents
    uint32_t q[kAhead][2][4];
    auto fetch = [&](uint32_t (&v)[2][4], int s) {
#pragma unroll
        for (int g = 0; g < kSub; ++g) {
            // (a group may lie behind the last one: zeros there, and nothing to multiply)
            const bool on = s < s1 && (GROUP == 128 || s * kSub + g < n_groups);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* p = wr[h] + (int64_t)s * 64 + g * (GROUP / 2);
                uint32_t* o = v[h] + g * kWords;
                if constexpr (kWords == 4) {
                    const uint4 y = on ? load_far(p) : make_uint4(0, 0, 0, 0);
                    o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
                } else if constexpr (kWords == 2) {
                    const uint2 y = on ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
                    o[0] = y.x; o[1] = y.y;
                } else {
                    o[0] = on ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0;
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) fetch(q[d], s0 + d);
    float acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    for (int c0 = s0; c0 < s1; c0 += S::kSteps) {
        __syncthreads();
        // the tokens' inputs, 8 at a time, where the lane that takes them has its four lanes' words in a row
#pragma unroll 2
        for (int j = threadIdx.x; j < S::kTok * S::kSteps * 16; j += kThreads4) {
            const int t = j / (S::kSteps * 16), c = j % (S::kSteps * 16);
            const int64_t row = (int64_t)blockIdx.y * S::kTok + t;
            const int k = c0 * 128 + c * 8;
            float2 v[4] = {};  // inputs 2i, 2i + 1
            if (row < L.rows && k < L.n_in) {
                const X* p = x + row * L.sx + k;
                constexpr int kAt = sizeof(X) == 4 ? 4 : 8;  // values of a load: fp32 rows lie on 16 bytes, not on 32
                Piece<X, kAt> y[8 / kAt];
                if (vec) {
#pragma unroll
                    for (int i = 0; i < 8 / kAt; ++i) y[i] = reinterpret_cast<const Piece<X, kAt>*>(p)[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i / kAt].x[i % kAt] = p[i];
                }
                if constexpr (sizeof(X) == 1) {
                    const float f = group_pow2((int)exps[row * x_groups + (L.x_group ? k >> x_shift : 0)] - 127);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(reinterpret_cast<const __nv_fp8x2_storage_t*>(y[0].x)[i], __NV_E4M3);
                        v[i] = mul2(__half22float2(__half2(h)), make_float2(f, f));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = make_float2(to_f32(y[2 * i / kAt].x[2 * i % kAt]), to_f32(y[2 * i / kAt].x[2 * i % kAt + 1]));
                }
            }
            constexpr int kIn = GROUP / 8;  // pieces of a group
            const int in = c % 16 % kIn, at = c / 16 * 16 + (c % 16 / kIn * kWords + in % kWords) * 4 + in / kWords;
            // pairs (i, i + 4), as the weights' nibbles are taken
            if constexpr (S::kParts == 1) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v[i].x, v[i + 2].x), b = __floats2bfloat162_rn(v[i].y, v[i + 2].y);
                    o[2 * i] = reinterpret_cast<const uint32_t&>(a);
                    o[2 * i + 1] = reinterpret_cast<const uint32_t&>(b);
                }
                *reinterpret_cast<uint4*>(sm + t * S::kPitch + at * 16) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                Piece<__nv_bfloat16, 8> o[3];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __nv_bfloat16 lo[3], hi[3];
                    three_parts(i & 1 ? v[i / 2].y : v[i / 2].x, lo);
                    three_parts(i & 1 ? v[i / 2 + 2].y : v[i / 2 + 2].x, hi);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        o[p].x[2 * i] = lo[p];
                        o[p].x[2 * i + 1] = hi[p];
                    }
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<Piece<__nv_bfloat16, 8>*>(sm + (p * S::kTok + t) * S::kPitch + at * 16) = o[p];
            }
            if constexpr (OFFS) {
                const float2 z = add2(add2(v[0], v[1]), add2(v[2], v[3]));
                float y = z.x + z.y;
#pragma unroll
                for (int o = kIn / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (in == 0) sm_sum[c / kIn * S::kTok + t] = y;
            }
        }
        const int g = threadIdx.x % S::kGroups, gg = c0 * kSub + g;
#pragma unroll 4
        for (int row = threadIdx.x / S::kGroups; row < S::kRows; row += kThreads4 / S::kGroups) {
            const int64_t from = (int64_t)min(n0 + row, L.n_out - 1) * n_groups + gg;
            sm_scale[g * S::kScalePitch + row] = gg < n_groups ? scales[from] : from_f32<T>(0.f);
            if constexpr (OFFS) sm_off[g * S::kScalePitch + row] = gg < n_groups ? offsets[from] : from_f32<T>(0.f);
        }
        __syncthreads();
        auto step = [&](uint32_t (&v)[2][4], int st) {
#pragma unroll
            for (int g = 0; g < kSub; ++g) {
                float part[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[m][i] = 0.f;
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t lo = v[0][g * kWords + k], hi = v[1][g * kWords + k];
                        a[s][0] = nibbles(lo, 8 * s);
                        a[s][1] = nibbles(hi, 8 * s);
                        a[s][2] = nibbles(lo, 8 * s + 4);
                        a[s][3] = nibbles(hi, 8 * s + 4);
                    }
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 b = *reinterpret_cast<const uint4*>(
                                sm + (p * S::kTok + m * 8 + gq) * S::kPitch + (st * 16 + (g * kWords + k) * 4 + tq) * 16);
                            mma16816(part[m], a[0], b.x, b.y);
                            mma16816(part[m], a[1], b.z, b.w);
                        }
                }
                const int gi = st * kSub + g, row = warp * 16 + gq;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float2 sum;
                    if constexpr (OFFS) sum = *reinterpret_cast<const float2*>(sm_sum + gi * S::kTok + m * 8 + tq * 2);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int at = gi * S::kScalePitch + row + h * 8;
                        const float sc = to_f32(sm_scale[at]);
                        float2 y = make_float2(acc[m][2 * h], acc[m][2 * h + 1]);
                        y = ffma2(make_float2(sc, sc), make_float2(part[m][2 * h], part[m][2 * h + 1]), y);
                        if constexpr (OFFS) {
                            const float of = to_f32(sm_off[at]);
                            y = ffma2(make_float2(of, of), sum, y);
                        }
                        acc[m][2 * h] = y.x;
                        acc[m][2 * h + 1] = y.y;
                    }
                }
            }
        };
        // (a group behind the last one: scale, offset and inputs are 0)
        for (int st = 0; st < S::kSteps; st += kAhead)
#pragma unroll
            for (int d = 0; d < kAhead; ++d)
                if (c0 + st + d < s1) {
                    step(q[d], st + d);
                    fetch(q[d], c0 + st + d + kAhead);
                }
    }
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(sm);  // [token][row]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[(m * 8 + tq * 2 + (i & 1)) * S::kRows + warp * 16 + (i >> 1) * 8 + gq] = acc[m][i];
    if (n_split > 1) cluster_sync_all();
    else __syncthreads();
    const int t0 = (int)(S::kTok * rank / n_split), t1 = (int)(S::kTok * (rank + 1) / n_split);
#pragma unroll 4
    for (int i = t0 * S::kRows + threadIdx.x; i < t1 * S::kRows; i += kThreads4) {
        const int64_t t = (int64_t)blockIdx.y * S::kTok + i / S::kRows;
        const int n = n0 + i % S::kRows;
        if (t >= L.rows || n >= L.n_out) continue;
        out[t * L.n_out + n] = from_f32<T>(n_split == 1 ? sums[i] : cluster_sum(sums + i, n_split));
    }
    if (n_split > 1) cluster_sync_all();  // no block leaves while its sums are read
}

// Rows as bf16 parts [parts][rows][n_in]: eight inputs a thread.
template <typename X>
__global__ void __launch_bounds__(256)
linear4_rows_kernel(const Linear4Dims L, const X* __restrict__ x, const uint8_t* __restrict__ exps,
                    __nv_bfloat16* __restrict__ parts) {
    const int per = L.n_in / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= L.rows * per) return;
    const int64_t row = i / per;
    const int k = (int)(i - row * per) * 8;
    const X* p = x + row * L.sx + k;
    Piece<__nv_bfloat16, 8> o[sizeof(X) == 4 ? 3 : 1];
    float scale = 1.f;
    if constexpr (sizeof(X) == 1) {
        const int group = L.x_group ? L.x_group : L.n_in;
        scale = group_pow2((int)exps[row * (L.n_in / group) + k / group] - 127);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(X) == 4) {
            __nv_bfloat16 y[3];
            three_parts(p[j], y);
#pragma unroll
            for (int s = 0; s < 3; ++s) o[s].x[j] = y[s];
        } else if constexpr (sizeof(X) == 1) {
            const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)p[j], __NV_E4M3);
            o[0].x[j] = from_f32<__nv_bfloat16>(__half2float(__half(h)) * scale);
        } else {
            o[0].x[j] = p[j];
        }
    }
#pragma unroll
    for (int s = 0; s < (sizeof(X) == 4 ? 3 : 1); ++s)
        *reinterpret_cast<Piece<__nv_bfloat16, 8>*>(parts + (s * L.rows + row) * L.n_in + k) = o[s];
}

// Weights to 4 bits, a warp per group.  Without offsets: scale = max |w| / 7 in T, q = round(w / scale) + 8, 1 to 15;
// with: scale = (max - min) / 15, offset = min + 8 scale, q = round((w - offset) / scale) + 8, 0 to 15.
template <typename T>
__global__ void __launch_bounds__(256)
linear4_quantize_kernel(const Linear4Dims L, const T* __restrict__ weight, uint8_t* __restrict__ w, T* __restrict__ scales,
                        T* __restrict__ offsets) {
    const int lane = threadIdx.x & 31, n_groups = L.n_in / L.group;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // (row, group)
    if (i >= (int64_t)L.n_out * n_groups) return;
    const T* p = weight + i * L.group;
    uint8_t* o = w + i * (L.group / 2);
    float lo = INFINITY, hi = -INFINITY;
    for (int k = lane; k < L.group; k += 32) {
        const float v = to_f32(p[k]);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    for (int s = 16; s; s >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, s));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, s));
    }
    const T scale = from_f32<T>(offsets ? hi / 15.f - lo / 15.f : fmaxf(hi, -lo) / 7.f);
    const float f = to_f32(scale);
    const T offset = from_f32<T>(offsets ? lo + 8.f * f : 0.f);
    const float off = to_f32(offset);
    auto quant = [&](int k) {
        const float v = f > 0.f ? rintf((to_f32(p[k]) - off) / f) : 0.f;
        return (uint32_t)(fminf(fmaxf(v, offsets ? -8.f : -7.f), 7.f) + 8.f);
    };
    for (int k = 2 * lane; k < L.group; k += 64) o[k / 2] = (uint8_t)(quant(k) | quant(k + 1) << 4);
    if (lane == 0) {
        scales[i] = scale;
        if (offsets) offsets[i] = offset;
    }
}

template <typename T, typename X, int MT, int GROUP, bool OFFS>
cudaError_t run(const Linear4Dims& L, const X* x, const uint8_t* exps, const uint8_t* w, const T* scales, const T* offsets,
                T* out, cudaStream_t st) {
    using S = Plan<T, X, MT, GROUP, OFFS>;
    const auto kernel = linear4_kernel<T, X, MT, GROUP, OFFS>;
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    });
    if (e != cudaSuccess) return e;
    // (three blocks an SM; one row through 4096 x 4096: 8.2 us, 9.3 where one block and two steps are counted)
    const int tiles = (L.n_out + S::kRows - 1) / S::kRows, c = linear4_split(tiles, (L.n_in + 127) / 128, 456, 4);
    ClusterCfg cfg(dim3((unsigned)(tiles * c), (unsigned)((L.rows + S::kTok - 1) / S::kTok)), kThreads4, S::kSmem, st, c);
    const bool vec = (uintptr_t)x % std::min<size_t>(16, 8 * sizeof(X)) == 0 && L.sx % 8 == 0;
    return cudaLaunchKernelEx(&cfg.cfg, kernel, L, x, exps, w, scales, offsets, out, c, vec);
}

template <typename T, typename X>
cudaError_t few(const Linear4Dims& L, const X* x, const uint8_t* exps, const uint8_t* w, const T* scales, const T* offsets,
                T* out, cudaStream_t st) {
    auto go = [&](auto mt, auto group, auto offs) {
        return run<T, X, decltype(mt)::value, decltype(group)::value, decltype(offs)::value>(L, x, exps, w, scales, offsets, out, st);
    };
    auto with_offsets = [&](auto mt, auto group) {
        return offsets ? go(mt, group, std::true_type()) : go(mt, group, std::false_type());
    };
    auto with_group = [&](auto mt) {
        if (L.group == 128) return with_offsets(mt, std::integral_constant<int, 128>());
        if (L.group == 64) return with_offsets(mt, std::integral_constant<int, 64>());
        return with_offsets(mt, std::integral_constant<int, 32>());
    };
    return L.rows <= 8 ? with_group(std::integral_constant<int, 1>()) : with_group(std::integral_constant<int, 2>());
}

}  // namespace

int linear4_split(int64_t tiles, int64_t stages, int64_t blocks, int64_t ends) {
    int best = 1;
    int64_t least = INT64_MAX;
    for (int c = 1; c <= 8; c *= 2) {
        if (c > 1 && c > stages) break;
        const int64_t cost = (tiles * c + blocks - 1) / blocks * ((stages + c - 1) / c + ends);
        if (cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}

int linear4_parts(Rows4 kind) { return kind == Rows4::kF32 ? 3 : 1; }

template <typename T>
cudaError_t launch_linear4(const Linear4Dims& L, Rows4 kind, const void* x, const uint8_t* x_exp, const uint8_t* w,
                           const T* scales, const T* offsets, T* out, __nv_bfloat16* parts, cudaStream_t st) {
    if (L.rows == 0) return cudaSuccess;
    if (L.rows <= kFewRows) {
        if (kind == Rows4::kE4m3) return few<T>(L, static_cast<const uint8_t*>(x), x_exp, w, scales, offsets, out, st);
        return few<T>(L, static_cast<const T*>(x), x_exp, w, scales, offsets, out, st);
    }
    Linear4Dims D = L;
    const __nv_bfloat16* rows = static_cast<const __nv_bfloat16*>(x);
    if (kind != Rows4::kBf16 || (uintptr_t)x % 16 || L.sx % 8) {
        const int64_t n = L.rows * (L.n_in / 8);
        const unsigned blocks = (unsigned)((n + 255) / 256);
        if (kind == Rows4::kF32) linear4_rows_kernel<<<blocks, 256, 0, st>>>(L, static_cast<const float*>(x), x_exp, parts);
        else if (kind == Rows4::kE4m3) linear4_rows_kernel<<<blocks, 256, 0, st>>>(L, static_cast<const uint8_t*>(x), x_exp, parts);
        else linear4_rows_kernel<<<blocks, 256, 0, st>>>(L, static_cast<const __nv_bfloat16*>(x), x_exp, parts);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        rows = parts;
        D.sx = L.n_in;
    }
    return launch_linear4_tc<T>(D, linear4_parts(kind), rows, w, scales, offsets, out, st);
}

template <typename T>
cudaError_t launch_linear4_quantize(const Linear4Dims& L, const T* weight, uint8_t* w, T* scales, T* offsets,
                                    cudaStream_t st) {
    const int64_t n = (int64_t)L.n_out * (L.n_in / L.group);
    linear4_quantize_kernel<T><<<(unsigned)((n + 7) / 8), 256, 0, st>>>(L, weight, w, scales, offsets);
    return cudaGetLastError();
}

#define HLA_LINEAR4(T)                                                                                                \
    template cudaError_t launch_linear4<T>(const Linear4Dims&, Rows4, const void*, const uint8_t*, const uint8_t*,    \
                                           const T*, const T*, T*, __nv_bfloat16*, cudaStream_t);                     \
    template cudaError_t launch_linear4_quantize<T>(const Linear4Dims&, const T*, uint8_t*, T*, T*, cudaStream_t);
HLA_LINEAR4(float)
HLA_LINEAR4(__nv_bfloat16)

}  // namespace hla
