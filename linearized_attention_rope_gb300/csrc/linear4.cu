// Products of a few rows with 4-bit weights: y = x W^T, W[n][k] = scale (q - 8)
// + offset, a scale (and offset) per row n and group of 32, 64 or 128 inputs k.
//
// Bound by the weights' bytes: half a byte each, read once per 64 rows of x.
// Products on the warp-level tensor instruction (m16n8k16, bf16 in, fp32 sums):
// the 16 rows are rows of W, the 8 columns tokens.  q - 8 is exact in bf16 and so
// is every product; a group's sum is scaled in fp32 as it is added to the row's.
// (Scaled weights would have to be rounded to bf16 each.)  Which k a lane's
// operands stand for is free, as long as both operands agree: a lane takes 16
// bytes of a weight row as they lie, and the same 32 inputs of its token.
// Offsets: the group's sum of x, from a product with ones, times the offset.
//
// fp32 rows enter as three bf16 parts, cut off 8 bits at a time (nothing is
// lost), 8-bit rows as bf16 (exact, too): a small launch before the product
// writes the parts.
#include <algorithm>

#include "layer.cuh"

namespace hla {

namespace {

constexpr int kWarps4 = 8;

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

// RT: tiles of 16 weight rows of a block; MT: tiles of 8 tokens; PARTS: of x.
// A block's eight warps take the row tiles' groups of 128 inputs in turn, and add up at the end, in order.
template <typename T, int RT, int MT, int GROUP, int PARTS, bool OFFS>
__global__ void __launch_bounds__(32 * kWarps4)
linear4_kernel(const Linear4Dims L, const __nv_bfloat16* __restrict__ x, int64_t part_stride, const uint8_t* __restrict__ w,
               const T* __restrict__ scales, const T* __restrict__ offsets, T* __restrict__ out) {
    constexpr int kWords = GROUP / 32;  // 32-bit words of a lane per group: 8 inputs each
    extern __shared__ float sums[];     // [warp][token][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const int n0 = blockIdx.x * 16 * RT;
    const int64_t m0 = (int64_t)blockIdx.y * 8 * MT;
    const int n_groups = L.n_in / GROUP;
    const uint8_t* wr[RT][2];
    int64_t sr[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = min(n0 + r * 16 + h * 8 + gq, L.n_out - 1);
            wr[r][h] = w + (int64_t)n * (L.n_in / 2) + tq * (kWords * 4);
            sr[r][h] = (int64_t)n * n_groups;
        }
    const __nv_bfloat16* xr[MT];
    bool on[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t t = m0 + m * 8 + gq;
        on[m] = t < L.rows;
        xr[m] = x + (on[m] ? t : 0) * L.sx + tq * (kWords * 8);
    }
    float acc[RT][MT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][m][i] = 0.f;
    const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll 2
    for (int g = warp; g < n_groups; g += kWarps4) {
        uint32_t q[RT][2][kWords];
        float sc[RT][2], of[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(wr[r][h] + (int64_t)g * (GROUP / 2));
                if constexpr (kWords == 4) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
                    q[r][h][0] = v.x; q[r][h][1] = v.y; q[r][h][2] = v.z; q[r][h][3] = v.w;
                } else if constexpr (kWords == 2) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                    q[r][h][0] = v.x; q[r][h][1] = v.y;
                } else {
                    q[r][h][0] = __ldg(p);
                }
                sc[r][h] = to_f32(scales[sr[r][h] + g]);
                if (OFFS) of[r][h] = to_f32(offsets[sr[r][h] + g]);
            }
        float part[RT][MT][4], total[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                total[m][i] = 0.f;
#pragma unroll
                for (int r = 0; r < RT; ++r) part[r][m][i] = 0.f;
            }
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            uint32_t a[RT][2][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    a[r][s][0] = nibbles(q[r][0][k], 8 * s);
                    a[r][s][1] = nibbles(q[r][1][k], 8 * s);
                    a[r][s][2] = nibbles(q[r][0][k], 8 * s + 4);
                    a[r][s][3] = nibbles(q[r][1][k], 8 * s + 4);
                }
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (on[m]) v = __ldg(reinterpret_cast<const uint4*>(xr[m] + p * part_stride + (int64_t)g * GROUP + k * 8));
                    const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
                    const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        mma16816(part[r][m], a[r][0], b0, b1);
                        mma16816(part[r][m], a[r][1], b2, b3);
                    }
                    if (OFFS) {
                        mma16816(total[m], ones, b0, b1);
                        mma16816(total[m], ones, b2, b3);
                    }
                }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[r][m][i] = fmaf(sc[r][i >> 1], part[r][m][i], acc[r][m][i]);
                    if (OFFS) acc[r][m][i] = fmaf(of[r][i >> 1], total[m][i], acc[r][m][i]);
                }
    }
    constexpr int kRows = 16 * RT, kTok = 8 * MT, kPitch = kRows + 1;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sums[(warp * kTok + m * 8 + tq * 2 + (i & 1)) * kPitch + r * 16 + (i >> 1) * 8 + gq] = acc[r][m][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kTok; i += 32 * kWarps4) {
        const int t = i / kRows, n = i - t * kRows;
        if (m0 + t >= L.rows || n0 + n >= L.n_out) continue;
        float y = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps4; ++u) y += sums[(u * kTok + t) * kPitch + n];
        out[(m0 + t) * L.n_out + n0 + n] = from_f32<T>(y);
    }
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
            float v = p[j];
            const bool fine = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
            if (v != v) v = __uint_as_float(0x7fc00000u);
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                const float top = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
                o[s].x[j] = from_f32<__nv_bfloat16>(top);
                v = fine ? v - top : 0.f;
            }
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

template <typename T, int RT, int MT, int GROUP, int PARTS, bool OFFS>
cudaError_t run(const Linear4Dims& L, const __nv_bfloat16* x, int64_t part_stride, const uint8_t* w, const T* scales,
                const T* offsets, T* out, cudaStream_t st) {
    constexpr size_t sm = (size_t)kWarps4 * 8 * MT * (16 * RT + 1) * sizeof(float);
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [](int, int*) {
        return cudaFuncSetAttribute(linear4_kernel<T, RT, MT, GROUP, PARTS, OFFS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
    });
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((L.n_out + 16 * RT - 1) / (16 * RT)), (unsigned)((L.rows + 8 * MT - 1) / (8 * MT)));
    linear4_kernel<T, RT, MT, GROUP, PARTS, OFFS><<<grid, 32 * kWarps4, sm, st>>>(L, x, part_stride, w, scales, offsets, out);
    return cudaGetLastError();
}

}  // namespace

int linear4_parts(Rows4 kind) { return kind == Rows4::kF32 ? 3 : 1; }

template <typename T>
cudaError_t launch_linear4(const Linear4Dims& L, Rows4 kind, const void* x, const uint8_t* x_exp, const uint8_t* w,
                           const T* scales, const T* offsets, T* out, __nv_bfloat16* parts, cudaStream_t st) {
    if (L.rows == 0) return cudaSuccess;
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
    if (L.rows > 8) return launch_linear4_tc<T>(D, linear4_parts(kind), rows, w, scales, offsets, out, st);
    const int64_t stride = L.rows * L.n_in;
    auto go = [&](auto group, auto np, auto offs) {
        return run<T, 1, 1, decltype(group)::value, decltype(np)::value, decltype(offs)::value>(D, rows, stride, w, scales, offsets, out, st);
    };
    auto with_offsets = [&](auto group, auto np) {
        return offsets ? go(group, np, std::true_type()) : go(group, np, std::false_type());
    };
    auto with_group = [&](auto np) {
        if (L.group == 128) return with_offsets(std::integral_constant<int, 128>(), np);
        if (L.group == 64) return with_offsets(std::integral_constant<int, 64>(), np);
        return with_offsets(std::integral_constant<int, 32>(), np);
    };
    if (kind == Rows4::kF32) return with_group(std::integral_constant<int, 3>());
    return with_group(std::integral_constant<int, 1>());
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
