// Products of more than sixteen rows with 4-bit weights on the 5th-generation tensor cores.
//
// D [128 rows of W, N tokens] = A B^T per group of inputs: A = q - 8 in bf16 (exact, as every product is), B the
// tokens' rows.  A row's sums of a group are read back, scaled in fp32 and added to the row's own registers, so that no
// weight is rounded; offsets times the group's sums of x, which a product with ones gives.
//
// A block takes 128 rows and, in a cluster of C blocks, a C-th of the inputs, 128 at a time:
//   one warp     brings tiles of W (128 x 64 bytes) and of x (N x 128, in two blocks of 64) by TMA through a ring;
//   four or eight warps  take their rows' words from the ring, form q - 8 and put them into tensor memory, which A is
//                read from (two buffers), so that shared memory holds a weight in half a byte only;
//   one warp     issues the products, a group into one of two to four buffers of sums;
//   four (eight) warps read a group's sums (32 tokens a thread at most), scale and add them up.
// The cluster's sums are added through distributed shared memory, in order of its blocks.
//
// Bound by the chain of waits of a tile of 128 inputs, about 1600 cycles with unpacking, products and adding in step: 61 rows
// through 5120 x 10240 35 us, of which the 20 tiles of a block take 17 and the cluster's sums 4 (blocks that share an SM 27).
// Buffers of 64 inputs 39 us; one wait for all loads of a group's sums 44.
#include <algorithm>

#include "layer.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace hla {

namespace {

constexpr int kTile = 128;           // rows of W
constexpr uint32_t kPolls = 1u << 22;
constexpr uint32_t kOnes = 128;      // columns: two buffers of A (128 inputs in 64 columns each), ones, sums

template <int N, int PARTS, bool OFFS>
struct Shape {
    static constexpr int kAdd = N > 32 ? 8 : 4;  // adding warps
    static constexpr int kPer = 32;             // tokens of an adding thread
    // Sets of four unpacking warps, a buffer of A in turn.  64 tokens: one, for the registers that adding takes.
    static constexpr int kSets = N > 32 ? 1 : 2;
    static constexpr int kLoad = 4 * kSets, kIssue = kLoad + 1, kAdd0 = kLoad + 2;  // warps
    static constexpr int kWarps = kAdd0 + kAdd, kThreads = 32 * kWarps;
    static constexpr uint32_t kSums = OFFS ? 160 : 128;
    static constexpr int kBufs = OFFS || N == 64 ? 2 : 4;  // of sums
    static constexpr uint32_t kCols = kSums + kBufs * N * (OFFS ? 2 : 1) > 256 ? 512 : 256;
    static constexpr int kW = kTile * 64, kX = N * 128;  // bytes of a stage's W, of 64 inputs of x
    static constexpr int kStage = kW + 2 * PARTS * kX;
    static constexpr int kStages = std::max(2, std::min(8, 102400 / kStage));
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage;
    static constexpr size_t kNeed = std::max<size_t>(kSmem, 1024 + (size_t)N * kTile * 4);
};

// Eight weights of a word less 8, as four pairs of bf16: 0x4300 | q is 128 + q.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t* o) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu, off = 0x43084308u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = (__byte_perm(even, odd, i | 4 << 4 | (4 + i) << 8 | 4 << 12) & 0x00ff00ffu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(reinterpret_cast<const __nv_bfloat162&>(y), reinterpret_cast<const __nv_bfloat162&>(off));
        o[i] = reinterpret_cast<const uint32_t&>(d);
    }
}

// A place in a ring of n barriers, and the parity of the phase it is in.
struct Ring {
    int i = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            turn ^= 1;
        }
    }
};

template <typename T, int N, int PARTS, bool OFFS>
__global__ void __launch_bounds__(Shape<N, PARTS, OFFS>::kThreads, Shape<N, PARTS, OFFS>::kCols == 256 && PARTS == 1 ? 2 : 1)
linear4_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Linear4Dims L,
                  const T* __restrict__ scales, const T* __restrict__ offsets, T* __restrict__ out, int n_split) {
    using S = Shape<N, PARTS, OFFS>;
    extern __shared__ uint8_t raw[];
    __shared__ alignas(8) uint64_t bars[2 * S::kStages + 4 + 2 * S::kBufs + 1];
    __shared__ uint32_t tmem_at;
    __shared__ int bad;
    const uint32_t ring = (umma::smem_addr(raw) + 1023u) & ~1023u;
    float* const part = reinterpret_cast<float*>(raw + (ring - umma::smem_addr(raw)));  // [token][row], at the end
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = n_split > 1 ? cluster_rank() : 0;
    const int n0 = blockIdx.x / n_split * kTile;
    const int64_t m0 = (int64_t)blockIdx.y * N;
    const int n_groups = L.n_in / L.group, stages = (L.n_in + 127) / 128, halves = (L.n_in + 63) / 64;
    const int s0 = (int)((int64_t)stages * rank / n_split), s1 = (int)((int64_t)stages * (rank + 1) / n_split);
    const int h1 = min(2 * s1, halves);  // (64 inputs each)
    auto bar = [&](int i) { return umma::smem_addr(bars + i); };
    const int kFull = 0, kEmpty = S::kStages, kAFull = 2 * S::kStages, kAEmpty = kAFull + 2, kDFull = kAEmpty + 2,
              kDEmpty = kDFull + S::kBufs, kEnd = kDEmpty + S::kBufs;
    if (threadIdx.x == 0) {
        bad = 0;
        for (int i = 0; i < S::kStages; ++i) {
            umma::mbar_init(bar(kFull + i), 1);
            umma::mbar_init(bar(kEmpty + i), 5);  // four unpacking warps, and the products
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar(kAFull + i), 4);
            umma::mbar_init(bar(kAEmpty + i), 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            umma::mbar_init(bar(kDFull + i), 1);
            umma::mbar_init(bar(kDEmpty + i), S::kAdd);
        }
        umma::mbar_init(bar(kEnd), 1);
        umma::fence_mbar_init();
    }
    if (warp == 0) umma::tmem_alloc(&tmem_at, S::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_at;
    // Every wait ends: one that runs out leaves the block's outputs NaN.
    auto wait = [&](int i, uint32_t parity) -> bool {
#pragma unroll 1
        for (int k = 0; k < 256; ++k)  // (the bounded wait below reads the time, which takes longer than most waits do)
            if (__all_sync(0xffffffffu, umma::mbar_try_wait(bar(i), parity))) return true;
        const bool ok = !*(volatile int*)&bad && umma::mbar_wait(bar(i), parity, kPolls);
        if (__all_sync(0xffffffffu, ok)) return true;
        bad = 1;
        return false;
    };
    float2 acc[S::kPer / 2];
#pragma unroll
    for (int i = 0; i < S::kPer / 2; ++i) acc[i] = make_float2(0.f, 0.f);

    if (warp < S::kLoad) {  // unpacking
        const int row = (warp & 3) * 32 + lane, set = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        if constexpr (OFFS) {
            if (set == 0) {
                uint32_t ones[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) ones[i] = 0x3f803f80u;
                umma::tmem_st16_async(lanes + kOnes, ones);
            }
        }
        Ring in;
        for (int i = 0; i < set; ++i) in.next(S::kStages);
        for (int s = s0 + set; s < s1; s += S::kSets) {
            const int i = s - s0, buf = i & 1;
            if (!wait(kFull + in.i, in.turn)) break;
            const uint32_t at = ring + in.i * S::kStage + row * 64;
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 4; ++c)  // 16-byte chunks, swizzled over 64 bytes
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                             : "r"(at + (((uint32_t)c ^ ((uint32_t)row >> 1 & 3u)) << 4)));
            if (!wait(kAEmpty + buf, (uint32_t)(i >> 1 & 1) ^ 1)) break;
            umma::fence_after_sync();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) unpack8(w[4 * c + k], o + 4 * k);
                umma::tmem_st16_async(lanes + buf * 64 + 16 * c, o);
            }
            umma::tmem_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                umma::mbar_arrive(bar(kAFull + buf));
                umma::mbar_arrive(bar(kEmpty + in.i));
            }
            for (int k = 0; k < S::kSets; ++k) in.next(S::kStages);
        }
    } else if (warp == S::kLoad) {  // loads
        Ring in;
        int loaded = 0;
        for (int s = s0; s < s1; ++s) {
            if (!wait(kEmpty + in.i, in.turn ^ 1)) break;
            if (lane == 0) {
                const uint32_t at = ring + in.i * S::kStage, full = bar(kFull + in.i);
                const int hs = min(2, h1 - 2 * s);
                tma::expect_tx(full, S::kW + hs * PARTS * S::kX);
                tma::tensor_load_2d(at, &map_w, s * 64, n0, full);
                for (int h = 0; h < hs; ++h)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
                        tma::tensor_load_2d(at + S::kW + (h * PARTS + p) * S::kX, &map_x, s * 128 + h * 64,
                                            (int)(p * L.rows + m0), full);
            }
            __syncwarp();
            ++loaded;
            in.next(S::kStages);
        }
        if (*(volatile int*)&bad) {  // copies in flight end before the block does
            Ring r;
            for (int k = 0; k < loaded; ++k) {
                if (k + S::kStages >= loaded) umma::mbar_wait(bar(kFull + r.i), r.turn, kPolls);
                r.next(S::kStages);
            }
        }
    } else if (warp == S::kIssue) {  // products
        const uint32_t lead = umma::elect_one(), idesc = umma::idesc_bf16(kTile, N, false, false);
        const uint64_t b0 = umma::kmajor(ring + S::kW, N, 0);
        // A group's sums over PER products; straight code, as one warp issues for all others (with the group's size as a
        // variable a product took 250 cycles to issue).
        auto issue = [&](auto per) -> bool {
            constexpr int PER = decltype(per)::value;
            Ring in, d;
            for (int s = s0; s < s1; ++s) {
                const int i = s - s0, buf = i & 1;
                // (those who unpacked the weights had waited for the stage, x and all)
                if (!wait(kAFull + buf, (uint32_t)(i >> 1 & 1))) return false;
                const uint64_t b = b0 + (uint64_t)(in.i * S::kStage >> 4);
                const uint32_t at = tmem + buf * 64;
                const bool half = 2 * s + 1 >= h1;  // a tile that ends after 64 inputs
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k == 4 && half) break;
                    const bool first = k % PER == 0;
                    if (first) {
                        if (!wait(kDEmpty + d.i, d.turn ^ 1)) return false;
                        umma::fence_after_sync();
                    }
                    const uint32_t sums = tmem + S::kSums + d.i * N * (OFFS ? 2 : 1);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const uint64_t bk = b + ((k >> 2) * PARTS + p) * (S::kX >> 4) + 2 * (k & 3);
                        umma::mma_ts_lead(sums, at + 8 * k, bk, idesc, !first || p > 0, lead);
                        if constexpr (OFFS) umma::mma_ts_lead(sums + N, tmem + kOnes, bk, idesc, !first || p > 0, lead);
                    }
                    if (k % PER == PER - 1) {
                        if (lead) umma::commit(bar(kDFull + d.i));
                        d.next(S::kBufs);
                    }
                }
                if (lead) {
                    umma::commit(bar(kAEmpty + buf));
                    umma::commit(bar(kEmpty + in.i));
                }
                in.next(S::kStages);
                __syncwarp();
            }
            return true;
        };
        const bool go = L.group == 128  ? issue(std::integral_constant<int, 8>())
                        : L.group == 64 ? issue(std::integral_constant<int, 4>())
                                        : issue(std::integral_constant<int, 2>());
        if (!go) {  // (otherwise every product has been waited for, by those who add)
            if (lead) umma::commit(bar(kEnd));
            __syncwarp();
            umma::mbar_wait(bar(kEnd), 0, kPolls);
        }
    } else {  // adding
        const int u = warp - S::kAdd0, quad = warp & 3, t0 = (u >> 2) * S::kPer;
        const int row = n0 + quad * 32 + lane;
        const int64_t at = (int64_t)min(row, L.n_out - 1) * n_groups;
        const int g0 = s0 * 128 / L.group, g1 = (h1 * 64 + L.group - 1) / L.group;
        auto scale_at = [&](const T* p, int g) { return to_f32(p[at + min(g, n_groups - 1)]); };
        float sc = scale_at(scales, g0), of = OFFS ? scale_at(offsets, g0) : 0.f;
        Ring d;
        for (int g = g0; g < g1; ++g) {
            const float sc1 = scale_at(scales, g + 1), of1 = OFFS ? scale_at(offsets, g + 1) : 0.f;
            if (!wait(kDFull + d.i, d.turn)) break;
            umma::fence_after_sync();
            const uint32_t sums = tmem + ((uint32_t)quad << 21) + S::kSums + d.i * N * (OFFS ? 2 : 1) + t0;
#pragma unroll
            for (int k = 0; k < (OFFS ? 2 : 1); ++k) {
                const float2 f = make_float2(k ? of : sc, k ? of : sc);
#pragma unroll
                for (int c = 0; c < S::kPer; c += 16) {
                    float v[16];
                    umma::tmem_ld16(sums + k * N + c, v);
                    if (k == (OFFS ? 1 : 0) && c + 16 == S::kPer) {
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(bar(kDEmpty + d.i));
                    }
                    if (g < n_groups) {  // (half a tile may lie behind the last group)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[c / 2 + i] = ffma2(f, make_float2(v[2 * i], v[2 * i + 1]), acc[c / 2 + i]);
                    }
                }
            }
            d.next(S::kBufs);
            sc = sc1;
            of = of1;
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const bool failed = bad;
    if (warp == 0) umma::tmem_dealloc(tmem, S::kCols);
    const float nan = __int_as_float(0x7fc00000);
    if (n_split == 1) {
        if (warp < S::kAdd0) return;
        const int u = warp - S::kAdd0, t0 = (u >> 2) * S::kPer, row = n0 + (warp & 3) * 32 + lane;
        if (row >= L.n_out) return;
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) {
            const int64_t t = m0 + t0 + i;
            const float y = i & 1 ? acc[i / 2].y : acc[i / 2].x;
            if (t < L.rows) out[t * L.n_out + row] = from_f32<T>(failed ? nan : y);
        }
        return;
    }
    if (warp >= S::kAdd0) {
        const int u = warp - S::kAdd0, t0 = (u >> 2) * S::kPer, row = (warp & 3) * 32 + lane;
#pragma unroll
        for (int i = 0; i < S::kPer; ++i) part[(t0 + i) * kTile + row] = failed ? nan : i & 1 ? acc[i / 2].y : acc[i / 2].x;
    }
    cluster_sync_all();
    const int t0 = (int)(N * rank / n_split), t1 = (int)(N * (rank + 1) / n_split);
#pragma unroll 4
    for (int i = t0 * kTile + threadIdx.x; i < t1 * kTile; i += S::kThreads) {
        const int64_t t = m0 + i / kTile;
        const int row = n0 + i % kTile;
        if (t >= L.rows || row >= L.n_out) continue;
        out[t * L.n_out + row] = from_f32<T>(cluster_sum(part + i, n_split));
    }
    cluster_sync_all();  // no block leaves while its sums are read
}

template <typename T, int N, int PARTS, bool OFFS>
cudaError_t run(const CUtensorMap& map_w, const CUtensorMap& map_x, const Linear4Dims& L, const T* scales, const T* offsets,
                T* out, int n_split, cudaStream_t st) {
    using S = Shape<N, PARTS, OFFS>;
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [](int, int*) {
        return cudaFuncSetAttribute(linear4_tc_kernel<T, N, PARTS, OFFS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kNeed);
    });
    if (e != cudaSuccess) return e;
    const int tiles = (L.n_out + kTile - 1) / kTile;
    ClusterCfg cfg(dim3((unsigned)(tiles * n_split), (unsigned)((L.rows + N - 1) / N)), S::kThreads, S::kNeed, st, n_split);
    return cudaLaunchKernelEx(&cfg.cfg, linear4_tc_kernel<T, N, PARTS, OFFS>, map_w, map_x, L, scales, offsets, out, n_split);
}

}  // namespace

template <typename T>
cudaError_t launch_linear4_tc(const Linear4Dims& L, int parts, const __nv_bfloat16* x, const uint8_t* w, const T* scales,
                              const T* offsets, T* out, cudaStream_t st) {
    const int n = L.rows <= 32 ? 32 : 64;
    CUtensorMap map_w, map_x;
    if (!tma::make_map_2d(&map_w, w, 1, (uint64_t)L.n_in / 2, (uint64_t)L.n_out, (uint64_t)L.n_in / 2, 64, kTile) ||
        !tma::make_map_2d(&map_x, x, 2, (uint64_t)L.n_in, (uint64_t)L.rows * parts, (uint64_t)L.sx * 2, 64, (uint32_t)n))
        return cudaErrorInvalidValue;
    // Two blocks an SM, one where offsets' sums or three parts of x take the room (24 rows through 4096 x 14336 with offsets: 25 us
    // in single blocks, 32 in clusters of two; 61 through 5120 x 10240 without: 39, 35 and, in clusters of four, 33: the rule
    // takes two there, as it counts a block's start and end as six steps, and loses those 2 us).
    const int resident = offsets || parts == 3 ? 152 : 304;
    const int c = linear4_split((int64_t)((L.n_out + kTile - 1) / kTile) * ((L.rows + n - 1) / n), (L.n_in + 127) / 128, resident, 6);
    auto go = [&](auto nn, auto np, auto offs) {
        return run<T, decltype(nn)::value, decltype(np)::value, decltype(offs)::value>(map_w, map_x, L, scales, offsets, out, c, st);
    };
    auto with_parts = [&](auto nn, auto offs) {
        return parts == 3 ? go(nn, std::integral_constant<int, 3>(), offs) : go(nn, std::integral_constant<int, 1>(), offs);
    };
    auto with_rows = [&](auto offs) {
        if (n == 32) return with_parts(std::integral_constant<int, 32>(), offs);
        return with_parts(std::integral_constant<int, 64>(), offs);
    };
    return offsets ? with_rows(std::true_type()) : with_rows(std::false_type());
}

template cudaError_t launch_linear4_tc<float>(const Linear4Dims&, int, const __nv_bfloat16*, const uint8_t*, const float*,
                                              const float*, float*, cudaStream_t);
template cudaError_t launch_linear4_tc<__nv_bfloat16>(const Linear4Dims&, int, const __nv_bfloat16*, const uint8_t*,
                                                      const __nv_bfloat16*, const __nv_bfloat16*, __nv_bfloat16*, cudaStream_t);

}  // namespace hla
