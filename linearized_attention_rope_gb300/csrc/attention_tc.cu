// Packed causal attention of bf16 layers on the tcgen05 tensor cores:
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  out = O / sum P
// in one pass over the keys with the running reference m and sum.
//
// A block takes two query tiles (128 rows each, see attention_tc.cuh) of one
// kv head and walks the keys they see in tiles of 128:
//   warp 8        TMA: both query tiles, then K and V tiles into a ring of
//                 slots; clears infinities and NaN in value rows that not all
//                 rows see (a probability of 0 would pass them on; the rows
//                 that do see them get them back at the end)
//   warp 9        issues every product; S of both tiles (128 columns each) and
//                 O of both (d columns each) in TMEM.  The whole warp runs the
//                 loop, one lane's instruction is active: a product issued from
//                 a branch that one lane took costs ~90 cycles, more than the 64
//                 that it takes the tensor cores
//   warp 10       waits for the scores' completion in place of the softmax warps
//                 and releases them by a hardware barrier: eight warps polling
//                 shared memory take issue slots from the exponentials
//   warp 11       asks for the next item while this one is worked on
//   warps 0 - 3   softmax of tile 0, one row per thread
//   warps 4 - 7   the same of tile 1
// Items go to the blocks that run first, the longest first (launch control
// cancels a block that has not started and takes its index): a grid that fits
// the SMs once, and no wave of short items behind long ones.
// While the tensor cores form P V and the next S of one tile (the probabilities
// overwrite the first half of their scores' columns and are read from TMEM as
// the A operand), the other tile's softmax runs.
//
// The reference m follows the running maximum only when it has grown by more
// than 2^8 (the sum and O use the same m, so the result is the same); a row's
// O is then rescaled in TMEM by its own softmax thread, after the products
// before it have completed (they complete before the scores it waits for).
//
// Query tiles that see one key tile take their probabilities in two bf16 parts,
// the rounded value and what that leaves, in two products: the roundings of a
// few keys do not average out as those of many do (outputs of a few rows were
// off by up to 1.5 times the rounding of the result, now by 1.00; 19 x 64 tokens
// 11.6 -> 12.3 us, 4 x 4096 385 -> 394).  Rows of more tiles keep the one: up to 1.5
// where few of their keys have weight.
//
// With fewer items than SMs (a short chunk of a prompt behind many keys, few
// heads), the keys of each item are cut into parts, an item each; a part leaves
// its rows' outputs in fp32 with their log-sum-exp, and a second kernel adds
// them in order.
//
// Long prompts are bound by the tensor cores: bf16, 32/8 heads of 128, 32768 tokens in 5.2 to 5.4 ms (1620 to
// 1690 TFLOP/s; a large library product sustains 1695).  4096 in 104 to 108 us (1300): there neither they (54 %
// active) nor the issue slots (1.2 instructions of 4 a cycle) are the limit, nor the masked half of the edge tiles (3 %
// more key tiles than the visible scores need) or the items' lengths; 4 x 4096 tokens, 32/8 heads of 64, 270 us, the
// same (35 % and 1.5).  What is, the exponentials' rate or the chain of steps within a tile, has not been measured.
// 64 rows over 131072 keys: 105 us.
#include <type_traits>

#include "attention_tc.cuh"

namespace hla {

namespace {

using namespace attn_tc;

constexpr float kLazy = 8.0f;
constexpr int kBarS = 1, kBarP = 3;  // hardware barriers: scores ready, probabilities ready (+ tile)

// Of an item: the keys found with infinities or NaN, one bit for each from key `some` on; where its keys lie.
struct alignas(16) Marks {
    uint32_t bit[8];
    int some, kv, k0, pad;
};

template <int D> struct Cfg {
    static constexpr uint32_t kTile = kRows * D * 2;  // bytes of a tile
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTile, kBar = kRing + kSlots * kTile;
    static constexpr int kMarks = 8;  // items whose marks are kept
    static constexpr uint32_t kMark = kBar + 320 + 96, kSmem = kMark + kMarks * sizeof(Marks) + 1024;
    static_assert(sizeof(ItemRing) <= 96, "shared memory layout");
    // TMEM columns
    static constexpr uint32_t kS = 0, kO = 256, kCols = 512;
};

template <int D>
__global__ void __launch_bounds__(kBlock, 1)
attention_tc_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                    const __nv_bfloat16* __restrict__ v, const int32_t* __restrict__ cu_q,
                    const int32_t* __restrict__ cu_k, int lpack, int parts,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, float* __restrict__ part_o,
                    float* __restrict__ part_lse, int32_t* __restrict__ err) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int pack = 1 << lpack, qb = kRows >> lpack, n_hg = A.Hq >> lpack;
    if (blockIdx.x == 0) {
        attn_check_table(cu_q, A.n_seqs, A.total_q, err);
        attn_check_table(cu_k, A.n_seqs, A.total_k, err);
    }
    const uint32_t base = umma::smem_addr(sm), bars = base + C::kBar;
    const uint32_t bar_q = bars, bar_qe = bar_q + 16, bar_full = bar_qe + 16, bar_empty = bar_full + 8 * C::kSlots;
    const uint32_t bar_s = bar_empty + 8 * C::kSlots, bar_o = bar_s + 16, bar_oe = bar_o + 16, bar_fix = bar_oe + 16;
    const uint32_t bar_it = bar_fix + 32, bar_ie = bar_it + 8 * kItems, bar_ask = bar_ie + 8 * kItems, bar_want = bar_ask + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kBar + 316);
    ItemRing* items = reinterpret_cast<ItemRing*>(sm + C::kBar + 320);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar_q + 8 * i, 1);
            umma::mbar_init(bar_qe + 8 * i, 1);
            umma::mbar_init(bar_s + 8 * i, 1);
            umma::mbar_init(bar_o + 8 * i, 1);
            umma::mbar_init(bar_oe + 8 * i, 4);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            umma::mbar_init(bar_full + 8 * i, 1);
            umma::mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) umma::mbar_init(bar_fix + 8 * i, 1);
        umma::mbar_init(bar_ask, 1);
        umma::mbar_init(bar_want, 1);
        for (int i = 0; i < kItems; ++i) {
            umma::mbar_init(bar_it + 8 * i, 1);
            umma::mbar_init(bar_ie + 8 * i, kItemWarps);
        }
        umma::fence_mbar_init();
    }
    if (warp == 9) umma::tmem_alloc(tmem_slot, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // what an item's two tiles see: keys [0, end), tile t in nt = n[t] key tiles
    // keys from `some` on are seen by some of the rows only, in key tiles from `mixed` on (the last tile at least).  With
    // one key tile, all of them: an infinity times the two parts of a probability is no infinity.
    struct Span { int end, n0, n1, n, some, mixed; };
    auto span = [&](const Item& it) {
        auto key_end = [&](int t) {
            const int p0 = it.first + t * qb;
            return p0 < it.lq ? max(0, min(it.lk, min(p0 + qb, it.lq) + it.off)) : 0;
        };
        const int e0 = key_end(0), e1 = key_end(1);
        const int n0 = __shfl_sync(0xffffffffu, (e0 + kRows - 1) / kRows, 0);
        const int n1 = __shfl_sync(0xffffffffu, (e1 + kRows - 1) / kRows, 0);
        const int end = max(e0, e1), some = n0 == 1 || n1 == 1 ? 0 : max(0, min(end, it.first + it.off + 1));
        return Span{end, n0, n1, max(n0, n1), some, __shfl_sync(0xffffffffu, min(max(n0, n1) - 1, some / kRows), 0)};
    };
    auto slot_of = [&](int use) { return use % C::kSlots; };
    auto par_of = [&](int use) { return (uint32_t)(use / C::kSlots) & 1u; };

    if (warp >= 8) {
        give_registers();
        bool ok = true;
        if (warp == 8) {
            // ---- loads: of an item, use 2 j of the ring is K tile j, use 2 j + 1 V tile j
            int use = 0, items_q[2] = {0, 0}, n_fix = 0;
            for (int i = 0;; ++i) {
                const Item it = next_item(items, i, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                const int kv = it.head / A.G, ask_at = max(0, 2 * sp.n - 3);
                // (kept for eight items; an item is handed out only once every warp has started on the one before last)
                Marks* marks = reinterpret_cast<Marks*>(sm + C::kMark) + (i & (C::kMarks - 1));
                if (lane < 8) marks->bit[lane] = 0u;
                if (lane == 0) {
                    marks->some = sp.some;
                    marks->kv = kv;
                    marks->k0 = it.k0;
                }
                __syncwarp();
                if (sp.n == 0 && lane == 0) umma::mbar_arrive(bar_want);
                for (int u = 0; u < 2 * sp.n; ++u) {
                    if (u == ask_at && lane == 0) umma::mbar_arrive(bar_want);  // time to look for the next item
                    if (!ok) continue;
                    const int slot = slot_of(use + u);
                    if (use + u >= C::kSlots)
                        ok = wait_or_flag(bar_empty + 8 * slot, par_of(use + u - C::kSlots), err);
                    if (!ok) continue;
                    if (lane == 0) {
                        tma::expect_tx(bar_full + 8 * slot, C::kTile);
                        for (int b = 0; b < D / 64; ++b)
                            tma::tensor_load_3d(base + C::kRing + slot * C::kTile + b * (kRows * 128),
                                                u & 1 ? &map_v : &map_k, 64 * b, kv, it.k0 + (u >> 1) * kRows,
                                                bar_full + 8 * slot);
                    }
                    if ((u & 1) && (u >> 1) >= sp.mixed) {
                        // (The ring holds at most four V tiles, so four barriers keep a tile's signal until the products
                        // have seen it.)
                        static_assert(C::kSlots <= 8, "tiles in the ring");
                        const int k0 = (u >> 1) * kRows;
                        ok = wait_or_flag(bar_full + 8 * slot, par_of(use + u), err);
                        if (!ok) continue;
                        unsigned char* tile = sm + C::kRing + slot * C::kTile;
                        clear_nonfinite<D>(tile, max(0, sp.some - k0), kRows, [&](int row) {
                            const int key = k0 + row;  // (a row behind the last visible key is cleared only)
                            if (key < sp.end) atomicOr(marks->bit + ((key - sp.some) >> 5), 1u << ((key - sp.some) & 31));
                        });
                        umma::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(bar_fix + 8 * (n_fix & 3));
                        ++n_fix;
                    }
                    if (u > 0) continue;
                    for (int t = 0; t < 2 && ok; ++t) {  // the query tiles, once the last item's scores are formed
                        if ((t ? sp.n1 : sp.n0) == 0) continue;
                        if (items_q[t] > 0) ok = wait_or_flag(bar_qe + 8 * t, (items_q[t] - 1) & 1, err);
                        ++items_q[t];
                        if (ok && lane == 0) {
                            tma::expect_tx(bar_q + 8 * t, C::kTile);
                            for (int b = 0; b < D / 64; ++b)
                                tma::tensor_load_3d(base + C::kQ + t * C::kTile + b * (kRows * 128), &map_q, 64 * b,
                                                    it.head, it.q0 + it.first + t * qb, bar_q + 8 * t);
                        }
                    }
                }
                use += 2 * sp.n;
            }
            // after a failed wait, copies may be in flight: let them land (a failed wait has taken two seconds,
            // a copy takes microseconds)
        } else if (warp == 9) {
            // ---- products: one lane issues, the warp stays together
            const uint32_t lead = umma::elect_one();
            const uint32_t id_s = umma::idesc_bf16(kRows, kRows, false, false);
            const uint32_t id_o = umma::idesc_bf16(kRows, D, false, true);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = __all_sync(0xffffffffu, ok && wait_or_flag(bar, parity, err));
            };
            auto done = [&](uint32_t bar) {
                if (ok && lead) umma::commit(bar);
            };
            // the ring is used in the order K 0, V 0, K 1, V 1, ... of every item
            using Use = RingPos<C::kSlots>;
            Use ring;
            const uint64_t q_tile[2] = {umma::kmajor(base + C::kQ, kRows, 0), umma::kmajor(base + C::kQ + C::kTile, kRows, 0)};
            const uint64_t k_ring = umma::kmajor(base + C::kRing, kRows, 0);
            const uint64_t v_ring = umma::mnmajor(base + C::kRing, kRows * 128, 0);
            auto scores = [&](int t, uint32_t k_slot) {
                if (!ok) return;
                const uint64_t a = q_tile[t], b = k_ring + (uint64_t)(k_slot * (C::kTile / 16));
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t ks = (uint64_t)((s >> 2) * (kRows * 128 / 16) + (s & 3) * 2);
                    umma::mma_lead(tmem + C::kS + t * kRows, a + ks, b + ks, id_s, s > 0, lead);
                }
                if (lead) umma::commit(bar_s + 8 * t);
            };
            auto values = [&](int t, uint32_t v_slot, bool add, bool fine) {
                if (!ok) return;
                const uint64_t b = v_ring + (uint64_t)(v_slot * (C::kTile / 16));
#pragma unroll
                for (int s = 0; s < kRows / 16; ++s)
                    umma::mma_ts_lead(tmem + C::kO + t * D, tmem + C::kS + t * kRows + 8 * s, b + (uint64_t)(s * 128),
                                      id_o, add || s > 0, lead);
                if (fine)  // what rounding the probabilities left
#pragma unroll 1
                    for (int s = 0; s < kRows / 16; ++s)
                        umma::mma_ts_lead(tmem + C::kO + t * D, tmem + C::kS + t * kRows + kRows / 2 + 8 * s,
                                          b + (uint64_t)(s * 128), id_o, true, lead);
            };
            int count[2] = {0, 0}, n_fix = 0;  // items with tile t, cleared tiles
            for (int i = 0;; ++i) {
                const Item it = next_item(items, i, bar_it, bar_ie, err);
                if (__shfl_sync(0xffffffffu, it.head, 0) < 0) break;
                const Span sp = span(it);
                const int n = sp.n;
                if (n == 0) continue;
                const Use first = ring.next();
                wait(bar_full + 8 * first.slot, first.par);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int nt = t ? sp.n1 : sp.n0;
                    if (nt == 0) continue;
                    wait(bar_q + 8 * t, count[t] & 1);
                    umma::fence_after_sync();
                    scores(t, first.slot);
                    if (nt == 1) done(bar_qe + 8 * t);
                }
                done(bar_empty + 8 * first.slot);
                // one key tile; the ones that all rows see have a loop of their own, without the wait for the clearing
                auto step = [&](int j, auto mixed) {
                    const bool more = !decltype(mixed)::value || j + 1 < n;
                    const Use v = ring.next(), k = more ? ring.next() : v;
                    wait(bar_full + 8 * v.slot, v.par);
                    if (more) wait(bar_full + 8 * k.slot, k.par);
                    if (decltype(mixed)::value) {
                        wait(bar_fix + 8 * (n_fix & 3), (n_fix >> 2) & 1);
                        ++n_fix;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int nt = t ? sp.n1 : sp.n0;
                        if (j >= nt) continue;
                        if (j == 0 && count[t] > 0) wait(bar_oe + 8 * t, (count[t] - 1) & 1);  // O has been read
                        named_sync(kBarP + t, 160);
                        umma::fence_after_sync();
                        values(t, v.slot, j > 0, decltype(mixed)::value && nt == 1);
                        if (j + 1 < nt) scores(t, k.slot);
                        else done(bar_o + 8 * t);
                        if (j + 2 == nt) done(bar_qe + 8 * t);  // Q has been read for the last time
                    }
                    done(bar_empty + 8 * v.slot);
                    if (more) done(bar_empty + 8 * k.slot);
                };
                int j = 0;
                for (; j < sp.mixed; ++j) step(j, std::false_type{});
                for (; j < n; ++j) step(j, std::true_type{});
                count[0] += sp.n0 > 0;
                count[1] += sp.n1 > 0;
            }
        } else if (warp == 10) {
            // ---- "scores ready" passed on to the softmax warps, in the order the products are issued
            int seen[2] = {0, 0};
            for (int i = 0;; ++i) {
                const Item it = next_item(items, i, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                for (int j = 0; j < sp.n; ++j)
                    for (int t = 0; t < 2; ++t) {
                        if (j >= (t ? sp.n1 : sp.n0)) continue;
                        ok = ok && wait_or_flag(bar_s + 8 * t, seen[t] & 1, err);
                        ++seen[t];
                        umma::fence_after_sync();
                        umma::fence_before_sync();
                        named_arrive(kBarS + t, 160);
                    }
            }
        } else {
            schedule_items(A, cu_q, cu_k, 2 * qb, n_hg, false, items, bar_it, bar_ie, bar_ask, bar_want, err,
                           [&](int hg) { return hg << lpack; }, parts);
        }
    } else {
        take_registers();
        // ---- softmax, one row per thread
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) << 5) << 16;
        const uint32_t ts = tmem + lanes + C::kS + t * kRows, to = tmem + lanes + C::kO + t * D;
        const float cs = A.scale * kLog2e;
        int count = 0;  // items with this tile
        bool ok = true;
        for (int i = 0;; ++i) {
            int nt, limit;  // key tiles of the query tile; keys the row sees: [0, limit)
            int64_t at;     // the row's place in the output, or among the parts' (-1: none)
            {
                const Item it = next_item(items, i, bar_it, bar_ie, err);
                if (it.head < 0) break;
                const Span sp = span(it);
                const int pos = it.first + t * qb + (row >> lpack);
                nt = t ? sp.n1 : sp.n0;
                limit = pos < it.lq ? min(it.lk, pos + it.off + 1) : 0;
                at = pos < it.lq ? (it.part * A.total_q + it.q0 + pos) * A.Hq + it.head + (row & (pack - 1)) : -1;
            }
            float m = -INFINITY;
            float2 l = make_float2(0.f, 0.f);
            auto tile = [&](int j, auto fine) {
                named_sync(kBarS + t, 160);
                umma::fence_after_sync();
                float x[128];
                {
                    uint32_t r[4][32];
#pragma unroll
                    for (int b = 0; b < 4; ++b) umma::tmem_ld32_async(ts + 32 * b, r[b]);
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        umma::reg_fence32(r[b]);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[32 * b + e] = __uint_as_float(r[b][e]);
                    }
                }
                const int seen = limit - j * kRows;
                if (__any_sync(0xffffffffu, seen < kRows)) {
#pragma unroll
                    for (int e = 0; e < 128; ++e) x[e] = e < seen ? x[e] : -INFINITY;
                }
                float top[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) top[b] = fmaxf(x[b], x[b + 4]);
#pragma unroll
                for (int e = 8; e < 128; e += 8)
#pragma unroll
                    for (int b = 0; b < 4; ++b) top[b] = fmaxf(top[b], fmaxf(x[e + b], x[e + b + 4]));
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cs;
                const bool grow = mx > m + kLazy;
                if (__any_sync(0xffffffffu, grow)) {
                    const float corr = grow ? (m == -INFINITY ? 0.f : ex2(m - mx)) : 1.f;
                    if (grow) m = mx;
                    l.x *= corr;
                    l.y *= corr;
                    if (j > 0) {
#pragma unroll
                        for (int b = 0; b < D / 32; ++b) {
                            float o[32];
                            umma::tmem_ld32(to + 32 * b, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= corr;
                            umma::tmem_st32(to + 32 * b, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const float2 c2 = make_float2(cs, cs), m2 = make_float2(-ref, -ref);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 y = ffma2(make_float2(x[64 * b + 2 * e], x[64 * b + 2 * e + 1]), c2, m2);
                        const float2 w = make_float2(ex2(y.x), ex2(y.y));
                        l = fadd2(l, w);
                        p[e] = pack_bf2(w.x, w.y);
                    }
                    umma::tmem_st32_async(ts + 32 * b, p);
                    if constexpr (decltype(fine)::value) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 y = ffma2(make_float2(x[64 * b + 2 * e], x[64 * b + 2 * e + 1]), c2, m2);
                            p[e] = pack_bf2(ex2(y.x) - __uint_as_float(p[e] << 16),
                                            ex2(y.y) - __uint_as_float(p[e] & 0xffff0000u));
                        }
                        umma::tmem_st32_async(ts + kRows / 2 + 32 * b, p);
                    }
                }
                umma::tmem_wait_st();
                umma::fence_before_sync();
                named_arrive(kBarP + t, 160);
            };
            if (nt == 1) {  // the one key tile of short prompts: probabilities in two bf16 parts
                tile(0, std::true_type{});
            } else {
                for (int j = 0; j < nt; ++j) tile(j, std::false_type{});
            }
            // ---- the row's output
            const float sum = l.x + l.y;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (at >= 0) (parts > 1 ? part_lse : lse)[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
            if (nt > 0) ok = ok && wait_or_flag(bar_o + 8 * t, count & 1, err);
            umma::fence_after_sync();
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                float o[32];
                if (nt > 0) {
                    umma::tmem_ld32(to + 32 * b, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (b == D / 32 - 1 && nt > 0) {  // O may be overwritten
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(bar_oe + 8 * t);
                    ++count;
                }
                if (at >= 0 && parts > 1) {
                    float* dst = part_o + at * D + 32 * b;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(dst + e) =
                            make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
                } else if (at >= 0) {
                    __nv_bfloat16* dst = out + at * D + 32 * b;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(dst + e) = make_uint4(
                            pack_bf2(o[e] * inv, o[e + 1] * inv), pack_bf2(o[e + 2] * inv, o[e + 3] * inv),
                            pack_bf2(o[e + 4] * inv, o[e + 5] * inv), pack_bf2(o[e + 6] * inv, o[e + 7] * inv));
                }
            }
            // infinities and NaN that were kept out of the product: to the rows that see their keys
            const Marks* marks = reinterpret_cast<const Marks*>(sm + C::kMark) + (i & (C::kMarks - 1));
            const uint4 lo = *reinterpret_cast<const uint4*>(marks->bit), hi = *reinterpret_cast<const uint4*>(marks->bit + 4);
            if (nt > 0 && (lo.x | lo.y | lo.z | lo.w | hi.x | hi.y | hi.z | hi.w) != 0u && at >= 0) {
#pragma unroll 1
                for (int w = 0; w < 8; ++w)
#pragma unroll 1
                    for (uint32_t left = marks->bit[w]; left; left &= left - 1) {
                        const int key = marks->some + 32 * w + __ffs(left) - 1;
                        if (key >= limit) continue;
                        const __nv_bfloat16* src = v + (int64_t)(marks->k0 + key) * A.sv + marks->kv * D;
#pragma unroll 1
                        for (int e = 0; e < D; ++e) {
                            const float x = __bfloat162float(src[e]);
                            if (fabsf(x) < INFINITY) continue;
                            if (parts > 1) part_o[at * D + e] += x;
                            else out[at * D + e] = __float2bfloat16_rn(__bfloat162float(out[at * D + e]) + x);
                        }
                    }
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 9) umma::tmem_dealloc(tmem, C::kCols);
}

// Items (pairs of query tiles) over all sequences and head groups: at most, and about.
int64_t items_bound(const AttnDims& A) {
    const int pack = pack_of(A.G);
    return (A.total_q / (2 * (kRows / pack)) + A.n_seqs) * (A.Hq / pack);
}
int64_t items_about(const AttnDims& A) {
    const int pack = pack_of(A.G), rows = 2 * (kRows / pack);
    return std::max<int64_t>(A.n_seqs, (A.total_q + rows - 1) / rows) * (A.Hq / pack);
}

// Items that do not fill the SMs leave some idle.  With keys enough for parts of
// eight tiles, they are cut into the number of parts that takes least:
// - rows that are few beside the keys: rounds over the SMs, plus what the parts'
//   results cost, 0.55 of an item's time per item and SM, which separates the
//   cases measured (700 rows behind 20000 keys, 88 items: 239 us whole, 187 in
//   three parts; 1512 rows behind 23000, 192 items: 196 whole, 218 in three; one
//   row of 131072: 8 items in 19 parts);
// - whole prompts, whose items differ in length: the longest walk at 1.5 us a
//   tile, plus 4 us and a microsecond per MB of results (4096 tokens, 1 head of
//   128: 51 us whole, 34 in four parts; 6000, 2/1 heads of 64: 67 and 35; 2048,
//   8/2 of 128: 30 and, in two, 39).
// (A workspace's size must not depend on the device: 152 SMs.)
int tc_parts(const AttnDims& A) {
    const int64_t items = items_about(A), sms = 152, tiles = A.total_k / (kRows * (int64_t)A.n_seqs);
    if (tiles < 16 || items > sms) return 1;
    const bool few = 4 * A.total_q <= A.total_k;
    const int64_t most = few ? std::min<int64_t>(32, std::max<int64_t>(4, sms / items))
                             : std::min<int64_t>({4, sms / items, tiles / 8});
    int best = 1;
    double least = few ? 1.0 : 1.5 * tiles;
    for (int p = 2; p <= most; ++p) {
        const double cost = few ? (double)((items * p + sms - 1) / sms) / p + 0.55 * items / sms
                                : 1.5 * tiles / p + 4.0 + 4e-6 * A.total_q * A.Hq * A.d * p;
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}
size_t part_bytes(const AttnDims& A, int64_t parts) {
    const int64_t rows = A.total_q * A.Hq;
    return parts > 1 ? (size_t)((parts * rows + 3) / 4 * 4 + parts * rows * A.d) * sizeof(float) : 0;
}

template <int D>
cudaError_t launch(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                   const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out, float* lse, void* part_ws, size_t room,
                   int32_t* err, cudaStream_t st) {
    static DeviceCache cache;
    cudaError_t e = device_cached(cache, nullptr, [](int, int*) {
        return prepare_kernel(attention_tc_kernel<D>, Cfg<D>::kSmem);
    });
    if (e != cudaSuccess) return e;
    const int pack = pack_of(A.G), qb = kRows / pack;
    int lpack = 0;
    while ((1 << lpack) < pack) ++lpack;
    CUtensorMap mq, mk, mv;
    if (!tma::make_map_3d_strided(&mq, q, true, D, (uint64_t)A.Hq, (uint64_t)A.total_q, (uint64_t)A.sq * 2, 64,
                                  (uint32_t)pack, (uint32_t)qb) ||
        !tma::make_map_3d_strided(&mk, k, true, D, (uint64_t)A.Hkv, (uint64_t)A.total_k, (uint64_t)A.sk * 2, 64, 1,
                                  kRows) ||
        !tma::make_map_3d_strided(&mv, v, true, D, (uint64_t)A.Hkv, (uint64_t)A.total_k, (uint64_t)A.sv * 2, 64, 1,
                                  kRows))
        return cudaErrorInvalidValue;
    const int parts = parts_within(tc_parts(A), room, [&](int p) { return part_bytes(A, p); });
    const int64_t blocks = items_bound(A) * parts, rows = A.total_q * A.Hq;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    float* part_lse = static_cast<float*>(part_ws);
    float* part_o = part_lse + (parts * rows + 3) / 4 * 4;
    attention_tc_kernel<D><<<(unsigned)blocks, kBlock, Cfg<D>::kSmem, st>>>(A, mq, mk, mv, v, cu_q, cu_k, lpack, parts, out,
                                                                             lse, part_o, part_lse, err);
    if (parts > 1)
        attention_join_kernel<D, __nv_bfloat16><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(A, cu_q, parts, part_o, part_lse, out, lse);
    return cudaGetLastError();
}

}  // namespace

size_t attention_tc_part_bytes(const AttnDims& A) { return part_bytes(A, tc_parts(A)); }

cudaError_t launch_attention_tc(const AttnDims& A, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                const __nv_bfloat16* v, const int32_t* cu_q, const int32_t* cu_k, __nv_bfloat16* out,
                                float* lse, void* parts, size_t room, int32_t* err, cudaStream_t st) {
    return A.d == 128 ? launch<128>(A, q, k, v, cu_q, cu_k, out, lse, parts, room, err, st)
                      : launch<64>(A, q, k, v, cu_q, cu_k, out, lse, parts, room, err, st);
}

}  // namespace hla
