// Host side of the full softmax layers' entry points: argument checks,
// workspace layout, launches.  Declarations and contracts: include/hla.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attention_tc.cuh"

using namespace hla;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good(const void* p) { return p && aligned16(p); }
int status(cudaError_t e) { return e == cudaSuccess ? HLA_OK : HLA_ERR_CUDA; }
size_t type_bytes(int dtype) { return dtype == HLA_DTYPE_F32 ? 4 : dtype == HLA_DTYPE_BF16 ? 2 : 1; }
constexpr int kMaxHeads = 65535;  // a grid dimension

// ---- rotary positions -------------------------------------------------------

int check_rope(const hla_rope_params* p) {
    if (!p || p->n_q_heads < 0 || p->n_kv_heads < 0 || p->n_q_heads + (int64_t)p->n_kv_heads > kMaxHeads)
        return HLA_ERR_INVALID_ARG;
    if (p->head_dim < 2 || p->head_dim % 2 || p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > p->head_dim)
        return HLA_ERR_INVALID_ARG;
    if (p->head_dim > 2 * kMaxRopePairs) return HLA_ERR_UNSUPPORTED;
    if (p->layout != HLA_ROPE_HALF && p->layout != HLA_ROPE_INTERLEAVED) return HLA_ERR_INVALID_ARG;
    if (p->dtype != HLA_DTYPE_F32 && p->dtype != HLA_DTYPE_BF16) return HLA_ERR_UNSUPPORTED;
    if (!(p->base > 1.0) || !std::isfinite(p->base)) return HLA_ERR_INVALID_ARG;
    if (p->scaling < HLA_ROPE_SCALE_NONE || p->scaling > HLA_ROPE_SCALE_YARN) return HLA_ERR_INVALID_ARG;
    if (p->scaling != HLA_ROPE_SCALE_NONE && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
        return HLA_ERR_INVALID_ARG;
    if (p->scaling >= HLA_ROPE_SCALE_BANDS) {
        if (p->original_len < 1) return HLA_ERR_INVALID_ARG;
        const bool unset = p->low == 0.0 && p->high == 0.0;
        if (!unset && (!(p->low > 0.0) || !(p->high > p->low) || !std::isfinite(p->high))) return HLA_ERR_INVALID_ARG;
    }
    const int64_t q = (int64_t)p->n_q_heads * p->head_dim, k = (int64_t)p->n_kv_heads * p->head_dim;
    if ((p->q_stride != 0 && p->q_stride < q) || (p->k_stride != 0 && p->k_stride < k)) return HLA_ERR_INVALID_ARG;
    return HLA_OK;
}

double rope_frequencies(const hla_rope_params* p, double* w) {
    const double two_pi = 6.283185307179586476925286766559;
    const int r = p->rot_dim;
    const double f = p->factor, orig = (double)p->original_len;
    const bool unset = p->low == 0.0 && p->high == 0.0;
    const double low = unset ? 1.0 : p->low, high = unset ? (p->scaling == HLA_ROPE_SCALE_YARN ? 32.0 : 4.0) : p->high;
    auto index = [&](double turns) { return r * std::log(orig / (two_pi * turns)) / (2.0 * std::log(p->base)); };
    const double lo = std::max(0.0, std::floor(index(high))), hi = std::min(r - 1.0, std::ceil(index(low)));
    const double step = -2.0 * std::log2(p->base) / r;
    for (int i = 0; i < r / 2; ++i) {
        const double x = std::exp2(i * step);  // base^(-2 i / r)
        double keep = 1.0;  // share of the unscaled angle
        if (p->scaling == HLA_ROPE_SCALE_LINEAR) keep = 0.0;
        if (p->scaling == HLA_ROPE_SCALE_BANDS)
            keep = std::min(1.0, std::max(0.0, (orig * x / two_pi - low) / (high - low)));
        if (p->scaling == HLA_ROPE_SCALE_YARN)
            keep = 1.0 - std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
        w[i] = p->scaling == HLA_ROPE_SCALE_NONE ? x : x * keep + x / f * (1.0 - keep);
    }
    return p->scaling == HLA_ROPE_SCALE_YARN ? 0.1 * std::log(f) + 1.0 : 1.0;
}

int run_rope(const hla_rope_params* p, const void* q, const void* k, const int64_t* positions, int64_t total, void* qo,
             void* ko, int sign, void* stream) {
    const int rc = check_rope(p);
    if (rc) return rc;
    if (total < 0 || total > (int64_t)INT32_MAX || !q != !qo || !k != !ko) return HLA_ERR_INVALID_ARG;
    if (total == 0 || (!q && !k)) return HLA_OK;
    // elements and positions at their own alignment; wider accesses are chosen where everything allows them
    const uintptr_t a = type_bytes(p->dtype) - 1;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)qo | (uintptr_t)ko) & a) return HLA_ERR_INVALID_ARG;
    if (!positions || ((uintptr_t)positions & 7)) return HLA_ERR_INVALID_ARG;
    RopeDims R;
    std::memset(&R, 0, sizeof(R));
    R.Hq = q ? p->n_q_heads : 0;
    R.Hkv = k ? p->n_kv_heads : 0;
    R.d = p->head_dim;
    R.r = p->rot_dim;
    R.interleaved = p->layout == HLA_ROPE_INTERLEAVED;
    R.sign = sign;
    R.total = total;
    const int64_t dense_q = (int64_t)p->n_q_heads * R.d, dense_k = (int64_t)p->n_kv_heads * R.d;
    R.q_in = p->q_stride ? p->q_stride : dense_q;
    R.k_in = p->k_stride ? p->k_stride : dense_k;
    R.q_out = qo == q ? R.q_in : dense_q;
    R.k_out = ko == k ? R.k_in : dense_k;
    double w[kMaxRopePairs];
    R.gain = (float)rope_frequencies(p, w);
    for (int i = 0; i < R.r / 2; ++i) {
        const double turns = w[i] / 6.283185307179586476925286766559;  // < 1: base > 1, factor >= 1
        R.freq[i] = (uint64_t)std::ldexp(turns, 64);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->dtype == HLA_DTYPE_F32)
        return status(launch_rope(R, static_cast<const float*>(q), static_cast<const float*>(k), positions,
                                  static_cast<float*>(qo), static_cast<float*>(ko), st));
    return status(launch_rope(R, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), positions,
                              static_cast<__nv_bfloat16*>(qo), static_cast<__nv_bfloat16*>(ko), st));
}

// ---- attention --------------------------------------------------------------

int check_attn(const hla_attn_params* p) {
    if (!p || p->n_q_heads <= 0 || p->n_kv_heads <= 0 || p->n_q_heads % p->n_kv_heads || p->n_q_heads > kMaxHeads)
        return HLA_ERR_INVALID_ARG;
    if (p->reserved != 0 || !std::isfinite(p->scale) || p->scale < 0.0f) return HLA_ERR_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return HLA_ERR_UNSUPPORTED;
    if (p->dtype != HLA_DTYPE_F32 && p->dtype != HLA_DTYPE_BF16) return HLA_ERR_UNSUPPORTED;
    const int64_t per16 = 16 / (int64_t)type_bytes(p->dtype);
    const int64_t s[3] = {p->q_stride, p->k_stride, p->v_stride};
    for (int i = 0; i < 3; ++i) {
        const int64_t dense = (int64_t)(i ? p->n_kv_heads : p->n_q_heads) * p->head_dim;
        if (s[i] != 0 && (s[i] < dense || s[i] % per16 || s[i] > ((int64_t)1 << 38))) return HLA_ERR_INVALID_ARG;
    }
    return HLA_OK;
}

AttnDims attn_dims(const hla_attn_params* p, int n_seqs, int64_t total_q, int64_t total_k) {
    AttnDims A;
    std::memset(&A, 0, sizeof(A));
    A.Hq = p->n_q_heads;
    A.Hkv = p->n_kv_heads;
    A.d = p->head_dim;
    A.G = p->n_q_heads / p->n_kv_heads;
    A.n_seqs = n_seqs;
    A.total_q = total_q;
    A.total_k = total_k;
    A.sq = p->q_stride ? p->q_stride : (int64_t)A.Hq * A.d;
    A.sk = p->k_stride ? p->k_stride : (int64_t)A.Hkv * A.d;
    A.sv = p->v_stride ? p->v_stride : (int64_t)A.Hkv * A.d;
    A.scale = p->scale > 0.0f ? p->scale : (float)(1.0 / std::sqrt((double)A.d));
    return A;
}

constexpr size_t kWsHead = 256;  // the error word

// parts: with the results of as many parts as suit the sizes, else of one, which is the least that a call needs.
size_t attn_ws_bytes(const hla_attn_params* p, int64_t total_q, int64_t total_k, int n_seqs, bool backward, bool parts) {
    const AttnDims A = attn_dims(p, n_seqs, total_q, total_k);
    const bool f32 = p->dtype == HLA_DTYPE_F32;
    if (backward)
        return kWsHead + (f32 ? attention_backward_f32_floats(A, parts) * sizeof(float) : attention_backward_tc_bytes(A, parts));
    return kWsHead + (!parts ? 0 : f32 ? attention_f32_part_bytes(A) : attention_tc_part_bytes(A));
}

bool sizes_ok(int n_seqs, int64_t total_q, int64_t total_k) {
    return n_seqs >= 1 && total_q >= 0 && total_k >= 0 && total_q <= (int64_t)INT32_MAX &&
           total_k <= (int64_t)INT32_MAX;
}

// ---- cache ------------------------------------------------------------------

int check_cache(const hla_cache_params* p) {
    if (!p || p->n_kv_heads <= 0 || p->n_kv_heads > kMaxHeads || p->page_size <= 0 || p->n_pages < 0 ||
        p->max_pages < 0 || p->reserved != 0)
        return HLA_ERR_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return HLA_ERR_UNSUPPORTED;
    if (p->dtype != HLA_DTYPE_F32 && p->dtype != HLA_DTYPE_BF16) return HLA_ERR_UNSUPPORTED;
    if (p->cache_dtype != HLA_DTYPE_E4M3 && p->cache_dtype != p->dtype) return HLA_ERR_UNSUPPORTED;
    if (p->page_size % 16) return HLA_ERR_UNSUPPORTED;
    return HLA_OK;
}

int check_buffers(const hla_cache_params* p, const hla_cache* c) {
    if (!c || !good(c->err)) return HLA_ERR_INVALID_ARG;
    const bool pool = p->n_pages > 0, table = p->max_pages > 0;
    if (pool && (!good(c->k) || !good(c->v))) return HLA_ERR_INVALID_ARG;
    if (pool && p->cache_dtype == HLA_DTYPE_E4M3 && (!good(c->k_exp) || !good(c->v_exp))) return HLA_ERR_INVALID_ARG;
    if (table && !good(c->page_table)) return HLA_ERR_INVALID_ARG;
    return HLA_OK;
}

CacheDims cache_dims(const hla_cache_params* p, int n_seqs, int64_t total) {
    return CacheDims{p->n_kv_heads, p->head_dim, p->page_size, p->n_pages, p->max_pages, n_seqs, total};
}

int run_cache(const hla_cache_params* p, const hla_cache* c, void* k, void* v, const int32_t* cu,
              const int64_t* start, int n_seqs, int64_t total, bool read, void* stream) {
    int rc = check_cache(p);
    if (!rc) rc = check_buffers(p, c);
    if (rc) return rc;
    if (n_seqs < 1 || total < 0 || total > (int64_t)INT32_MAX) return HLA_ERR_INVALID_ARG;
    if (!good(cu) || !good(start) || (total > 0 && (!good(k) || !good(v)))) return HLA_ERR_INVALID_ARG;
    if (total == 0) return HLA_OK;
    const CacheDims C = cache_dims(p, n_seqs, total);
    const bool e4m3 = p->cache_dtype == HLA_DTYPE_E4M3;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto* kk, auto* vv) {
        return status(read ? launch_cache_read(C, e4m3, *c, kk, vv, cu, start, st)
                           : launch_cache_write(C, e4m3, *c, kk, vv, cu, start, st));
    };
    return p->dtype == HLA_DTYPE_F32 ? run(static_cast<float*>(k), static_cast<float*>(v))
                                     : run(static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
}

}  // namespace

extern "C" {

HLA_API int hla_rope_frequencies(const hla_rope_params* p, double* w, double* gain) {
    const int rc = check_rope(p);
    if (rc) return rc;
    if (!w || !gain) return HLA_ERR_INVALID_ARG;
    *gain = rope_frequencies(p, w);
    return HLA_OK;
}

HLA_API int hla_rope(const hla_rope_params* p, const void* q, const void* k, const int64_t* positions,
                     int64_t total_tokens, void* q_out, void* k_out, void* stream) {
    return run_rope(p, q, k, positions, total_tokens, q_out, k_out, 1, stream);
}

HLA_API int hla_rope_backward(const hla_rope_params* p, const void* dq_out, const void* dk_out,
                              const int64_t* positions, int64_t total_tokens, void* dq, void* dk, void* stream) {
    return run_rope(p, dq_out, dk_out, positions, total_tokens, dq, dk, -1, stream);
}

HLA_API int hla_attention_workspace_bytes(const hla_attn_params* p, int64_t total_q, int64_t total_k, int n_seqs,
                                          int backward, size_t* bytes) {
    const int rc = check_attn(p);
    if (rc) return rc;
    if (!sizes_ok(n_seqs, total_q, total_k) || !bytes) return HLA_ERR_INVALID_ARG;
    *bytes = attn_ws_bytes(p, total_q, total_k, n_seqs, backward != 0, true);
    return HLA_OK;
}

HLA_API int hla_attention(const hla_attn_params* p, const void* q, const void* k, const void* v,
                          const int32_t* cu_q, const int32_t* cu_k, int n_seqs, int64_t total_q, int64_t total_k,
                          void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const int rc = check_attn(p);
    if (rc) return rc;
    if (!sizes_ok(n_seqs, total_q, total_k) || !good(cu_q) || !good(ws)) return HLA_ERR_INVALID_ARG;
    if (cu_k ? !aligned16(cu_k) : total_k != total_q) return HLA_ERR_INVALID_ARG;
    if (total_q > 0 && (!good(q) || !good(out) || !good(lse))) return HLA_ERR_INVALID_ARG;
    if (total_k > 0 && (!good(k) || !good(v))) return HLA_ERR_INVALID_ARG;
    if (ws_bytes < attn_ws_bytes(p, total_q, total_k, n_seqs, false, false)) return HLA_ERR_WORKSPACE;
    if (total_q == 0) return HLA_OK;
    if (!cu_k) cu_k = cu_q;
    const AttnDims A = attn_dims(p, n_seqs, total_q, total_k);
    int32_t* err = static_cast<int32_t*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    const bool f32 = p->dtype == HLA_DTYPE_F32;
    if (total_k == 0)  // no row sees a key
        return status(f32 ? launch_attention_empty(total_q, total_k, n_seqs, cu_q, cu_k, A.Hq, A.d,
                                                   static_cast<float*>(out), static_cast<float*>(nullptr), lse, err, st)
                          : launch_attention_empty(total_q, total_k, n_seqs, cu_q, cu_k, A.Hq, A.d,
                                                   static_cast<bf*>(out), static_cast<bf*>(nullptr), lse, err, st));
    if (f32)
        return status(launch_attention_f32(A, static_cast<const float*>(q), static_cast<const float*>(k),
                                           static_cast<const float*>(v), cu_q, cu_k, static_cast<float*>(out), lse,
                                           reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHead), ws_bytes - kWsHead, err, st));
    return status(launch_attention_tc(A, static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v),
                                      cu_q, cu_k, static_cast<bf*>(out), lse, static_cast<char*>(ws) + kWsHead, ws_bytes - kWsHead, err,
                                      st));
}

HLA_API int hla_attention_backward(const hla_attn_params* p, const void* q, const void* k, const void* v,
                                   const void* out, const float* lse, const void* dout, const int32_t* cu_q,
                                   const int32_t* cu_k, int n_seqs, int64_t total_q, int64_t total_k, void* dq,
                                   void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    const int rc = check_attn(p);
    if (rc) return rc;
    if (!sizes_ok(n_seqs, total_q, total_k) || !good(cu_q) || !good(ws)) return HLA_ERR_INVALID_ARG;
    if (cu_k ? !aligned16(cu_k) : total_k != total_q) return HLA_ERR_INVALID_ARG;
    const void* rows[] = {q, out, lse, dout, dq};
    for (const void* x : rows)
        if (total_q > 0 && !good(x)) return HLA_ERR_INVALID_ARG;
    const void* keys[] = {k, v, dk, dv};
    for (const void* x : keys)
        if (total_k > 0 && !good(x)) return HLA_ERR_INVALID_ARG;
    if (ws_bytes < attn_ws_bytes(p, total_q, total_k, n_seqs, true, false)) return HLA_ERR_WORKSPACE;
    if (total_q == 0 && total_k == 0) return HLA_OK;
    if (!cu_k) cu_k = cu_q;
    const AttnDims A = attn_dims(p, n_seqs, total_q, total_k);
    int32_t* err = static_cast<int32_t*>(ws);
    void* rows_ws = static_cast<char*>(ws) + kWsHead;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    const bool f32 = p->dtype == HLA_DTYPE_F32;
    if (total_q == 0 || total_k == 0) {  // no row sees a key: every gradient is zero
        auto zero = [&](auto* rq, auto* rk, auto* rv) {
            cudaError_t e = launch_attention_empty(total_q, total_k, n_seqs, cu_q, cu_k, A.Hq, A.d, rq,
                                                   decltype(rq)(nullptr), nullptr, err, st);
            if (e == cudaSuccess)
                e = launch_attention_empty(total_k, total_q, n_seqs, cu_k, cu_q, A.Hkv, A.d, rk, rv, nullptr, err, st);
            return status(e);
        };
        return f32 ? zero(static_cast<float*>(dq), static_cast<float*>(dk), static_cast<float*>(dv))
                   : zero(static_cast<bf*>(dq), static_cast<bf*>(dk), static_cast<bf*>(dv));
    }
    if (f32)
        return status(launch_attention_backward_f32(
            A, static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v),
            static_cast<const float*>(out), lse, static_cast<const float*>(dout), cu_q, cu_k, static_cast<float*>(dq),
            static_cast<float*>(dk), static_cast<float*>(dv), static_cast<float*>(rows_ws), ws_bytes - kWsHead, err, st));
    return status(launch_attention_backward_tc(
        A, static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v), static_cast<const bf*>(out),
        lse, static_cast<const bf*>(dout), cu_q, cu_k, static_cast<bf*>(dq), static_cast<bf*>(dk), static_cast<bf*>(dv),
        rows_ws, ws_bytes - kWsHead, err, st));
}

HLA_API int hla_cache_bytes(const hla_cache_params* p, size_t* rows, size_t* exponents) {
    const int rc = check_cache(p);
    if (rc) return rc;
    if (!rows || !exponents) return HLA_ERR_INVALID_ARG;
    const size_t n = (size_t)p->n_pages * p->n_kv_heads * p->page_size;
    *rows = n * p->head_dim * type_bytes(p->cache_dtype);
    *exponents = p->cache_dtype == HLA_DTYPE_E4M3 ? n : 0;
    return HLA_OK;
}

HLA_API int hla_cache_write(const hla_cache_params* p, const hla_cache* cache, const void* k, const void* v,
                            const int32_t* cu_seqlens, const int64_t* start, int n_seqs, int64_t total_tokens,
                            void* stream) {
    return run_cache(p, cache, const_cast<void*>(k), const_cast<void*>(v), cu_seqlens, start, n_seqs, total_tokens,
                     false, stream);
}

HLA_API int hla_cache_read(const hla_cache_params* p, const hla_cache* cache, const int32_t* cu_seqlens,
                           const int64_t* start, int n_seqs, int64_t total_tokens, void* k, void* v, void* stream) {
    return run_cache(p, cache, k, v, cu_seqlens, start, n_seqs, total_tokens, true, stream);
}

HLA_API int hla_attention_decode_workspace_bytes(const hla_attn_params* p, const hla_cache_params* cp, size_t* bytes) {
    int rc = check_attn(p);
    if (!rc) rc = check_cache(cp);
    if (rc) return rc;
    if (!bytes || p->n_kv_heads != cp->n_kv_heads || p->head_dim != cp->head_dim || p->dtype != cp->dtype)
        return HLA_ERR_INVALID_ARG;
    *bytes = attention_decode_ws_bytes(p->n_q_heads, p->n_kv_heads, p->head_dim);
    return HLA_OK;
}

HLA_API int hla_attention_decode(const hla_attn_params* p, const hla_cache_params* cp, const hla_cache* cache,
                                 const void* q, const int64_t* lens, int n_seqs, void* out, void* ws, size_t ws_bytes,
                                 void* stream) {
    size_t need = 0;
    int rc = hla_attention_decode_workspace_bytes(p, cp, &need);
    if (!rc) rc = check_buffers(cp, cache);
    if (rc) return rc;
    if (n_seqs < 0) return HLA_ERR_INVALID_ARG;
    if ((uint64_t)cp->n_pages * cp->n_kv_heads * cp->page_size > 0xfffffffeull) return HLA_ERR_UNSUPPORTED;  // rows
    if (n_seqs == 0) return HLA_OK;
    if (!good(q) || !good(lens) || !good(out) || !good(ws)) return HLA_ERR_INVALID_ARG;
    if (ws_bytes < need) return HLA_ERR_WORKSPACE;
    const AttnDims A = attn_dims(p, n_seqs, n_seqs, 0);
    const CacheDims C = cache_dims(cp, n_seqs, n_seqs);
    const bool e4m3 = cp->cache_dtype == HLA_DTYPE_E4M3;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto t) {
        using T = decltype(t);
        return status(launch_attention_decode(A, C, e4m3, *cache, static_cast<const T*>(q), lens, static_cast<T*>(out),
                                              static_cast<float*>(ws), st));
    };
    return p->dtype == HLA_DTYPE_F32 ? run(float()) : run(__nv_bfloat16());
}

HLA_API int hla_check_cache_error(const hla_cache* cache, void* stream, int32_t* code) {
    if (!cache || !good(cache->err)) return HLA_ERR_INVALID_ARG;
    return hla_check_workspace_error(cache->err, stream, code);
}

}  // extern "C"
