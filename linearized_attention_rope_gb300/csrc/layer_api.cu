// Host side of the norms, the gated recurrence and the 4-bit products: argument
// checks, workspace layout, launches.  Contracts: include/hla.h.
#include <cmath>
#include <type_traits>

#include "layer.cuh"

using namespace hla;

namespace {

using bf = __nv_bfloat16;
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good(const void* p) { return p && aligned16(p); }
int status(cudaError_t e) { return e == cudaSuccess ? HLA_OK : HLA_ERR_CUDA; }
bool is_type(int t) { return t == HLA_DTYPE_F32 || t == HLA_DTYPE_BF16; }
size_t type_bytes(int t) { return t == HLA_DTYPE_F32 ? 4 : t == HLA_DTYPE_BF16 ? 2 : 1; }
// elements at their own alignment; wider accesses are chosen where everything allows them
bool own(const void* p, int t) { return p && (reinterpret_cast<uintptr_t>(p) & (type_bytes(t) - 1)) == 0; }
constexpr int64_t kMaxStride = (int64_t)1 << 38;
bool stride_ok(int64_t s, int64_t dense) { return s == 0 || (s >= dense && s <= kMaxStride); }
constexpr size_t kWsHead = 256;  // the error word

template <class F> int by_type(int t, F f) { return t == HLA_DTYPE_F32 ? f(float()) : f(bf()); }

int check_norm(const hla_norm_params* p) {
    if (!p || p->n_cols < 1 || p->n_heads < 1 || p->reserved != 0) return HLA_ERR_INVALID_ARG;
    if (!std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->offset)) return HLA_ERR_INVALID_ARG;
    if (p->n_cols > 1 << 20 || p->n_heads > 65535) return HLA_ERR_UNSUPPORTED;
    if (!is_type(p->dtype)) return HLA_ERR_UNSUPPORTED;
    if (p->out_dtype != p->dtype && p->out_dtype != HLA_DTYPE_E4M3) return HLA_ERR_UNSUPPORTED;
    const int64_t dense = (int64_t)p->n_heads * p->n_cols;
    if (!stride_ok(p->x_stride, dense) || !stride_ok(p->residual_stride, dense)) return HLA_ERR_INVALID_ARG;
    if (p->out_dtype == HLA_DTYPE_E4M3) {
        if (p->group != 0 && p->group != 32 && p->group != 128) return HLA_ERR_UNSUPPORTED;
        if (p->n_cols % (p->group ? p->group : 16)) return HLA_ERR_INVALID_ARG;
        if ((p->x_stride | p->residual_stride) * (int64_t)type_bytes(p->dtype) % 16) return HLA_ERR_INVALID_ARG;
    } else if (p->group != 0) {
        return HLA_ERR_INVALID_ARG;
    }
    return HLA_OK;
}

NormDims norm_dims(const hla_norm_params* p, int64_t tokens) {
    NormDims N;
    const int64_t dense = (int64_t)p->n_heads * p->n_cols;
    N.rows = tokens * p->n_heads;
    N.sx = p->x_stride ? p->x_stride : dense;
    N.sr = p->residual_stride ? p->residual_stride : dense;
    N.cols = p->n_cols;
    N.heads = p->n_heads;
    N.group = p->group;
    N.eps = p->eps;
    N.offset = p->offset;
    if (N.sx == dense && N.sr == dense) {  // heads of dense tokens are rows like any other
        N.heads = 1;
        N.sx = N.sr = N.cols;
    }
    return N;
}
bool rows_ok(const hla_norm_params* p, int64_t tokens) {
    return tokens >= 0 && tokens <= INT32_MAX && tokens * p->n_heads <= INT32_MAX;
}

int check_recurrence(const hla_recurrence_params* p) {
    if (!p || p->n_channels < 1 || p->gate_dim < 1 || p->n_channels % p->gate_dim) return HLA_ERR_INVALID_ARG;
    if (p->gate_dim != 1 && p->gate_dim != 64 && p->gate_dim != 128) return HLA_ERR_UNSUPPORTED;
    if (p->n_channels > 1 << 20) return HLA_ERR_UNSUPPORTED;
    if (!is_type(p->dtype) || !is_type(p->gate_dtype)) return HLA_ERR_UNSUPPORTED;
    if (!stride_ok(p->x_stride, p->n_channels) || !stride_ok(p->g_stride, p->n_channels / p->gate_dim))
        return HLA_ERR_INVALID_ARG;
    return p->x_stride > UINT32_MAX || p->g_stride > UINT32_MAX ? HLA_ERR_UNSUPPORTED : HLA_OK;
}

RecDims rec_dims(const hla_recurrence_params* p, int n_seqs, int64_t total) {
    RecDims R;
    R.total = total;
    R.sx = p->x_stride ? p->x_stride : p->n_channels;
    R.sg = p->g_stride ? p->g_stride : p->n_channels / p->gate_dim;
    R.channels = p->n_channels;
    R.gate_dim = p->gate_dim;
    R.n_seqs = n_seqs;
    return R;
}
// Tiles are counted in 32 bits: at most (total / 64 + 1) (channels / 64 + 1) of them.
bool tokens_ok(const hla_recurrence_params* p, int64_t total) {
    return total >= 0 && total <= INT32_MAX && (total / 64 + 1) * ((int64_t)p->n_channels / 64 + 1) <= INT32_MAX;
}

int check_linear4(const hla_linear4_params* p) {
    if (!p || p->n_in < 1 || p->n_out < 1) return HLA_ERR_INVALID_ARG;
    if (p->group != 32 && p->group != 64 && p->group != 128) return HLA_ERR_UNSUPPORTED;
    if (p->n_in % p->group) return HLA_ERR_INVALID_ARG;
    if (p->n_in > 1 << 24 || p->n_out > 1 << 24) return HLA_ERR_UNSUPPORTED;
    if (!is_type(p->dtype) || (p->x_dtype != p->dtype && p->x_dtype != HLA_DTYPE_E4M3)) return HLA_ERR_UNSUPPORTED;
    if (p->x_dtype == HLA_DTYPE_E4M3) {
        if (p->x_group != 0 && p->x_group != 32 && p->x_group != 128) return HLA_ERR_UNSUPPORTED;
        if (p->x_group && p->n_in % p->x_group) return HLA_ERR_INVALID_ARG;
    } else if (p->x_group != 0) {
        return HLA_ERR_INVALID_ARG;
    }
    return stride_ok(p->x_stride, p->n_in) ? HLA_OK : HLA_ERR_INVALID_ARG;
}
// 64 tokens a block row, 65535 of those
bool linear4_tokens_ok(int64_t tokens) { return tokens >= 0 && tokens <= 64 * 65535; }

Rows4 rows_kind(const hla_linear4_params* p) {
    return p->x_dtype == HLA_DTYPE_F32 ? Rows4::kF32 : p->x_dtype == HLA_DTYPE_BF16 ? Rows4::kBf16 : Rows4::kE4m3;
}
Linear4Dims linear4_dims(const hla_linear4_params* p, int64_t tokens) {
    return {tokens, p->x_stride ? p->x_stride : p->n_in, p->n_in, p->n_out, p->group, p->x_group};
}

}  // namespace

extern "C" {

HLA_API int hla_rms_norm(const hla_norm_params* p, const void* x, const void* residual, const void* weight,
                         int64_t tokens, void* out, uint8_t* exp, void* sum, void* stream) {
    const int rc = check_norm(p);
    if (rc) return rc;
    const bool eight = p->out_dtype == HLA_DTYPE_E4M3;
    if (!rows_ok(p, tokens) || (residual && !sum && tokens > 0) || (eight ? !exp && tokens > 0 : exp != nullptr))
        return HLA_ERR_INVALID_ARG;
    if (tokens == 0) return HLA_OK;
    const void* ins[] = {x, residual, weight, sum};
    for (const void* y : ins)
        if (y ? (eight ? !aligned16(y) : !own(y, p->dtype)) : y == x) return HLA_ERR_INVALID_ARG;
    if (!x || (eight ? !good(out) : !own(out, p->dtype))) return HLA_ERR_INVALID_ARG;
    const NormDims N = norm_dims(p, tokens);
    return by_type(p->dtype, [&](auto t) {
        using T = decltype(t);
        return status(launch_norm<T>(N, static_cast<const T*>(x), static_cast<const T*>(residual),
                                     static_cast<const T*>(weight), eight ? nullptr : static_cast<T*>(out),
                                     eight ? static_cast<uint8_t*>(out) : nullptr, exp, static_cast<T*>(sum),
                                     static_cast<cudaStream_t>(stream)));
    });
}

HLA_API int hla_rms_norm_backward_workspace_bytes(const hla_norm_params* p, size_t* bytes) {
    const int rc = check_norm(p);
    if (rc) return rc;
    if (!bytes) return HLA_ERR_INVALID_ARG;
    *bytes = (size_t)norm_parts(p->n_cols) * p->n_cols * sizeof(float);
    return HLA_OK;
}

HLA_API int hla_rms_norm_backward(const hla_norm_params* p, const void* s, const void* weight, const void* dout,
                                  const void* dsum, int64_t tokens, void* dx, float* dweight, void* ws, size_t ws_bytes,
                                  void* stream) {
    size_t need = 0;
    const int rc = hla_rms_norm_backward_workspace_bytes(p, &need);
    if (rc) return rc;
    if (!rows_ok(p, tokens) || (dweight && (!own(dweight, HLA_DTYPE_F32) || !good(ws)))) return HLA_ERR_INVALID_ARG;
    if (dweight && tokens > 0 && !weight) return HLA_ERR_INVALID_ARG;
    if (tokens > 0 && (!own(s, p->dtype) || !own(dout, p->dtype) || !own(dx, p->dtype) ||
                       (weight && !own(weight, p->dtype)) || (dsum && !own(dsum, p->dtype))))
        return HLA_ERR_INVALID_ARG;
    if (dweight && ws_bytes < need) return HLA_ERR_WORKSPACE;
    if (tokens == 0 && !dweight) return HLA_OK;
    NormDims N = norm_dims(p, tokens);
    N.sr = N.sx;
    return by_type(p->dtype, [&](auto t) {
        using T = decltype(t);
        return status(launch_norm_backward<T>(N, static_cast<const T*>(s), static_cast<const T*>(weight),
                                              static_cast<const T*>(dout), static_cast<const T*>(dsum),
                                              static_cast<T*>(dx), dweight, static_cast<float*>(ws),
                                              static_cast<cudaStream_t>(stream)));
    });
}

HLA_API int hla_recurrence_workspace_bytes(const hla_recurrence_params* p, int64_t total, size_t* bytes) {
    const int rc = check_recurrence(p);
    if (rc) return rc;
    if (!tokens_ok(p, total) || !bytes) return HLA_ERR_INVALID_ARG;
    *bytes = kWsHead + recurrence_carry_bytes(rec_dims(p, 1, total), p->dtype == HLA_DTYPE_F32);
    return HLA_OK;
}

HLA_API int hla_recurrence(const hla_recurrence_params* p, const void* g, const void* x, const float* h0,
                           const int32_t* cu, int n_seqs, int64_t total, void* out, float* h_last, float* states,
                           void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    const int rc = hla_recurrence_workspace_bytes(p, total, &need);
    if (rc) return rc;
    if (n_seqs < 1 || !own(cu, HLA_DTYPE_F32) || !good(ws)) return HLA_ERR_INVALID_ARG;
    if (total > 0 && (!own(g, p->gate_dtype) || !own(x, p->dtype) || !own(out, p->dtype))) return HLA_ERR_INVALID_ARG;
    if ((h0 && !aligned16(h0)) || (h_last && !aligned16(h_last)) || (states && !aligned16(states)))
        return HLA_ERR_INVALID_ARG;
    if (ws_bytes < need) return HLA_ERR_WORKSPACE;
    const RecDims R = rec_dims(p, n_seqs, total);
    return by_type(p->dtype, [&](auto t) {
        return by_type(p->gate_dtype, [&](auto u) {
            using T = decltype(t);
            using G = decltype(u);
            return status(launch_recurrence<T, G>(R, static_cast<const G*>(g), static_cast<const T*>(x), h0, cu,
                                                  static_cast<T*>(out), h_last, states, static_cast<char*>(ws) + kWsHead,
                                                  static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
        });
    });
}

HLA_API int hla_recurrence_backward(const hla_recurrence_params* p, const void* g, const void* x, const float* h0,
                                    const float* states, const int32_t* cu, int n_seqs, int64_t total, const void* dout,
                                    const float* dh_last, void* dg, void* dx, float* dh0, void* ws, size_t ws_bytes,
                                    void* stream) {
    size_t need = 0;
    const int rc = hla_recurrence_workspace_bytes(p, total, &need);
    if (rc) return rc;
    if (n_seqs < 1 || !own(cu, HLA_DTYPE_F32) || !good(ws)) return HLA_ERR_INVALID_ARG;
    if (total > 0 && (!own(g, p->gate_dtype) || !own(x, p->dtype) || !own(dout, p->dtype) || !own(dg, p->gate_dtype) ||
                      !own(dx, p->dtype) || !good(states)))
        return HLA_ERR_INVALID_ARG;
    if ((h0 && !aligned16(h0)) || (dh_last && !aligned16(dh_last)) || (dh0 && !aligned16(dh0))) return HLA_ERR_INVALID_ARG;
    if (ws_bytes < need) return HLA_ERR_WORKSPACE;
    const RecDims R = rec_dims(p, n_seqs, total);
    return by_type(p->dtype, [&](auto t) {
        return by_type(p->gate_dtype, [&](auto u) {
            using T = decltype(t);
            using G = decltype(u);
            return status(launch_recurrence_backward<T, G>(
                R, static_cast<const G*>(g), static_cast<const T*>(x), h0, states, cu, static_cast<const T*>(dout), dh_last,
                static_cast<G*>(dg), static_cast<T*>(dx), dh0, static_cast<char*>(ws) + kWsHead,
                static_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
        });
    });
}

HLA_API int hla_recurrence_step(const hla_recurrence_params* p, const void* g, const void* x, float* h, int n_seqs,
                                void* out, void* stream) {
    const int rc = check_recurrence(p);
    if (rc) return rc;
    // a thread takes four channels, or one: 32 bits of blocks
    if (n_seqs < 0 || (int64_t)n_seqs * p->n_channels / 256 >= INT32_MAX) return HLA_ERR_INVALID_ARG;
    if (n_seqs == 0) return HLA_OK;
    if (!own(g, p->gate_dtype) || !own(x, p->dtype) || !own(out, p->dtype) || !own(h, HLA_DTYPE_F32))
        return HLA_ERR_INVALID_ARG;
    const RecDims R = rec_dims(p, n_seqs, n_seqs);
    return by_type(p->dtype, [&](auto t) {
        return by_type(p->gate_dtype, [&](auto u) {
            using T = decltype(t);
            using G = decltype(u);
            return status(launch_recurrence_step<T, G>(R, static_cast<const G*>(g), static_cast<const T*>(x), h,
                                                       static_cast<T*>(out), static_cast<cudaStream_t>(stream)));
        });
    });
}

HLA_API int hla_linear4_workspace_bytes(const hla_linear4_params* p, int64_t tokens, size_t* bytes) {
    const int rc = check_linear4(p);
    if (rc) return rc;
    if (!linear4_tokens_ok(tokens) || !bytes) return HLA_ERR_INVALID_ARG;
    *bytes = (size_t)linear4_parts(rows_kind(p)) * tokens * p->n_in * 2;
    return HLA_OK;
}

HLA_API int hla_linear4(const hla_linear4_params* p, const void* x, const uint8_t* x_exp, const uint8_t* w,
                        const void* scales, const void* offsets, int64_t tokens, void* out, void* ws, size_t ws_bytes,
                        void* stream) {
    size_t need = 0;
    const int rc = hla_linear4_workspace_bytes(p, tokens, &need);
    if (rc) return rc;
    const bool eight = p->x_dtype == HLA_DTYPE_E4M3;
    if (tokens > 0 && (!own(x, p->x_dtype) || !good(w) || !own(scales, p->dtype) || (offsets && !own(offsets, p->dtype)) ||
                       !own(out, p->dtype) || (eight ? !x_exp : x_exp != nullptr)))
        return HLA_ERR_INVALID_ARG;
    if (tokens == 0) return HLA_OK;
    const bool parts = p->x_dtype != HLA_DTYPE_BF16 || !aligned16(x) || p->x_stride % 8;
    if (parts && !good(ws)) return HLA_ERR_INVALID_ARG;
    if (parts && ws_bytes < need) return HLA_ERR_WORKSPACE;
    const Linear4Dims L = linear4_dims(p, tokens);
    return by_type(p->dtype, [&](auto t) {
        using T = decltype(t);
        return status(launch_linear4<T>(L, rows_kind(p), x, x_exp, w, static_cast<const T*>(scales),
                                        static_cast<const T*>(offsets), static_cast<T*>(out),
                                        static_cast<bf*>(ws), static_cast<cudaStream_t>(stream)));
    });
}

HLA_API int hla_linear4_quantize(const hla_linear4_params* p, const void* weight, uint8_t* w, void* scales, void* offsets,
                                 void* stream) {
    const int rc = check_linear4(p);
    if (rc) return rc;
    if (!own(weight, p->dtype) || !good(w) || !own(scales, p->dtype) || (offsets && !own(offsets, p->dtype)))
        return HLA_ERR_INVALID_ARG;
    // a warp per group, eight a block: 32 bits of blocks
    if ((int64_t)p->n_out * (p->n_in / p->group) / 8 >= INT32_MAX) return HLA_ERR_UNSUPPORTED;
    const Linear4Dims L = linear4_dims(p, 0);
    return by_type(p->dtype, [&](auto t) {
        using T = decltype(t);
        return status(launch_linear4_quantize<T>(L, static_cast<const T*>(weight), w, static_cast<T*>(scales),
                                                 static_cast<T*>(offsets), static_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
