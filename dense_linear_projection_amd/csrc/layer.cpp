// layer.cpp -- C ABI of a decoding layer's operators in 8-bit integers, the
// normed append and attention over a shared prefix (declared in
// include/proj.h): argument checks, then the launchers (int8.hip, kvcache.hip,
// prefix.hip). None of them allocates, synchronises or tunes.
#include <hip/hip_runtime.h>

#include <climits>
#include <utility>

#include "checks.hpp"
#include "layer.hpp"

using namespace proj;

namespace {

constexpr int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }

// What the two products share: N, the weights' row length, the epilogue and the output side.
proj_status check_int(proj_ctx *ctx, const int8_t *W, const float *w_scales, const void *bias, int epilogue, int64_t M,
                      int64_t N, int64_t K, const void *Y, int out_dtype) {
    if (M < 0 || N < 0 || K < 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                             (long long)K);
    if (K > kIntMaxK)
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "K=%lld: sums of more than %lld products may pass 32 bits",
                             (long long)K, (long long)kIntMaxK);
    if (epilogue < PROJ_EPI_NONE || epilogue > PROJ_EPI_BIAS_GELU_TANH)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
    if (!known_dtype(out_dtype)) return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown output dtype %d", out_dtype);
    if (M == 0 || N == 0) return PROJ_OK;
    if (M > kMost / N || (K > 0 && (M > kMost / K || N > kMost / K)))
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "M*N, M*K or N*K too large");
    if (!Y || (K > 0 && (!W || !w_scales)) || ((epilogue & 1) && !bias))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "W, w_scales, Y or the epilogue's bias is NULL");
    const uintptr_t ya = out_dtype == PROJ_OUT_F32 ? 4 : 2;
    if (!aligned(W, 16) || !aligned(w_scales, 4) || !aligned(bias, 2) || !aligned(Y, ya))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "W not 16-byte aligned, or another not to its type");
    const uint64_t yb = static_cast<uint64_t>(M) * N * ya;
    if (overlap(Y, yb, W, static_cast<uint64_t>(N) * padded(K)) || overlap(Y, yb, w_scales, static_cast<uint64_t>(N) * 4) ||
        ((epilogue & 1) && overlap(Y, yb, bias, static_cast<uint64_t>(N) * 2)))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "Y overlaps an input");
    return PROJ_OK;
}

// bf16 rows: their stride and address.
proj_status check_rows(proj_ctx *ctx, const void *X, int64_t x_stride, int64_t M, int64_t K) {
    if (M < 0 || K < 0 || x_stride < K)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "M=%lld K=%lld, rows %lld apart", (long long)M, (long long)K,
                             (long long)x_stride);
    if (M > 0 && x_stride > kMost / M) return context_error(ctx, PROJ_ERR_UNSUPPORTED, "X too large");
    if ((M > 0 && K > 0 && !X) || !aligned(X, 2))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "X is NULL or not aligned to its type");
    return PROJ_OK;
}

uint64_t rows_bytes(int64_t M, int64_t K, int64_t stride) {
    return M > 0 ? (static_cast<uint64_t>(M - 1) * stride + K) * 2 : 0;
}

}  // namespace

extern "C" {

proj_status proj_quantize_rows(proj_ctx *ctx, const void *X, int64_t x_stride, int64_t M, int64_t K, int8_t *q,
                               int64_t q_stride, float *scales, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    s = check_rows(ctx, X, x_stride, M, K);
    if (s != PROJ_OK) return s;
    if (q_stride < K || q_stride % 16 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "rows of q %lld apart (a multiple of 16, at least %lld)",
                             (long long)q_stride, (long long)K);
    if (M == 0) return PROJ_OK;
    if (q_stride > kMost / M) return context_error(ctx, PROJ_ERR_UNSUPPORTED, "q too large");
    if ((q_stride > 0 && !q) || !scales || !aligned(q, 16) || !aligned(scales, 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q or scales is NULL, q not 16-byte or scales not 4-byte aligned");
    const uint64_t xb = rows_bytes(M, K, x_stride), qb = static_cast<uint64_t>(M) * q_stride, sb = static_cast<uint64_t>(M) * 4;
    if (overlap(X, xb, q, qb) || overlap(X, xb, scales, sb) || overlap(q, qb, scales, sb))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "operands overlap");
    DeviceGuard g(v.device);
    return finish(ctx, launch_quantize_rows(RowsArgs{static_cast<const uint16_t *>(X), x_stride, M, K, q, q_stride, scales},
                                            static_cast<hipStream_t>(stream)));
}

proj_status proj_run_int(proj_ctx *ctx, const int8_t *X, const float *x_scales, const int8_t *W, const float *w_scales,
                         const void *bias, int epilogue, int64_t M, int64_t N, int64_t K, void *Y, int out_dtype,
                         void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    if (K % 16 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "K=%lld (a multiple of 16: pad both operands with zeros)", (long long)K);
    s = check_int(ctx, W, w_scales, bias, epilogue, M, N, K, Y, out_dtype);
    if (s != PROJ_OK || M == 0 || N == 0) return s;
    if ((K > 0 && (!X || !x_scales)) || !aligned(X, 16) || !aligned(x_scales, 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "X or x_scales is NULL, or X not 16-byte aligned");
    const uint64_t yb = static_cast<uint64_t>(M) * N * (out_dtype == PROJ_OUT_F32 ? 4 : 2);
    if (overlap(Y, yb, X, static_cast<uint64_t>(M) * K) || overlap(Y, yb, x_scales, static_cast<uint64_t>(M) * 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "Y overlaps an input");
    DeviceGuard g(v.device);
    return finish(ctx, launch_int(IntArgs{X, W, x_scales, w_scales, static_cast<const uint16_t *>(bias), Y, M, N, K, N, epilogue,
                                          out_dtype, reinterpret_cast<int32_t *>(v.ws), v.ws_bytes, v.cus, v.counters, v.ncounters},
                                  static_cast<hipStream_t>(stream)));
}

proj_status proj_run_int_dynamic(proj_ctx *ctx, const void *X, int64_t x_stride, const int8_t *W, const float *w_scales,
                                 const void *bias, int epilogue, int64_t M, int64_t N, int64_t K, void *Y, int out_dtype,
                                 void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    s = check_rows(ctx, X, x_stride, M, K);
    if (s != PROJ_OK) return s;
    s = check_int(ctx, W, w_scales, bias, epilogue, M, N, K, Y, out_dtype);
    if (s != PROJ_OK || M == 0 || N == 0) return s;
    const int64_t ysize = out_dtype == PROJ_OUT_F32 ? 4 : 2, k = padded(K);
    if (overlap(Y, static_cast<uint64_t>(M) * N * ysize, X, rows_bytes(M, K, x_stride)))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "Y overlaps an input");
    // The tokens' integers and scales lie in the workspace, as many rows at a time as it holds
    // (less what aligning the two takes); what is left of it is the product's.
    const int64_t room = static_cast<int64_t>(v.ws_bytes) - 512;
    int64_t rows = room < 0 ? 0 : room / (k + 4);
    if (rows < 1)
        return context_error(ctx, PROJ_ERR_NO_MEMORY, "a row of K=%lld needs %lld bytes of workspace, the context has %lld",
                             (long long)K, (long long)(k + 4 + 512), (long long)v.ws_bytes);
    if (rows > M) rows = M;
    DeviceGuard g(v.device);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (int_fuses(M, N, k)) {
        IntArgs a{nullptr, W, nullptr, w_scales, static_cast<const uint16_t *>(bias), Y, M, N, k, N, epilogue,
                  out_dtype, reinterpret_cast<int32_t *>(v.ws), v.ws_bytes, v.cus, v.counters, v.ncounters};
        a.rows = static_cast<const uint16_t *>(X);
        a.rows_stride = x_stride;
        a.rows_k = K;
        return finish(ctx, launch_int_fused(a, st));
    }
    float *scales = v.ws;
    const int64_t sb = (rows * 4 + 255) / 256 * 256, qb = (rows * k + 255) / 256 * 256;
    int8_t *q = reinterpret_cast<int8_t *>(v.ws) + sb;
    int32_t *rest = reinterpret_cast<int32_t *>(q + qb);
    const size_t rest_bytes = v.ws_bytes - static_cast<size_t>(sb + qb);
    for (int64_t m = 0; m < M; m += rows) {
        const int64_t r = M - m < rows ? M - m : rows;
        hipError_t e = launch_quantize_rows(RowsArgs{static_cast<const uint16_t *>(X) + m * x_stride, x_stride, r, K, q, k, scales}, st);
        if (e == hipSuccess)
            e = launch_int(IntArgs{q, W, scales, w_scales, static_cast<const uint16_t *>(bias),
                                   static_cast<char *>(Y) + m * N * ysize, r, N, k, N, epilogue, out_dtype, rest, rest_bytes, v.cus,
                                   v.counters, v.ncounters},
                           st);
        if (e != hipSuccess) return finish(ctx, e);
    }
    return PROJ_OK;
}

proj_status proj_kv_append_norm(proj_ctx *ctx, const proj_kv_cache *cache, const void *qkv, int64_t qkv_stride, int64_t T,
                                int q_heads, const void *q_norm, const void *k_norm, int norm_dtype, int norm_per_head,
                                float eps, const float *rope, int64_t rope_rows, int rot, int interleaved,
                                const int32_t *positions, const int64_t *slots, void *q_out, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    AppendArgs a;
    s = check_append(ctx, cache, qkv, qkv_stride, T, q_heads, rope, rope_rows, rot, interleaved, positions, slots, q_out, &a);
    if (s != PROJ_OK) return s;
    if (!known_dtype(norm_dtype)) return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown norm dtype %d", norm_dtype);
    if (!(eps >= 0.f) || eps > 3e38f) return context_error(ctx, PROJ_ERR_INVALID_ARG, "eps %g (not negative, finite)", (double)eps);
    if (!aligned(q_norm, 16) || !aligned(k_norm, 16))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q_norm or k_norm not 16-byte aligned");
    if (T == 0) return PROJ_OK;
    const uint64_t row = static_cast<uint64_t>(cache->head_dim) * (norm_dtype == PROJ_OUT_F32 ? 4 : 2);
    const uint64_t qb = static_cast<uint64_t>(T) * q_heads * cache->head_dim * 2;
    for (const auto &in : {std::make_pair(q_norm, row * (norm_per_head ? static_cast<uint64_t>(q_heads) : 1)),
                           std::make_pair(k_norm, row * (norm_per_head ? static_cast<uint64_t>(cache->heads) : 1))})
        if (overlap(q_out, qb, in.first, in.second) || meets_cache(cache, in.first, in.second))
            return context_error(ctx, PROJ_ERR_INVALID_ARG, "q_out or the cache overlaps a norm's weights");
    DeviceGuard g(v.device);
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.norm_f32 = norm_dtype == PROJ_OUT_F32;
    a.norm_per_head = norm_per_head != 0;
    a.eps = eps;
    return finish(ctx, launch_append(a, static_cast<hipStream_t>(stream)));
}

proj_status proj_kv_attend_shared(proj_ctx *ctx, const proj_kv_cache *cache, const void *q, int64_t q_stride, int64_t B,
                                  int q_heads, const int32_t *prefix, int64_t prefix_len, const int32_t *tables,
                                  int64_t table_stride, int64_t table_width, const int32_t *lengths, int64_t max_len,
                                  int64_t window, float scale, void *out, int out_dtype, float *lse, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    PrefixArgs p;
    // the kernel counts the tokens of a part, which may be all of them, in 32 bits, up to a whole step
    if (prefix_len < 0 || prefix_len > INT32_MAX - 127 || (prefix_len > 0 && B > 0 && !prefix) || !aligned(prefix, 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "prefix of %lld tokens, or its pages NULL or not aligned",
                             (long long)prefix_len);
    s = check_attend(ctx, cache, q, q_stride, B, q_heads, tables, table_stride, table_width, lengths, max_len, prefix_len,
                     window, scale, out, out_dtype, lse, v, &p.a);
    if (s != PROJ_OK || B == 0) return s;
    const uint64_t pb = static_cast<uint64_t>((prefix_len + cache->page_size - 1) / cache->page_size) * 4;
    const uint64_t ob = static_cast<uint64_t>(B) * q_heads * cache->head_dim * (out_dtype == PROJ_OUT_F32 ? 4 : 2);
    if (overlap(out, ob, prefix, pb) || overlap(lse, lse ? static_cast<uint64_t>(B) * q_heads * 4 : 0, prefix, pb))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "out or lse overlaps an input");
    DeviceGuard g(v.device);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (prefix_len == 0) return finish(ctx, launch_attend(p.a, st));
    p.a.prefix = prefix_len;
    p.pages = prefix;
    const hipError_t e = launch_attend_shared(p, st);
    if (e == hipErrorOutOfMemory)
        return context_error(ctx, PROJ_ERR_NO_MEMORY, "the workspace of %lld bytes does not hold the parts of one sequence",
                             (long long)v.ws_bytes);
    return finish(ctx, e);
}

}  // extern "C"
