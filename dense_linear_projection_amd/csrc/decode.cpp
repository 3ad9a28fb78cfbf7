// decode.cpp -- C ABI of the decoding operators (declared in
// include/proj.h): argument checks, then one launcher each (quant.hip,
// kvcache.hip, attend.hip).  None of them allocates, synchronises or tunes.
#include <hip/hip_runtime.h>

#include <climits>
#include <utility>

#include "checks.hpp"

using namespace proj;

namespace {

// N, K and group of 4-bit weights.
proj_status check_quant_shape(proj_ctx *ctx, int64_t N, int64_t K, int group) {
    if (N < 0 || K < 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "negative size N=%lld K=%lld", (long long)N, (long long)K);
    if (K % 8 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "4-bit weights need K a multiple of 8, got %lld", (long long)K);
    if (group != 32 && group != 64 && group != 128)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "group %d is not 32, 64 or 128", group);
    if (K > 0 && N > kMost / K)
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "N*K too large");
    return PROJ_OK;
}

}  // namespace

extern "C" {

proj_status proj_pack_codes(proj_ctx *ctx, const uint8_t *q, int64_t N, int64_t K, uint32_t *codes, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    s = check_quant_shape(ctx, N, K, 32);
    if (s != PROJ_OK || N == 0 || K == 0) return s;
    if (!q || !codes || !aligned(codes, 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q or codes is NULL, or codes not 4-byte aligned");
    if (overlap(q, static_cast<uint64_t>(N) * K, codes, static_cast<uint64_t>(N) * K / 2))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "codes overlaps q");
    DeviceGuard g(v.device);
    return finish(ctx, launch_pack_codes(q, N, K, codes, static_cast<hipStream_t>(stream)));
}

proj_status proj_quantize_weights(proj_ctx *ctx, const void *W, int64_t N, int64_t K, int group, uint32_t *codes,
                                  void *scales, int scale_dtype, uint8_t *zeros, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    s = check_quant_shape(ctx, N, K, group);
    if (s != PROJ_OK) return s;
    if (!known_dtype(scale_dtype))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown scale dtype %d", scale_dtype);
    if (N == 0 || K == 0) return PROJ_OK;
    if (!W || !codes || !scales || !aligned(W, 2) || !aligned(codes, 4) ||
        !aligned(scales, scale_dtype == PROJ_OUT_F32 ? 4 : 2))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "W, codes or scales is NULL or not aligned to its type");
    const uint64_t wb = static_cast<uint64_t>(N) * K * 2, gb = static_cast<uint64_t>(N) * ((K + group - 1) / group);
    const uint64_t sb = gb * (scale_dtype == PROJ_OUT_F32 ? 4 : 2);
    if (overlap(W, wb, codes, wb / 4) || overlap(W, wb, scales, sb) || overlap(W, wb, zeros, gb) ||
        overlap(codes, wb / 4, scales, sb) || overlap(codes, wb / 4, zeros, gb) || overlap(scales, sb, zeros, gb))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "operands overlap");
    DeviceGuard g(v.device);
    return finish(ctx, launch_quantize(static_cast<const uint16_t *>(W), N, K, group, codes, scales,
                                       scale_dtype == PROJ_OUT_F32, zeros, static_cast<hipStream_t>(stream)));
}

proj_status proj_run_quant(proj_ctx *ctx, const void *X, const uint32_t *codes, const void *scales, int scale_dtype,
                           const uint8_t *zeros, int group, const void *bias, int epilogue, int64_t M, int64_t N,
                           int64_t K, void *Y, int out_dtype, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    if (M < 0) return context_error(ctx, PROJ_ERR_INVALID_ARG, "negative size M=%lld", (long long)M);
    s = check_quant_shape(ctx, N, K, group);
    if (s != PROJ_OK) return s;
    if (epilogue < PROJ_EPI_NONE || epilogue > PROJ_EPI_BIAS_GELU_TANH)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
    if (!known_dtype(out_dtype) || !known_dtype(scale_dtype))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown output dtype %d or scale dtype %d", out_dtype,
                             scale_dtype);
    if (M == 0 || N == 0) return PROJ_OK;
    if (M > kMost / N || (K > 0 && M > kMost / K)) return context_error(ctx, PROJ_ERR_UNSUPPORTED, "M*N or M*K too large");
    const uintptr_t ya = out_dtype == PROJ_OUT_F32 ? 4 : 2, sa = scale_dtype == PROJ_OUT_F32 ? 4 : 2;
    if (!Y || (K > 0 && (!X || !codes || !scales)) || ((epilogue & 1) && !bias))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "X, codes, scales, Y or the epilogue's bias is NULL");
    if (!aligned(Y, ya) || !aligned(X, 2) || !aligned(codes, 4) || !aligned(scales, sa) || !aligned(bias, 2))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
    const int64_t G = (K + group - 1) / group;
    const uint64_t yb = static_cast<uint64_t>(M) * N * ya;
    if (overlap(Y, yb, X, static_cast<uint64_t>(M) * K * 2) || overlap(Y, yb, codes, static_cast<uint64_t>(N) * K / 2) ||
        overlap(Y, yb, scales, static_cast<uint64_t>(N) * G * sa) ||
        overlap(Y, yb, zeros, static_cast<uint64_t>(N) * G) ||
        ((epilogue & 1) && overlap(Y, yb, bias, static_cast<uint64_t>(N) * 2)))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "Y overlaps an input");
    DeviceGuard g(v.device);
    QuantArgs a;
    a.X = static_cast<const uint16_t *>(X);
    a.codes = codes;
    a.scales = scales;
    a.zeros = zeros;
    a.bias = static_cast<const uint16_t *>(bias);
    a.Y = Y;
    a.M = M, a.N = N, a.K = K, a.G = G;
    a.group = group;
    a.scales_f32 = scale_dtype == PROJ_OUT_F32;
    a.epi = epilogue;
    a.out = out_dtype;
    a.ws = v.ws;
    a.ws_bytes = v.ws_bytes;
    a.cus = v.cus;
    return finish(ctx, launch_quant(a, static_cast<hipStream_t>(stream)));
}

proj_status proj_kv_append(proj_ctx *ctx, const proj_kv_cache *cache, const void *qkv, int64_t qkv_stride, int64_t T,
                           int q_heads, const float *rope, int64_t rope_rows, int rot, int interleaved,
                           const int32_t *positions, const int64_t *slots, void *q_out, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    AppendArgs a;
    s = check_append(ctx, cache, qkv, qkv_stride, T, q_heads, rope, rope_rows, rot, interleaved, positions, slots, q_out, &a);
    if (s != PROJ_OK || T == 0) return s;
    DeviceGuard g(v.device);
    return finish(ctx, launch_append(a, static_cast<hipStream_t>(stream)));
}

proj_status proj_kv_attend(proj_ctx *ctx, const proj_kv_cache *cache, const void *q, int64_t q_stride, int64_t B,
                           int q_heads, const int32_t *tables, int64_t table_stride, int64_t table_width,
                           const int32_t *lengths, int64_t max_len, int64_t window, float scale, void *out,
                           int out_dtype, float *lse, void *stream) {
    ContextView v;
    proj_status s = context_view(ctx, &v);
    if (s != PROJ_OK) return s;
    AttendArgs a;
    s = check_attend(ctx, cache, q, q_stride, B, q_heads, tables, table_stride, table_width, lengths, max_len, 0, window, scale,
                     out, out_dtype, lse, v, &a);
    if (s != PROJ_OK || B == 0) return s;
    DeviceGuard g(v.device);
    return finish(ctx, launch_attend(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
