// decode.cpp -- C ABI of the decoding operators (declared in
// include/proj.h): argument checks, then one launcher each (quant.hip,
// kvcache.hip, attend.hip).  None of them allocates, synchronises or tunes.
#include <hip/hip_runtime.h>

#include <climits>
#include <utility>

#include "../../include/proj.h"
#include "context.hpp"
#include "decode.hpp"

using namespace proj;

namespace {

// Sizes beyond this cannot be addressed (and keep every product below in 64 bits).
constexpr int64_t kMost = int64_t{1} << 40;

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

proj_status finish(proj_ctx *ctx, hipError_t e) {
    if (e == hipSuccess) return PROJ_OK;
    (void)hipGetLastError();
    return context_error(ctx, PROJ_ERR_HIP, "launch: %s", hipGetErrorString(e));
}

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

bool known_dtype(int d) { return d == PROJ_OUT_F32 || d == PROJ_OUT_BF16; }

// The cache's own fields, and the view that kernels take.
proj_status check_cache(proj_ctx *ctx, const proj_kv_cache *c, CacheArgs *out) {
    if (!c) return context_error(ctx, PROJ_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype != PROJ_KV_BF16 && c->dtype != PROJ_KV_FP8)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown cache dtype %d", (int)c->dtype);
    if (c->heads <= 0 || c->pages < 0 || c->page_size <= 0 || (c->page_size & (c->page_size - 1)) != 0 ||
        c->page_size > (1 << 20) || c->heads > (1 << 16))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "cache: heads %d, pages %lld, page size %d (a power of two)",
                             (int)c->heads, (long long)c->pages, (int)c->page_size);
    if (!attend_dim(c->head_dim))
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "head size %d (64, 80, 96, 128, 192 or 256)", (int)c->head_dim);
    // a cache without pages has no memory either
    if ((c->pages > 0 && (!c->k || !c->v)) || !aligned(c->k, 16) || !aligned(c->v, 16))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "cache: k or v is NULL or not 16-byte aligned");
    const int64_t unit = c->dtype == PROJ_KV_FP8 ? 16 : 8;
    for (int i = 0; i < 3; ++i)
        for (int64_t s : {c->k_strides[i], c->v_strides[i]})
            if (s <= 0 || s % unit != 0 || s > kMost)
                return context_error(ctx, PROJ_ERR_INVALID_ARG, "cache: stride %lld (a positive multiple of %lld)",
                                     (long long)s, (long long)unit);
    if (c->pages > INT32_MAX ||
        (c->pages > 0 && (c->k_strides[0] > kMost / c->pages || c->v_strides[0] > kMost / c->pages)))
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "cache too large");
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || c->k_scale > 3e38f || c->v_scale > 3e38f ||
        (c->dtype == PROJ_KV_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f)))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "cache scales %g, %g (positive; 1 for bf16)",
                             (double)c->k_scale, (double)c->v_scale);
    CacheArgs a;
    a.k = c->k;
    a.v = c->v;
    a.kp = c->k_strides[0], a.kh = c->k_strides[1], a.kt = c->k_strides[2];
    a.vp = c->v_strides[0], a.vh = c->v_strides[1], a.vt = c->v_strides[2];
    a.pages = c->pages;
    a.fp8 = c->dtype == PROJ_KV_FP8;
    a.heads = c->heads;
    a.dim = c->head_dim;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    *out = a;
    return PROJ_OK;
}

// Bytes from the first element to past the last one of k or v.
uint64_t cache_bytes(const proj_kv_cache *c, const int64_t *s) {
    if (c->pages == 0) return 0;
    const uint64_t last = static_cast<uint64_t>(c->pages - 1) * s[0] + static_cast<uint64_t>(c->heads - 1) * s[1] +
                          static_cast<uint64_t>(c->page_size - 1) * s[2] + c->head_dim;
    return last * (c->dtype == PROJ_KV_FP8 ? 1 : 2);
}

bool meets_cache(const proj_kv_cache *c, const void *p, uint64_t n) {
    return overlap(p, n, c->k, cache_bytes(c, c->k_strides)) || overlap(p, n, c->v, cache_bytes(c, c->v_strides));
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
    s = check_cache(ctx, cache, &a.c);
    if (s != PROJ_OK) return s;
    if (T < 0 || q_heads < 0 || q_heads > (1 << 16) || rope_rows < 0 || rot < 0 || rot > cache->head_dim || rot % 2 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "T=%lld q_heads=%d rope_rows=%lld rot=%d (even, at most %d)",
                             (long long)T, q_heads, (long long)rope_rows, rot, (int)cache->head_dim);
    const int64_t width = (static_cast<int64_t>(q_heads) + 2 * cache->heads) * cache->head_dim;
    if (qkv_stride < width || qkv_stride % 8 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "qkv row stride %lld (a multiple of 8, at least %lld)",
                             (long long)qkv_stride, (long long)width);
    if (T == 0) return PROJ_OK;
    if (qkv_stride > kMost / T || rope_rows > kMost / (rot > 0 ? rot : 1))
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "qkv or rope too large");
    if (!qkv || !positions || !slots || (rot > 0 && rope_rows > 0 && !rope))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "qkv, positions, slots or rope is NULL");
    if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(rope, 4) || !aligned(positions, 4) || !aligned(slots, 8))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "qkv or q_out not 16-byte aligned, or an index not aligned");
    const uint64_t xb = (static_cast<uint64_t>(T - 1) * qkv_stride + width) * 2;
    const uint64_t qb = static_cast<uint64_t>(T) * q_heads * cache->head_dim * 2;
    const uint64_t rb = static_cast<uint64_t>(rope_rows) * rot * 4;
    for (const auto &in : {std::make_pair(qkv, xb), std::make_pair(static_cast<const void *>(rope), rb),
                           std::make_pair(static_cast<const void *>(positions), static_cast<uint64_t>(T) * 4),
                           std::make_pair(static_cast<const void *>(slots), static_cast<uint64_t>(T) * 8)})
        if (overlap(q_out, qb, in.first, in.second) || meets_cache(cache, in.first, in.second))
            return context_error(ctx, PROJ_ERR_INVALID_ARG, "q_out or the cache overlaps an input");
    if (meets_cache(cache, q_out, qb))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q_out overlaps the cache");
    DeviceGuard g(v.device);
    a.qkv = static_cast<const uint16_t *>(qkv);
    a.stride = qkv_stride;
    a.T = T;
    a.q_heads = q_heads;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.rope = rope;
    a.rope_rows = rope_rows;
    a.positions = positions;
    a.slots = slots;
    a.q_out = static_cast<uint16_t *>(q_out);
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
    s = check_cache(ctx, cache, &a.c);
    if (s != PROJ_OK) return s;
    if (B < 0 || B > INT32_MAX / 65536 || q_heads <= 0 || q_heads % cache->heads != 0 || q_heads > (1 << 16))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "B=%lld q_heads=%d (a multiple of the cache's %d heads)",
                             (long long)B, q_heads, (int)cache->heads);
    if (table_width < 0 || table_stride < table_width || max_len < 0 || max_len > INT32_MAX || window < 0 ||
        table_width > kMost || max_len > table_width * cache->page_size)
        return context_error(ctx, PROJ_ERR_INVALID_ARG,
                             "max_len %lld, window %lld, tables of %lld pages of %d tokens, rows %lld apart",
                             (long long)max_len, (long long)window, (long long)table_width, (int)cache->page_size,
                             (long long)table_stride);
    if (!known_dtype(out_dtype)) return context_error(ctx, PROJ_ERR_INVALID_ARG, "unknown output dtype %d", out_dtype);
    const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
    if (q_stride < width || q_stride % 8 != 0)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q row stride %lld (a multiple of 8, at least %lld)",
                             (long long)q_stride, (long long)width);
    if (!(scale == scale) || scale > 3e38f || scale < -3e38f)
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "scale is not finite");
    if (B == 0) return PROJ_OK;
    if (q_stride > kMost / B || table_stride > kMost / B)
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "q or tables too large");
    if (!q || !lengths || !out || (max_len > 0 && !tables))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q, tables, lengths or out is NULL");
    const uintptr_t oa = out_dtype == PROJ_OUT_F32 ? 4 : 2;
    if (!aligned(q, 16) || !aligned(tables, 4) || !aligned(lengths, 4) || !aligned(out, 16) || !aligned(lse, 4))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "q or out not 16-byte aligned, or another not to its type");
    const uint64_t ob = static_cast<uint64_t>(B) * width * oa, lb = lse ? static_cast<uint64_t>(B) * q_heads * 4 : 0;
    for (const auto &in : {std::make_pair(q, (static_cast<uint64_t>(B - 1) * q_stride + width) * 2),
                           std::make_pair(static_cast<const void *>(tables),
                                          (static_cast<uint64_t>(B - 1) * table_stride + table_width) * 4),
                           std::make_pair(static_cast<const void *>(lengths), static_cast<uint64_t>(B) * 4)})
        if (overlap(out, ob, in.first, in.second) || overlap(lse, lb, in.first, in.second))
            return context_error(ctx, PROJ_ERR_INVALID_ARG, "out or lse overlaps an input");
    if (meets_cache(cache, out, ob) || meets_cache(cache, lse, lb) || overlap(out, ob, lse, lb))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "out or lse overlaps the cache or each other");
    DeviceGuard g(v.device);
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.B = B;
    a.q_heads = q_heads;
    a.tables = tables;
    a.table_stride = table_stride;
    a.lengths = lengths;
    a.max_len = max_len;
    a.window = window;
    a.scale = scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse;
    a.ws = v.ws;
    a.ws_bytes = v.ws_bytes;
    a.cus = v.cus;
    a.counters = v.counters;
    a.ncounters = v.ncounters;
    return finish(ctx, launch_attend(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
