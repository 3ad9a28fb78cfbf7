// checks.hpp -- argument checks that the decoding operators' entry points
// share (decode.cpp, layer.cpp).
#pragma once

#include <cfloat>
#include <climits>
#include <utility>

#include "../../include/proj.h"
#include "context.hpp"
#include "decode.hpp"

namespace proj {

// Sizes beyond this cannot be addressed (and keep every product below in 64 bits).
constexpr int64_t kMost = int64_t{1} << 40;

inline bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline proj_status finish(proj_ctx *ctx, hipError_t e) {
    if (e == hipSuccess) return PROJ_OK;
    (void)hipGetLastError();
    return context_error(ctx, PROJ_ERR_HIP, "launch: %s", hipGetErrorString(e));
}

inline bool known_dtype(int d) { return d == PROJ_OUT_F32 || d == PROJ_OUT_BF16; }

// The cache's own fields, and the view that kernels take.
inline proj_status check_cache(proj_ctx *ctx, const proj_kv_cache *c, CacheArgs *out) {
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
inline uint64_t cache_bytes(const proj_kv_cache *c, const int64_t *s) {
    if (c->pages == 0) return 0;
    const uint64_t last = static_cast<uint64_t>(c->pages - 1) * s[0] + static_cast<uint64_t>(c->heads - 1) * s[1] +
                          static_cast<uint64_t>(c->page_size - 1) * s[2] + c->head_dim;
    return last * (c->dtype == PROJ_KV_FP8 ? 1 : 2);
}

inline bool meets_cache(const proj_kv_cache *c, const void *p, uint64_t n) {
    return overlap(p, n, c->k, cache_bytes(c, c->k_strides)) || overlap(p, n, c->v, cache_bytes(c, c->v_strides));
}

// A call of the append: its arguments, and what the kernel takes.
inline proj_status check_append(proj_ctx *ctx, const proj_kv_cache *cache, const void *qkv, int64_t qkv_stride, int64_t T,
                                int q_heads, const float *rope, int64_t rope_rows, int rot, int interleaved,
                                const int32_t *positions, const int64_t *slots, void *q_out, AppendArgs *to) {
    AppendArgs a;
    const proj_status s = check_cache(ctx, cache, &a.c);
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
    *to = a;
    return PROJ_OK;
}

// A call of the attention, the first `prefix` tokens of whose sequences are not in the tables: its arguments, and what
// the kernels take.
inline proj_status check_attend(proj_ctx *ctx, const proj_kv_cache *cache, const void *q, int64_t q_stride, int64_t B,
                                int q_heads, const int32_t *tables, int64_t table_stride, int64_t table_width,
                                const int32_t *lengths, int64_t max_len, int64_t prefix, int64_t window, float scale,
                                void *out, int out_dtype, float *lse, const ContextView &v, AttendArgs *to) {
    AttendArgs a;
    const proj_status s = check_cache(ctx, cache, &a.c);
    if (s != PROJ_OK) return s;
    if (B < 0 || B > INT32_MAX / 65536 || q_heads <= 0 || q_heads % cache->heads != 0 || q_heads > (1 << 16))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "B=%lld q_heads=%d (a multiple of the cache's %d heads)",
                             (long long)B, q_heads, (int)cache->heads);
    if (table_width < 0 || table_stride < table_width || max_len < 0 || max_len > INT32_MAX || window < 0 ||
        table_width > kMost || max_len - prefix > table_width * cache->page_size)
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
    if (!(static_cast<double>(scale < 0.f ? -scale : scale) * cache->k_scale <= static_cast<double>(FLT_MAX)))
        return context_error(ctx, PROJ_ERR_INVALID_ARG, "scale %g times the cache's k_scale %g is past the largest float",
                             (double)scale, (double)cache->k_scale);
    if (B == 0) return PROJ_OK;
    if (q_stride > kMost / B || table_stride > kMost / B)
        return context_error(ctx, PROJ_ERR_UNSUPPORTED, "q or tables too large");
    if (!q || !lengths || !out || (max_len > prefix && !tables))
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
    *to = a;
    return PROJ_OK;
}

}  // namespace proj
