// kvcache.hip -- norms of query and key heads, rotary positions and the storing
// of keys and values into a paged key-value cache.
#include "decode.hpp"

namespace proj {

// fp32 -> e4m3 bits (to nearest even), clamped to the largest finite value
// first: the conversion itself has no infinity to saturate to.  NaN stays.
__device__ __forceinline__ uint8_t f32_to_fp8_bits(float v) {
    const float c = v > 448.f ? 448.f : v < -448.f ? -448.f : v;
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xff);
}

typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

// The rotation of one token's item in registers.  An item is 16 elements of a
// head, as x[0][8] and x[1][8]:
//   kHalves      pair j is (j, j + rot / 2), rot a multiple of 16: for c < rot / 16
//                elements 8 c .. + 7 and their partners rot / 2 further on, for
//                the rest (not rotated) 16 c .. + 15
//   kNeighbours  pair j is (2 j, 2 j + 1), rot a multiple of 16: 16 c .. + 15
//   kAny         either pairing, any rot and alignment: 16 c .. + 15, partners
//                and table entries read one by one, out of the caches
enum Pairing { kHalves = 0, kNeighbours = 1, kAny = 2 };

__device__ __forceinline__ void load8(const uint16_t *p, float *x) {
    const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store8(uint16_t *p, const float *x) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f32_to_bf16_bits(x[2 * i]) | static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i + 1])) << 16;
    *reinterpret_cast<u32x4 *>(p) = w;
}

__device__ __forceinline__ void store8_fp8(uint8_t *p, const float *x, float scale) {
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= static_cast<uint32_t>(f32_to_fp8_bits(x[i] / scale)) << (8 * (i % 4));
    *reinterpret_cast<u32x2 *>(p) = w;
}

// A norm's weights of an item's eight elements.
__device__ __forceinline__ void load8_weights(const AppendArgs &a, const void *norm, int64_t at, float *w) {
    if (a.norm_f32) {
        const float *p = static_cast<const float *>(norm) + at;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(p + 4 * v);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * v + k] = x[k];
        }
    } else {
        load8(static_cast<const uint16_t *>(norm) + at, w);
    }
}

// A thread has one item of TOK tokens, T / TOK apart in no order that
// matters: their loads are in flight together, and the item's head and place
// are worked out once.  Bound by bytes: each is read and written once, the
// table's rows come from the caches; 8192 tokens of 80 heads of 128 into an 8-bit
// cache 64.5 us, 5.0 TB/s, a copy's rate (an element to a thread: 203 us).
//
// NORM: a query or key head is first divided by the root of its mean square
// (plus eps) and multiplied by its weights. A head's items are then neighbouring
// lanes of one wave, 4, 8 or 16 of them (those past D / 16 have no elements), and
// exchange their sums of squares, which are fp32 unless they near its ends: then
// 64 bits, so that no bf16 input overflows or vanishes (64 bits for all heads took
// 81 us where this takes 73, 8192 tokens back to back, their conversions at a quarter of
// the rate).
template <int PAIRING, int TOK, bool NORM>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, uint32_t blocks) {
    const int D = a.c.dim, per = NORM ? a.norm_lanes : D / 16;
    const int item = static_cast<int>(blockIdx.x % blocks) * 256 + threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / blocks) * TOK;
    const int head = item / per, Hq = a.q_heads, Hkv = a.c.heads;
    int c = item % per;
    const int kind = head < Hq ? 0 : head < Hq + Hkv ? 1 : 2;  // query, key, value
    if (head >= Hq + 2 * Hkv || (kind == 0 && !a.q_out)) return;
    const bool idle = NORM && c >= D / 16;  // a lane that only takes part in the exchange
    if (idle) c = D / 16 - 1;
    const int half = a.rot / 2;
    // the item's two runs of eight, and whether they are rotated
    int e0 = 16 * c, e1 = 16 * c + 8;
    bool turns = kind != 2 && e0 < a.rot;
    if (PAIRING == kHalves && kind != 2) {
        turns = 8 * c < half;
        if (turns) {
            e0 = 8 * c;
            e1 = half + 8 * c;
        }
    }
    const uint16_t *row = a.qkv + t0 * a.stride + static_cast<int64_t>(head) * D;
    const void *norm = !NORM || kind == 2 ? nullptr : kind == 0 ? a.q_norm : a.k_norm;
    const int64_t norm_at = a.norm_per_head ? static_cast<int64_t>(kind == 0 ? head : head - Hq) * D : 0;
    float weight[2][8];
    if (NORM && norm) {
        load8_weights(a, norm, norm_at + e0, weight[0]);
        load8_weights(a, norm, norm_at + e1, weight[1]);
    }

    float x[TOK][2][8];
    int64_t slot[TOK];
    int32_t pos[TOK];
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        const int64_t t = t0 + i < a.T ? i : a.T - 1 - t0;  // past the end: the last one, not stored
        load8(row + t * a.stride + e0, x[i][0]);
        load8(row + t * a.stride + e1, x[i][1]);
        pos[i] = a.positions[t0 + t];
        slot[i] = a.slots[t0 + t];
    }
    float sum[TOK];  // of the head's squares
    if (NORM && norm) {
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            sum[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[i] = __builtin_fmaf(x[i][k / 8][k % 8], x[i][k / 8][k % 8], sum[i]);
            if (idle) sum[i] = 0.f;
        }
        for (int h = 1; h < per; h <<= 1)
#pragma unroll
            for (int i = 0; i < TOK; ++i) sum[i] += __shfl_xor(sum[i], h, 64);
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        if (t0 + i >= a.T) break;
        const bool known = a.rot == 0 || (pos[i] >= 0 && pos[i] < a.rope_rows);
        const float *cs = a.rope + static_cast<int64_t>(known ? pos[i] : 0) * a.rot;
        float root = 1.f, up = 1.f;  // a normed element is x * up * root * weight
        if (NORM && norm) {
            if (sum[i] > 0x1p-60f && sum[i] < 0x1p100f) {
                root = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[i], a.norm_share, a.eps));
            } else {  // squares, or their sum, near the ends of fp32 (or no numbers): in 64 bits
                double wide = 0.0;
#pragma unroll
                for (int k = 0; k < 16; ++k) wide = __builtin_fma(x[i][k / 8][k % 8], static_cast<double>(x[i][k / 8][k % 8]), wide);
                if (idle) wide = 0.0;
                for (int h = 1; h < per; h <<= 1) wide += __shfl_xor(wide, h, 64);
                const double r = 1.0 / sqrt(wide / D + static_cast<double>(a.eps));
                // up to 2^133 and down to 2^-128: brought near one by a power of two on either side
                up = r > 0x1p60 ? 0x1p64f : r < 0x1p-60 ? 0x1p-64f : 1.f;
                root = static_cast<float>(r / up);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[i][k / 8][k % 8] *= up;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) x[i][k / 8][k % 8] = x[i][k / 8][k % 8] * root * weight[k / 8][k % 8];
        }
        if (turns && known) {
            if constexpr (PAIRING == kHalves) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const f32x4 co = *reinterpret_cast<const f32x4 *>(cs + e0 + 4 * v);
                    const f32x4 si = *reinterpret_cast<const f32x4 *>(cs + half + e0 + 4 * v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p = x[i][0][4 * v + k], q = x[i][1][4 * v + k];
                        x[i][0][4 * v + k] = p * co[k] - q * si[k];
                        x[i][1][4 * v + k] = q * co[k] + p * si[k];
                    }
                }
            } else if constexpr (PAIRING == kNeighbours) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const f32x4 co = *reinterpret_cast<const f32x4 *>(cs + 8 * c + 4 * v);
                    const f32x4 si = *reinterpret_cast<const f32x4 *>(cs + half + 8 * c + 4 * v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p = x[i][v][2 * k], q = x[i][v][2 * k + 1];
                        x[i][v][2 * k] = p * co[k] - q * si[k];
                        x[i][v][2 * k + 1] = q * co[k] + p * si[k];
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int d = 16 * c + 8 * v + k;
                        if (d < a.rot) {
                            const int j = a.interleaved ? d >> 1 : d < half ? d : d - half;
                            const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
                            const int partner = a.interleaved ? d ^ 1 : second ? d - half : d + half;
                            float u = bf16_bits_to_f32(row[i * a.stride + partner]);
                            if (NORM && norm)
                                u = u * up * root *
                                    (a.norm_f32 ? static_cast<const float *>(norm)[norm_at + partner]
                                                : bf16_bits_to_f32(static_cast<const uint16_t *>(norm)[norm_at + partner]));
                            const float co = cs[j], si = cs[half + j];
                            x[i][v][k] = second ? x[i][v][k] * co + u * si : x[i][v][k] * co - u * si;
                        }
                    }
            }
        }
        if (idle) continue;
        if (kind == 0) {
            if (!known)
#pragma unroll
                for (int k = 0; k < 8; ++k) x[i][0][k] = x[i][1][k] = __builtin_nanf("");
            uint16_t *to = a.q_out + ((t0 + i) * Hq + head) * D;
            store8(to + e0, x[i][0]);
            store8(to + e1, x[i][1]);
            continue;
        }
        const int64_t page = slot[i] >> a.c.page_shift, place = slot[i] & ((int64_t{1} << a.c.page_shift) - 1);
        if (!known || slot[i] < 0 || page >= a.c.pages) continue;
        const bool is_v = kind == 2;
        const int64_t at = is_v ? page * a.c.vp + (head - Hq - Hkv) * a.c.vh + place * a.c.vt
                                : page * a.c.kp + (head - Hq) * a.c.kh + place * a.c.kt;
        if (a.c.fp8) {
            uint8_t *to = static_cast<uint8_t *>(is_v ? a.c.v : a.c.k) + at;
            const float scale = is_v ? a.c.v_scale : a.c.k_scale;
            store8_fp8(to + e0, x[i][0], scale);
            store8_fp8(to + e1, x[i][1], scale);
        } else {
            uint16_t *to = static_cast<uint16_t *>(is_v ? a.c.v : a.c.k) + at;
            store8(to + e0, x[i][0]);
            store8(to + e1, x[i][1]);
        }
    }
}

#define PROJ_APPEND_INST(P)                                                    \
    template __global__ void append_kernel<P, 1, false>(AppendArgs, uint32_t); \
    template __global__ void append_kernel<P, 4, false>(AppendArgs, uint32_t); \
    template __global__ void append_kernel<P, 1, true>(AppendArgs, uint32_t);
PROJ_APPEND_INST(kHalves)
PROJ_APPEND_INST(kNeighbours)
PROJ_APPEND_INST(kAny)

#ifndef __HIP_DEVICE_COMPILE__
template <int PAIRING, bool NORM>
static hipError_t launch_append_as(AppendArgs a, hipStream_t st) {
    a.norm_lanes = a.c.dim <= 64 ? 4 : a.c.dim <= 128 ? 8 : 16;
    a.norm_share = 1.f / a.c.dim;
    const int64_t items = (static_cast<int64_t>(a.q_heads) + 2 * a.c.heads) * (NORM ? a.norm_lanes : a.c.dim / 16);
    const int64_t blocks = (items + 255) / 256;
    // four tokens to a thread once that leaves enough threads for the chip; normed, one: four are no faster (8192
    // tokens of 80 heads 73 us back to back with either, 65 alone)
    const int tok = !NORM && a.T * items >= (int64_t{1} << 20) ? 4 : 1;
    auto kernel = append_kernel<PAIRING, 1, NORM>;
    if constexpr (!NORM)
        if (tok == 4) kernel = append_kernel<PAIRING, 4, false>;
    // as many tokens at a time as one launch can have threads for
    const int64_t most = most_groups(256) / blocks * tok;
    AppendArgs s = a;
    for (int64_t t = 0; t < a.T; t += most) {
        s.T = a.T - t < most ? a.T - t : most;
        s.qkv = a.qkv + t * a.stride;
        s.positions = a.positions + t;
        s.slots = a.slots + t;
        s.q_out = a.q_out ? a.q_out + t * a.q_heads * a.c.dim : nullptr;
        const int64_t grid = (s.T + tok - 1) / tok * blocks;
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, s, static_cast<uint32_t>(blocks));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool NORM>
static hipError_t launch_append_norm(const AppendArgs &a, hipStream_t st) {
    if (a.rot % 16 != 0 || reinterpret_cast<uintptr_t>(a.rope) % 16 != 0) return launch_append_as<kAny, NORM>(a, st);
    return a.interleaved ? launch_append_as<kNeighbours, NORM>(a, st) : launch_append_as<kHalves, NORM>(a, st);
}

hipError_t launch_append(const AppendArgs &a, hipStream_t st) {
    return a.q_norm || a.k_norm ? launch_append_norm<true>(a, st) : launch_append_norm<false>(a, st);
}
#endif

}  // namespace proj
