// attend.hip -- attention of one new token for each sequence over its pages
// of a key-value cache, split over the length and joined.
//
// For a key-value head and the `per` query heads that share it, over the
// tokens t of one part of the length,
//     w[t][h] = scale <q[h], k[t]>,  m = max_t w,  l = sum_t exp(w - m),
//     o[h][:] = sum_t exp(w[t][h] - m) v[t][:],
// and parts with (m, l, o) join as (M = max m, sum exp(m - M) l, ...): one
// pass over keys and values, which bound the call (each serves `per` query
// heads: about per operations a byte, far below the matrix cores' rate).
//
// A workgroup is four waves on one (sequence, key-value head, part); wave w
// takes tiles w, w + 4, ... of 32 tokens, with its own running maximum, sum
// and output, joined through LDS at the end, so the loop has no barrier.
//   * w: v_mfma_f32_16x16x32_bf16 with A = 16 tokens of K (lane l: token
//     l % 16, 8 elements) and B = 16 heads of q, held for the whole call.  A
//     lane of the result has head l % 16 and tokens 4 (l / 16) + r.
//   * o: A = V transposed (16 elements of the head x 32 tokens), B = the
//     probabilities.  Two results of the first product, as they lie, are the
//     32 tokens of B if slot 8 g + i of the product's k axis is token
//     4 g + i (i < 4) or 16 + 4 g + i - 4; V follows by being read in that
//     order with LDS's transposing loads.  So the probabilities never leave
//     the registers.
//   * a probability enters as three bf16 terms of 8 bits each, which together
//     are its 24 bits.  Two would be faster by 1% (6% with 8-bit keys: 64
//     sequences of 2000 tokens 40.6 us, with three 43), but four of a thousand
//     bf16 results were then not the correctly rounded ones, where fp32 sums
//     leave half of one.  The terms are cut, so that what is left is never
//     negative; those after the first are at least 2^-30 of it, so that an
//     infinite value does not meet a zero, and zero where it is, so that a
//     vanished probability takes nothing from a large value.
//   * K and V are read a KB at a time (whole rows, in the order they lie) into
//     registers, put into LDS and read from there as the products need them;
//     those of the next tile are on their way while this one is computed, 16 KB
//     a wave at 128 elements in bf16, and nothing waits for anything but its own
//     operands.  They are kept out of the caches (non-temporal loads, ONCE)
//     unless heads share memory lines: a workgroup reads them once, for 16
//     query heads (32 where D <= 128); those of more are other workgroups, which
//     read them again.
// Bound by bytes where lengths are large: one sequence of 131072 tokens (8
// heads of 128 in bf16, 537 MB) 91 us, 6.0 TB/s; 32 sequences up to 16384 tokens
// 205 us, 5.6 TB/s; by latency where they are small: 500 tokens 8.5 us.
// The running maximum moves only when a logit passes it by more than 5 (a
// factor of 148): sums stay in range, and most tiles need no rescaling and no
// exchange between lanes.  Logits are kept in natural units, and scaled to base
// 2 once the maximum is taken off: scaled first, those past 2.36e38 overflowed.
#include <type_traits>

#include "decode.hpp"

namespace proj {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

constexpr int kTerms = 3;          // bf16 terms of a probability
constexpr int kChunk = 2048;       // tokens whose pages are staged at once
constexpr int kJoined = 32;         // parts that the attention kernel joins itself (500 tokens: 8.0 us, in two kernels 9.3)
constexpr float kLowest = -0x1.fffffep127f;  // a running maximum before the first logit: the lowest finite one
constexpr float kLog2e = 1.4426950408889634f;

// Four e4m3 bytes -> bf16, exact; two 32-bit words of pairs.
__device__ __forceinline__ u32x2 fp8x4_to_bf16(uint32_t w) {
    u32x2 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    return r;
}

__device__ __forceinline__ bf16x8 fp8x8_to_bf16(uint32_t lo, uint32_t hi) {
    const u32x2 a = fp8x4_to_bf16(lo), b = fp8x4_to_bf16(hi);
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// exp(x - most)
__device__ __forceinline__ float exp_above(float x, float most) { return __builtin_amdgcn_exp2f((x - most) * kLog2e); }

template <int D, bool FP8, int QT>
struct AttendCfg {
    static constexpr int ROW = D * (FP8 ? 1 : 2);        // bytes of a token
    static constexpr int NC = ROW / 16;                  // its 16-byte chunks
    static constexpr int KS = (D + 31) / 32;             // steps of the first product
    static constexpr int DT = D / 16;                    // tiles of the second
    static constexpr int VI = (32 * NC + 63) / 64;       // chunks of V to a lane
    static constexpr int TILE = 32 * ROW;                // bytes of a tile of K or V in LDS
    static constexpr int ORED = 4 * 16 * (D + 4) * 4;    // the waves' outputs, 16 heads at a time
    static constexpr int LDS = 8 * TILE > ORED ? 8 * TILE : ORED;
    // rows after which a row starts at the same LDS bank again
    static constexpr int PERIOD = ROW % 256 == 0 ? 1 : ROW % 128 == 0 ? 2 : ROW % 64 == 0 ? 4 : ROW % 32 == 0 ? 8 : 16;
    // where chunk c of row r of K lies: turned by the row, so that one chunk of 16 rows falls on different banks
    static __device__ __forceinline__ int place_k(int c, int r) { return (c + r / PERIOD) % NC; }
    // the same for V and the rows of one transposing load
    static __device__ __forceinline__ int place(int c, int r) {
        const int turn = FP8 ? r / PERIOD + (r >= 16 ? 4 : 0) : 2 * (r / PERIOD);
        return (c + turn) % NC;
    }
    // first element of the 8 that lane group g has in step i (the same order for q and k)
    static __device__ __forceinline__ int element(int i, int g) {
        return FP8 && i < 2 * (D / 64) ? 64 * (i / 2) + 16 * g + 8 * (i % 2) : 32 * i + 8 * g;
    }
};

// First token of a sequence that is seen, and how many parts its tokens make.
__device__ __forceinline__ int64_t first_seen(const AttendArgs &a, int64_t n) {
    return a.window > 0 && n > a.window ? n - a.window : 0;
}
__device__ __forceinline__ int parts_of(const AttendArgs &a, int64_t n) {
    if (n <= 0 || n > a.max_len) return 0;
    return static_cast<int>((n - first_seen(a, n) + a.part - 1) / a.part);
}

// Four elements of a finished head (and, with the first, its logarithm of the sum).
__device__ __forceinline__ void finish_head(const AttendArgs &a, int64_t at, int64_t row, int d, f32x4 v, float most,
                                            float total) {
    const float f = total == 0.f ? 0.f : a.c.v_scale / total;
    v = total == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * f;
    if (a.out_dtype == OUT_F32) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = v;
    } else {
        const uint32_t lo = f32_to_bf16_bits(v[0]) | static_cast<uint32_t>(f32_to_bf16_bits(v[1])) << 16;
        const uint32_t hi = f32_to_bf16_bits(v[2]) | static_cast<uint32_t>(f32_to_bf16_bits(v[3])) << 16;
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + at) = u32x2{lo, hi};
    }
    if (d == 0 && a.lse)
        a.lse[row] = total == 0.f ? -__builtin_inff() : most + __builtin_amdgcn_logf(total) * 0.6931471805599453f;
}

// Two floats of a part's result: through the device's memory where another
// workgroup of the same launch reads them.
__device__ __forceinline__ void put_part(float *to, float x, float y, int shared) {
    const uint64_t v = static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
    if (shared)
        __hip_atomic_store(reinterpret_cast<uint64_t *>(to), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else
        *reinterpret_cast<uint64_t *>(to) = v;
}
__device__ __forceinline__ float2 get_part(const float *from) {
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t *>(from), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return float2{__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32))};
}

// Two workgroups to a compute unit where their registers (and 160 KB of LDS) allow it.
template <int D, bool FP8, int QT, bool ONCE>
__global__ __launch_bounds__(256, D * QT <= 128 ? 2 : 1) void attend_kernel(AttendArgs a) {
    using C = AttendCfg<D, FP8, QT>;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    __shared__ uint32_t pages[kChunk + 2];
    __shared__ float top[4][16], sum[4][16];
    __shared__ int wrong, is_last;

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = a.q_heads / a.c.heads;
    // workgroup -> (sequence, part, head, chunk of the head's queries), heads
    // fastest.  Ids go round the eight dies in turn: where the heads share
    // memory lines, the heads of a part are given to one die (and the parts of a
    // sequence to different ones), whose L2 then reads a line once.
    const uint32_t hh = static_cast<uint32_t>(a.c.heads * a.chunks);
    uint32_t u = blockIdx.x / hh, hc = blockIdx.x % hh;
    if (a.by_die) {
        const uint32_t die = blockIdx.x % 8, local = blockIdx.x / 8, group = local / hh;
        hc = local % hh;
        u = group * 8 + (die + group * 3) % 8;
        if (u >= static_cast<uint32_t>(a.B * a.parts)) return;
    }
    const int64_t b = u / static_cast<uint32_t>(a.parts);
    const int part = static_cast<int>(u % static_cast<uint32_t>(a.parts));
    const int h = static_cast<int>(hc) / a.chunks, q0 = static_cast<int>(hc) % a.chunks * (16 * QT);
    const int64_t n = a.lengths[b];
    const int parts = parts_of(a, n);
    if (part >= (parts > 0 ? parts : 1)) return;
    const int64_t first = first_seen(a, n) + part * a.part;
    const int64_t last = parts == 0 ? first : n < first + a.part ? n : first + a.part;
    if (tid == 0) wrong = n < 0 || n > a.max_len;

    bf16x8 q[QT][C::KS];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
            const int hq = q0 + 16 * t + c16, e = C::element(i, g);
            q[t][i] = bf16x8{};
            if (hq < per && e < D) q[t][i] = load16(a.q + b * a.q_stride + (static_cast<int64_t>(h) * per + hq) * D + e);
        }
    f32x4 o[QT][C::DT];
    float m[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = kLowest;
        l[t] = 0.f;
#pragma unroll
        for (int i = 0; i < C::DT; ++i) o[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const char *kb = static_cast<const char *>(a.c.k) + h * a.c.kh * (FP8 ? 1 : 2);
    const char *vb = static_cast<const char *>(a.c.v) + h * a.c.vh * (FP8 ? 1 : 2);
    const int64_t place_mask = (int64_t{1} << a.c.page_shift) - 1;
    const float to_logit = a.scale * a.c.k_scale;
    char *kt = lds + wave * 2 * C::TILE, *vt = kt + C::TILE;
    u32x4 kr[C::VI], vr[C::VI];

    for (int64_t base = first; base < last; base += kChunk) {
        const int64_t end = last < base + kChunk ? last : base + kChunk;
        const int64_t page0 = base >> a.c.page_shift;
        const int npages = static_cast<int>(((end - 1) >> a.c.page_shift) - page0) + 1;
        __syncthreads();  // the pages of the chunk before are no longer read
        for (int i = tid; i < npages; i += 256) {
            const int32_t p = a.tables[b * a.table_stride + page0 + i];
            const bool ok = p >= 0 && p < a.c.pages;
            pages[i] = ok ? static_cast<uint32_t>(p) : 0u;
            if (!ok) wrong = 1;
        }
        __syncthreads();
        if (wrong) break;  // nothing is read through a wrong table
        const int tiles = static_cast<int>((end - base + 31) / 32), left = static_cast<int>(end - base);
        const int in_page = static_cast<int>(base & place_mask);

        // byte offset of a token of the chunk (one past its end: the last one, masked later)
        auto offset = [&](int t, int64_t page_stride, int64_t token_stride) -> int64_t {
            const int at = in_page + (t < left ? t : left - 1);
            const int64_t e = static_cast<int64_t>(pages[at >> a.c.page_shift]) * page_stride +
                              static_cast<int64_t>(at & static_cast<int>(place_mask)) * token_stride;
            return FP8 ? e : 2 * e;
        };
        auto load = [&](u32x4 *r, const char *from, int j, int64_t page_stride, int64_t token_stride) {
#pragma unroll
            for (int i = 0; i < C::VI; ++i) {
                const int id = i * 64 + lane < 32 * C::NC ? i * 64 + lane : 32 * C::NC - 1;
                const u32x4 *p = reinterpret_cast<const u32x4 *>(
                    from + offset(32 * j + id / C::NC, page_stride, token_stride) + id % C::NC * 16);
                r[i] = ONCE ? __builtin_nontemporal_load(p) : *p;
            }
        };
        auto load_k = [&](int j) { load(kr, kb, j, a.c.kp, a.c.kt); };
        auto load_v = [&](int j) { load(vr, vb, j, a.c.vp, a.c.vt); };

        // Workgroups start at different tiles: many run in step, and their
        // tiles lie a power of two apart, which would gather their reads on
        // few memory channels.
        const int turn = static_cast<int>((static_cast<uint32_t>(part) * 5u + hc * 3u + static_cast<uint32_t>(b) * 7u) %
                                          static_cast<uint32_t>(tiles));
        auto tile_of = [&](int i) { return i >= tiles ? tiles : i + turn < tiles ? i + turn : i + turn - tiles; };
        if (wave < tiles) {
            load_k(tile_of(wave));
            load_v(tile_of(wave));
        }
        for (int i0 = wave; i0 < tiles; i0 += 4) {
            const int j = tile_of(i0), next = tile_of(i0 + 4);
            const bool whole = 32 * j + 32 <= left;
            f32x4 s[QT][2];
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::VI; ++i) {
                const int id = i * 64 + lane, r = id / C::NC;
                if (64 * C::VI == 32 * C::NC || id < 32 * C::NC)
                    *reinterpret_cast<u32x4 *>(kt + r * C::ROW + C::place_k(id % C::NC, r) * 16) = kr[i];
            }
            load_k(next);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < C::KS; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 16 * x + c16, e = C::element(i, g);
                    bf16x8 k = bf16x8{};
                    if (e < D) {
                        const char *at = kt + r * C::ROW;
                        if constexpr (FP8) {
                            const u32x2 w = *reinterpret_cast<const u32x2 *>(at + C::place_k(e / 16, r) * 16 + e % 16);
                            k = fp8x8_to_bf16(w[0], w[1]);
                        } else {
                            k = *reinterpret_cast<const bf16x8 *>(at + C::place_k(e / 8, r) * 16);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t) s[t][x] = mfma16x16x32(k, q[t][i], s[t][x]);
                }

            bf16x8 prob[QT][kTerms];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float w[8], most = kLowest;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[i] = s[t][i / 4][i % 4] * to_logit;
                    if (!whole && 32 * j + 16 * (i / 4) + 4 * g + i % 4 >= left) w[i] = -__builtin_inff();
                    most = fmaxf(most, w[i]);
                }
                if (__any(most > m[t] + 5.f)) {
                    most = fmaxf(most, __shfl_xor(most, 16, 64));
                    most = fmaxf(fmaxf(most, __shfl_xor(most, 32, 64)), m[t]);
                    const float f = exp_above(m[t], most);
                    m[t] = most;
                    l[t] *= f;
#pragma unroll
                    for (int i = 0; i < C::DT; ++i) o[t][i] *= f;
                }
                uint32_t bits[kTerms][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p[2], least[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[e] = exp_above(w[2 * i + e], m[t]);
                        l[t] += p[e];
                        least[e] = p[e] * 0x1p-30f;
                    }
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) {
                        const uint32_t u0 = __float_as_uint(p[0]) & 0xffff0000u, u1 = __float_as_uint(p[1]) & 0xffff0000u;
                        bits[k][i] = (u0 >> 16) | u1;
                        p[0] = fmaxf(p[0] - __uint_as_float(u0), least[0]);
                        p[1] = fmaxf(p[1] - __uint_as_float(u1), least[1]);
                    }
                }
#pragma unroll
                for (int k = 0; k < kTerms; ++k)
                    prob[t][k] = __builtin_bit_cast(bf16x8, u32x4{bits[k][0], bits[k][1], bits[k][2], bits[k][3]});
            }

#pragma unroll
            for (int i = 0; i < C::VI; ++i) {
                const int id = i * 64 + lane, r = id / C::NC;
                // what lies past the sequence is zero here: its probability is too, and zero times NaN is not
                if (!whole && 32 * j + r >= left) vr[i] = u32x4{0u, 0u, 0u, 0u};
                if (64 * C::VI == 32 * C::NC || id < 32 * C::NC)
                    *reinterpret_cast<u32x4 *>(vt + r * C::ROW + C::place(id % C::NC, r) * 16) = vr[i];
            }
            load_v(next);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < C::DT; ++i) {
                bf16x8 v;
                if constexpr (FP8) {
                    const int r = c16 < 8 ? 4 * g + c16 / 2 : 12 + 4 * g + c16 / 2;  // rows 16 + 4 g + (c16 / 2 - 4)
                    const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (__attribute__((address_space(3))) i32x2 *)(vt + r * C::ROW + C::place(i, r) * 16 + (c16 & 1) * 8));
                    v = fp8x8_to_bf16(static_cast<uint32_t>(x[0]), static_cast<uint32_t>(x[1]));
                } else {
                    s16x4 x[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 16 * y + 4 * g + c16 / 4, ch = 2 * i + (c16 & 3) / 2;
                        x[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4 *)(vt + r * C::ROW + C::place(ch, r) * 16 + (c16 & 1) * 8));
                    }
                    v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) o[t][i] = mfma16x16x32(v, prob[t][k], o[t][i]);
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
        }
    }

    // join the waves, 16 heads at a time
    const float nan = __builtin_nanf("");
    float *red = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float all = l[t];
        all += __shfl_xor(all, 16, 64);
        all += __shfl_xor(all, 32, 64);
        __syncthreads();
        if (g == 0) {
            top[wave][c16] = m[t];
            sum[wave][c16] = all;
        }
#pragma unroll
        for (int i = 0; i < C::DT; ++i)
            *reinterpret_cast<f32x4 *>(red + (wave * 16 + c16) * (D + 4) + 16 * i + 4 * g) = o[t][i];
        __syncthreads();
        for (int e = tid; e < 16 * (D / 4); e += 256) {
            const int hq = e / (D / 4), d = e % (D / 4) * 4;
            if (q0 + 16 * t + hq >= per) continue;
            const float most = fmaxf(fmaxf(top[0][hq], top[1][hq]), fmaxf(top[2][hq], top[3][hq]));
            float total = 0.f;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = exp_above(top[w][hq], most);
                total += f * sum[w][hq];
                v += *reinterpret_cast<const f32x4 *>(red + (w * 16 + hq) * (D + 4) + d) * f;
            }
            if (wrong) {
                total = nan;
                v = f32x4{nan, nan, nan, nan};
            }
            const int64_t row = b * a.q_heads + static_cast<int64_t>(h) * per + q0 + 16 * t + hq;
            if (parts > 1) {
                float *to = a.ws + (row * a.parts + part) * (D + 4);
                put_part(to + d, v[0], v[1], a.join);
                put_part(to + d + 2, v[2], v[3], a.join);
                if (d == 0) put_part(to + D, most, total, a.join);
            } else {
                finish_head(a, row * D + d, row, d, v, most, total);
            }
        }
    }
    if (!a.join || parts <= 1) return;

    // The last of the sequence's parts to finish joins them all: each
    // workgroup counts itself once its stores have arrived, and the one that
    // finds all others counted reads them.  The parts are stored and read past
    // the dies' own caches, so waiting for the stores is all the order needed (a
    // fence of device scope writes back a die's whole L2: with one in every
    // workgroup 32 sequences of up to 16384 tokens took 724 us instead of 234).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
        uint32_t *counter = a.counters + b * hh + hc;
        is_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                  static_cast<uint32_t>(parts);
        if (is_last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!is_last) return;
    const int heads = per - q0 < 16 * QT ? per - q0 : 16 * QT;
    for (int e = tid; e < heads * (D / 4); e += 256) {
        const int d = e % (D / 4) * 4;
        const int64_t row = b * a.q_heads + static_cast<int64_t>(h) * per + q0 + e / (D / 4);
        const float *from = a.ws + row * a.parts * (D + 4);
        float most = kLowest, total = 0.f;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int p = 0; p < parts; ++p) most = fmaxf(most, get_part(from + p * (D + 4) + D).x);
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float *x = from + p * (D + 4);
            const float2 ml = get_part(x + D), lo = get_part(x + d), hi = get_part(x + d + 2);
            const float f = exp_above(ml.x, most);
            total += ml.y * f;
            v += f32x4{lo.x, lo.y, hi.x, hi.y} * f;
        }
        finish_head(a, row * D + d, row, d, v, most, total);
    }
}

// Joins the parts of one sequence's head: D / 4 threads over the elements,
// the rest over the parts.
template <int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int COLS = D / 4, SLICES = 256 / COLS;
    __shared__ float red[SLICES][D + 4], peak[4];
    const int64_t row = blockIdx.x;
    const int parts = parts_of(a, a.lengths[row / a.q_heads]);
    if (parts <= 1) return;  // written by its only part
    const float *from = a.ws + row * a.parts * (D + 4);
    const int tid = threadIdx.x;
    float most = kLowest;
    for (int p = tid; p < parts; p += 256) most = fmaxf(most, from[p * (D + 4) + D]);
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor(most, x, 64));
    if ((tid & 63) == 0) peak[tid >> 6] = most;
    __syncthreads();
    most = fmaxf(fmaxf(peak[0], peak[1]), fmaxf(peak[2], peak[3]));
    const int slice = tid / COLS, d = tid % COLS * 4;
    if (slice < SLICES) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        float total = 0.f;
        for (int p = slice; p < parts; p += SLICES) {
            const float *x = from + static_cast<int64_t>(p) * (D + 4);
            const float f = exp_above(x[D], most);
            v += *reinterpret_cast<const f32x4 *>(x + d) * f;
            total += x[D + 1] * f;
        }
        *reinterpret_cast<f32x4 *>(&red[slice][d]) = v;
        if (d == 0) red[slice][D] = total;
    }
    __syncthreads();
    if (tid >= COLS) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
#pragma unroll
    for (int s = 0; s < SLICES; ++s) {
        v += *reinterpret_cast<const f32x4 *>(&red[s][d]);
        total += red[s][D];
    }
    finish_head(a, row * D + d, row, d, v, most, total);
}

// Instantiated here: the launchers below are compiled for the host only.
#define PROJ_ATTEND_QT(D, QT)                                              \
    template __global__ void attend_kernel<D, false, QT, false>(AttendArgs); \
    template __global__ void attend_kernel<D, true, QT, false>(AttendArgs);  \
    template __global__ void attend_kernel<D, false, QT, true>(AttendArgs);  \
    template __global__ void attend_kernel<D, true, QT, true>(AttendArgs);
#define PROJ_ATTEND_INST(D) \
    PROJ_ATTEND_QT(D, 1)    \
    template __global__ void attend_join_kernel<D>(AttendArgs);
#define PROJ_ATTEND_INST2(D) \
    PROJ_ATTEND_INST(D)      \
    PROJ_ATTEND_QT(D, 2)
PROJ_ATTEND_INST2(64)
PROJ_ATTEND_INST2(80)
PROJ_ATTEND_INST2(96)
PROJ_ATTEND_INST2(128)
PROJ_ATTEND_INST(192)
PROJ_ATTEND_INST(256)

#ifndef __HIP_DEVICE_COMPILE__
bool attend_dim(int dim) {
    return dim == 64 || dim == 80 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

template <int D>
static hipError_t launch_attend_dim(AttendArgs a, hipStream_t st) {
    // two tiles of 16 query heads to a workgroup where their outputs fit its
    // registers; else another workgroup reads the same keys and values
    constexpr bool kTwo = D <= 128;
    const int per = a.q_heads / a.c.heads, qt = kTwo && per > 16 ? 2 : 1;
    a.chunks = (per + 16 * qt - 1) / (16 * qt);
    const int64_t hh = static_cast<int64_t>(a.c.heads) * a.chunks, rows = a.B * hh, most_rows = most_groups(256) - 7 * hh;
    if (a.B > 1 && (rows > most_rows || a.B * a.q_heads > most_groups(256))) {
        // more than one launch can have workgroups for: half the sequences at a time
        AttendArgs x = a, y = a;
        x.B = a.B / 2;
        y.B = a.B - x.B;
        y.q = a.q + x.B * a.q_stride;
        y.tables = a.tables + x.B * a.table_stride;
        y.lengths = a.lengths + x.B;
        const int64_t heads = x.B * a.q_heads;
        y.out = static_cast<char *>(a.out) + heads * D * (a.out_dtype == OUT_F32 ? 4 : 2);
        y.lse = a.lse ? a.lse + heads : nullptr;
        const hipError_t e = launch_attend_dim<D>(x, st);
        return e != hipSuccess ? e : launch_attend_dim<D>(y, st);
    }
    const int64_t span = a.window > 0 && a.window < a.max_len ? a.window : a.max_len;
    // Parts of the length: enough workgroups for four to a compute unit, none
    // shorter than one tile for each wave, and none so long that units idle at
    // the end where lengths differ.  One sequence has parts of one length: all
    // of its workgroups (two to a unit) run at once.
    const int64_t want = (a.B == 1 ? 2 : 4) * static_cast<int64_t>(a.cus), most = a.B == 1 ? kChunk : kChunk / 2;
    int64_t part = (span * rows + want - 1) / want;
    part = part < 128 ? 128 : part > most ? most : (part + 127) / 128 * 128;
    int64_t parts = span > part ? (span + part - 1) / part : 1;
    // no more than the workspace holds and one launch can have
    const int64_t held = static_cast<int64_t>(a.ws_bytes / (sizeof(float) * (D + 4))) / (a.B * a.q_heads);
    const int64_t room = held < most_rows / rows ? held : most_rows / rows;
    if (parts > 1 && parts > room) {
        parts = room < 1 ? 1 : room;
        part = ((span + parts - 1) / parts + 127) / 128 * 128;
        parts = span > part ? (span + part - 1) / part : 1;
    }
    if (parts == 1) part = span > 0 ? span : 1;
    a.part = part;
    a.parts = static_cast<int>(parts);
    // few parts are joined by the last workgroup; for many, one workgroup to
    // each sequence's head is faster and the launch is hidden by the first kernel
    a.join = parts > 1 && parts <= kJoined && rows <= a.ncounters;
    // Heads between a head's tokens (token-major pages): neighbouring heads'
    // rows may share 128-byte lines
    const int64_t size = a.c.fp8 ? 1 : 2;
    const bool mixed = a.c.kt != D || a.c.vt != D;
    const bool once = !mixed || (D * size % 128 == 0 && (a.c.kt | a.c.vt | a.c.kh | a.c.vh) * size % 128 == 0 &&
                                 (reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v)) % 128 == 0);
    a.by_die = mixed && a.B * parts >= 8;
    const int64_t grid = a.by_die ? (a.B * parts + 7) / 8 * 8 * hh : rows * parts;
    auto pick = [&](auto two) {
        constexpr int QT = decltype(two)::value;
        if (a.c.fp8) return once ? attend_kernel<D, true, QT, true> : attend_kernel<D, true, QT, false>;
        return once ? attend_kernel<D, false, QT, true> : attend_kernel<D, false, QT, false>;
    };
    auto kernel = pick(std::integral_constant<int, 1>());
    if constexpr (kTwo)
        if (qt == 2) kernel = pick(std::integral_constant<int, 2>());
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1 || a.join) return e;
    hipLaunchKernelGGL((attend_join_kernel<D>), dim3(static_cast<unsigned>(a.B * a.q_heads)), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_attend(const AttendArgs &a, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_attend_dim<64>(a, st);
        case 80: return launch_attend_dim<80>(a, st);
        case 96: return launch_attend_dim<96>(a, st);
        case 128: return launch_attend_dim<128>(a, st);
        case 192: return launch_attend_dim<192>(a, st);
        case 256: return launch_attend_dim<256>(a, st);
    }
    return hipErrorInvalidValue;
}
#endif

}  // namespace proj
