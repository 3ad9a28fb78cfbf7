// parts.hpp -- the parts of a row of attention (attend.hip, prefix.hip) where a
// sum passes the largest float.
//
// A part of a row over some of its tokens lies in the workspace as head_dim + 4
// floats: the sums o = sum_t exp(w[t] - m) v[t], then m and l = sum_t exp(w[t] - m).
// The result, the mean o / l, is no larger than the largest value, but o is up to l
// times that (m lags the true maximum by up to 5, and tokens are many), so with
// values near the largest float it may be infinite, or NaN, where the result is not.
// Such a row is worked out again in 64 bits, and its part holds the mean instead of
// the sums, with l negative as the sign of it. The joins add shares of means where
// they meet one, or where their own sum is not finite.
#pragma once

#include "decode.hpp"

namespace proj {

// Whether sums are not finite though their probabilities are numbers (infinity times 0 is NaN).
__device__ __forceinline__ bool past_largest(f32x4 v, float total) {
    const float z = v[0] * 0.f + v[1] * 0.f + v[2] * 0.f + v[3] * 0.f;
    return z != z && total == total;
}

// A row to work out again: its query of D elements, and the tokens first .. last - 1 that it sees.
struct RowAgain {
    const uint16_t *q;
    int64_t first, last;
};
struct RowMean {
    float most, total;  // m and l
    float mean;         // an element of o / l
};

constexpr int kRowsAgain = 8, kTokensAgain = 192;  // rows, and tokens with their probabilities in LDS, at a time
// bytes of LDS that rows_again needs, 16-byte aligned
constexpr int rows_again_lds(int D) { return (kRowsAgain + 1) * kTokensAgain * 8 + kRowsAgain * (4 * 4 + 2 * 8 + D * 4) + 128 * 4; }

// The marked ones (bit x % 32 of marks[x / 32], `words` of them, at most 4) of the rows
// of key-value head h over a list of pages, by a workgroup of 256 threads: a token to a
// thread for the logits, an element of all 8 rows that are taken at a time, or of half
// of them, to a thread for the sums. row(x) gives a RowAgain; put(x, d, mean) takes
// element d (m and l are the same for all of them). A value whose probability vanishes
// even in 64 bits counts only where it is infinite or no number. scale: of <q, k> as
// stored. Every logit is worked out twice, and everything comes from memory: only for
// rows that are not finite otherwise. Eight rows with 512 tokens of 128 elements take a
// workgroup about 100 us: every row of 64 sequences behind 8192 tokens 2.4 ms where sums
// do it in 0.08.
template <int D, bool FP8, class Row, class Put>
__device__ __forceinline__ void rows_again(const CacheArgs &c, const int32_t *pages, int h, double scale, const uint32_t *marks,
                                           int words, char *lds, Row row, Put put) {
    typedef __attribute__((__vector_size__(2 * sizeof(double)))) double f64x2;
    constexpr int R = kRowsAgain, TOK = kTokensAgain;
    double *prob = reinterpret_cast<double *>(lds);                   // [TOK][R]
    int64_t *place = reinterpret_cast<int64_t *>(prob + R * TOK);     // [TOK]
    float *part = reinterpret_cast<float *>(place + TOK);             // [R][4], of the waves
    int64_t *range = reinterpret_cast<int64_t *>(part + R * 4);       // [R][2], first and last
    float *query = reinterpret_cast<float *>(range + R * 2);          // [R][D]
    int *list = reinterpret_cast<int *>(query + R * D);               // [128]
    const int tid = threadIdx.x, wave = tid >> 6;
    int count = 0, before = 0;
    for (int i = 0; i < words; ++i) {
        if (i == tid / 32) before = count + __popc(marks[i] & ((1u << tid % 32) - 1));
        count += __popc(marks[i]);
    }
    count = __builtin_amdgcn_readfirstlane(count);
    if (tid / 32 < words && (marks[tid / 32] >> tid % 32 & 1)) list[before] = tid;
    const int64_t place_mask = (int64_t{1} << c.page_shift) - 1;
    auto page_of = [&](int64_t t) -> int64_t {
        const int32_t p = pages[t >> c.page_shift];
        return p >= 0 && p < c.pages ? p : 0;  // the caller has seen that all are inside
    };
    auto logits = [&](int64_t t, float (&w)[R]) {
        const int64_t at = page_of(t) * c.kp + h * c.kh + (t & place_mask) * c.kt;
#pragma unroll
        for (int i = 0; i < R; ++i) w[i] = 0.f;
        constexpr int LOADS = FP8 ? 1 : 2;  // 16-byte loads of 16 elements; those of the next are on their way
        const u32x4 *from = reinterpret_cast<const u32x4 *>(static_cast<const char *>(c.k) + (FP8 ? at : 2 * at));
        u32x4 next[LOADS];
#pragma unroll
        for (int v = 0; v < LOADS; ++v) next[v] = from[v];
#pragma unroll 1
        for (int d = 0; d < D; d += 16) {
            float k[16];
#pragma unroll
            for (int v = 0; v < LOADS; ++v)
#pragma unroll
                for (int e = 0; e < 16 / LOADS; ++e) {
                    const uint32_t w = next[v][e * (FP8 ? 1 : 2) / 4];
                    if constexpr (FP8)
                        k[e] = __builtin_amdgcn_cvt_f32_fp8(w >> (8 * (e % 4)), 0);
                    else
                        k[8 * v + e] = __uint_as_float(e % 2 ? w & 0xffff0000u : w << 16);
                }
            if (d + 16 < D)
#pragma unroll
                for (int v = 0; v < LOADS; ++v) next[v] = from[(d / 16 + 1) * LOADS + v];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f32x4 q = *reinterpret_cast<const f32x4 *>(query + i * D + d + e);
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[i] = __builtin_fmaf(q[x], k[e + x], w[i]);
                }
                __builtin_amdgcn_sched_barrier(0);  // not all rows' reads first: this is to take few registers
            }
        }
        // where a row sees the token
#pragma unroll
        for (int i = 0; i < R; ++i)
            w[i] = t >= range[2 * i] && t < range[2 * i + 1] ? static_cast<float>(w[i] * scale) : -__builtin_inff();
    };
    for (int x0 = 0; x0 < count; x0 += R) {
        __syncthreads();
        {
            const int i = tid / 32;
            const RowAgain r = row(list[x0 + i < count ? x0 + i : x0]);
            if (tid % 32 == 0) {
                range[2 * i] = r.first;
                range[2 * i + 1] = r.last;
            }
            for (int d = tid % 32; d < D; d += 32) query[i * D + d] = bf16_bits_to_f32(r.q[d]);
        }
        __syncthreads();
        int64_t first = range[0], last = range[1];
        for (int i = 1; i < R; ++i) {
            first = range[2 * i] < first ? range[2 * i] : first;
            last = range[2 * i + 1] > last ? range[2 * i + 1] : last;
        }
        float most[R];
#pragma unroll
        for (int i = 0; i < R; ++i) most[i] = -0x1.fffffep127f;
#pragma unroll 1
        for (int64_t t = first + tid; t < last; t += 256) {
            float w[R];
            logits(t, w);
#pragma unroll
            for (int i = 0; i < R; ++i) most[i] = fmaxf(most[i], w[i]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll 1
            for (int x = 32; x >= 1; x >>= 1) most[i] = fmaxf(most[i], __shfl_xor(most[i], x, 64));
            if ((tid & 63) == 0) part[4 * i + wave] = most[i];
        }
        __syncthreads();
        auto top = [&](int i) { return fmaxf(fmaxf(part[4 * i], part[4 * i + 1]), fmaxf(part[4 * i + 2], part[4 * i + 3])); };
        constexpr int HALVES = D <= 128 ? 2 : 1, ROWS = R / HALVES;  // of the threads, and their rows
        const int d = HALVES == 2 ? tid % 128 : tid, row0 = HALVES == 2 ? tid / 128 * ROWS : 0;
        double total[ROWS], sum[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) total[i] = sum[i] = 0.;
#pragma unroll 1
        for (int64_t base = first; base < last; base += TOK) {
            const int n = static_cast<int>(last - base < TOK ? last - base : TOK);
            __syncthreads();  // the probabilities before are done with
            if (tid < n) {
                float w[R];
                logits(base + tid, w);
#pragma unroll
                for (int i = 0; i < R; ++i) prob[tid * R + i] = w[i];
                place[tid] = page_of(base + tid) * c.vp + h * c.vh + ((base + tid) & place_mask) * c.vt;
#pragma unroll 1
                for (int i = 0; i < R; ++i) {
                    const double x = prob[tid * R + i], p = exp(x - top(i));
                    prob[tid * R + i] = p == 0. && x > -__builtin_inf() ? 0x1p-1074 : p;
                }
            }
            __syncthreads();
            if (d < D)
#pragma unroll 1
                for (int t0 = 0; t0 < n; t0 += 8) {
                    float v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int64_t at = place[t0 + x < n ? t0 + x : n - 1] + d;
                        v[x] = FP8 ? __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t *>(c.v)[at], 0)
                                   : bf16_bits_to_f32(static_cast<const uint16_t *>(c.v)[at]);
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        if (t0 + x >= n) break;
#pragma unroll
                        for (int i = 0; i < ROWS; i += 2) {
                            const f64x2 p = *reinterpret_cast<const f64x2 *>(prob + (t0 + x) * R + row0 + i);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                total[i + y] += p[y];
                                sum[i + y] += p[y] != 0. ? p[y] * v[x] : 0.;
                            }
                        }
                        if (x % 2) __builtin_amdgcn_sched_barrier(0);
                    }
                }
        }
        if (d < D)
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (x0 + row0 + i < count)
                    put(list[x0 + row0 + i], d, RowMean{top(row0 + i), static_cast<float>(total[i]),
                                                        total[i] == 0. ? 0.f : static_cast<float>(sum[i] / total[i])});
    }
}

}  // namespace proj
