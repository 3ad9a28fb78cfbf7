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

struct RowMean {
    float most, total;  // m and l
    float mean;         // element threadIdx.x of o / l, for threads below D
};

constexpr int kRowMeanLds = 256 * 16 + 16;  // bytes of LDS that row_mean needs, 8-byte aligned

// One row over tokens first .. last - 1 of a list of pages, by a workgroup of 256
// threads: a token to a thread for its logit, an element to a thread for the sums. A
// value whose probability vanishes even in 64 bits counts only where it is infinite or
// no number. For rows that are not finite otherwise: every logit is worked out twice,
// from memory. q: the row's D elements; h: its key-value head; scale: of <q, k> as
// stored.
template <int D, bool FP8>
__device__ __forceinline__ RowMean row_mean(const CacheArgs &c, const int32_t *pages, const uint16_t *q, int h, int64_t first,
                                            int64_t last, double scale, char *lds) {
    double *prob = reinterpret_cast<double *>(lds);
    int64_t *place = reinterpret_cast<int64_t *>(lds + 256 * 8);
    float *peak = reinterpret_cast<float *>(lds + 256 * 16);
    const int tid = threadIdx.x;
    const int64_t place_mask = (int64_t{1} << c.page_shift) - 1;
    auto page_of = [&](int64_t t) -> int64_t {
        const int32_t p = pages[t >> c.page_shift];
        return p >= 0 && p < c.pages ? p : 0;  // the caller has seen that all are inside
    };
    auto logit = [&](int64_t t) {
        const int64_t at = page_of(t) * c.kp + h * c.kh + (t & place_mask) * c.kt;
        float dot = 0.f;
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
            float k[16];
            if constexpr (FP8) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(c.k) + at + 16 * i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    k[4 * e] = __builtin_amdgcn_cvt_f32_fp8(w[e], 0);
                    k[4 * e + 1] = __builtin_amdgcn_cvt_f32_fp8(w[e], 1);
                    k[4 * e + 2] = __builtin_amdgcn_cvt_f32_fp8(w[e], 2);
                    k[4 * e + 3] = __builtin_amdgcn_cvt_f32_fp8(w[e], 3);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) k[e] = bf16_bits_to_f32(static_cast<const uint16_t *>(c.k)[at + 16 * i + e]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) dot = __builtin_fmaf(bf16_bits_to_f32(q[16 * i + e]), k[e], dot);
        }
        return dot * scale;
    };
    float most = -0x1.fffffep127f;
    for (int64_t t = first + tid; t < last; t += 256) most = fmaxf(most, static_cast<float>(logit(t)));
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor(most, x, 64));
    __syncthreads();
    if ((tid & 63) == 0) peak[tid >> 6] = most;
    __syncthreads();
    most = fmaxf(fmaxf(peak[0], peak[1]), fmaxf(peak[2], peak[3]));
    double total = 0., sum = 0.;
    for (int64_t base = first; base < last; base += 256) {
        const int n = static_cast<int>(last - base < 256 ? last - base : 256);
        __syncthreads();  // the probabilities before are done with
        if (tid < n) {
            const double w = logit(base + tid), p = exp(w - most);
            prob[tid] = p == 0. && w > -__builtin_inf() ? 0x1p-1074 : p;
            place[tid] = page_of(base + tid) * c.vp + h * c.vh + ((base + tid) & place_mask) * c.vt;
        }
        __syncthreads();
        if (tid < D)
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const double p = prob[i];
                const float v = FP8 ? __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t *>(c.v)[place[i] + tid], 0)
                                    : bf16_bits_to_f32(static_cast<const uint16_t *>(c.v)[place[i] + tid]);
                total += p;
                sum += p != 0. ? p * v : 0.;
            }
    }
    __syncthreads();  // the row behind uses the same memory
    if (tid == 0) peak[0] = static_cast<float>(total);
    __syncthreads();
    return RowMean{most, peak[0], total == 0. ? 0.f : static_cast<float>(sum / total)};
}

}  // namespace proj
