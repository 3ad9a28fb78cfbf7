// quant.hip -- projection with 4-bit weights and group scales, and the
// layout and making of such weights.
//
//     Y[m, n] = sum_g s[n, g] * (sum_{k in g} X[m, k] c[n, k] - z[n, g] sum_{k in g} X[m, k])
#include "decode.hpp"

namespace proj {

// Bit position of code j of a word of eight.
__host__ __device__ constexpr int code_shift(int j) { return 4 * (j / 2) + 16 * (j % 2); }

__device__ __forceinline__ float group_scale(const QuantArgs &a, int64_t i) {
    return a.scales_f32 ? static_cast<const float *>(a.scales)[i]
                        : bf16_bits_to_f32(static_cast<const uint16_t *>(a.scales)[i]);
}

// Any K (a multiple of 8) and alignment: one wave per output, lane l taking
// words l, l + 64, ... of the row.  A word lies within one group.
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (idx >= a.M * a.N) return;
    const int64_t m = idx / a.N, n = idx % a.N, words = a.K / 8;
    float acc = 0.f;
    for (int64_t w = lane; w < words; w += 64) {
        const uint32_t word = a.codes[n * words + w];
        const int64_t g = n * a.G + w * 8 / a.group;
        const float z = a.zeros ? static_cast<float>(a.zeros[g]) : 8.f;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = static_cast<float>((word >> code_shift(j)) & 15u);
            s = __builtin_fmaf(bf16_bits_to_f32(a.X[m * a.K + w * 8 + j]), c - z, s);
        }
        acc = __builtin_fmaf(s, group_scale(a, g), acc);
    }
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) acc += __shfl_xor(acc, h, 64);
    if (lane == 0) {
        const float b = (a.epi & 1) ? bf16_bits_to_f32(a.bias[n]) : 0.f;
        store_out(a.Y, a.out, idx, apply_epilogue(acc, a.epi, b));
    }
}

__global__ __launch_bounds__(256) void pack_codes_kernel(const uint8_t *q, int64_t words, uint32_t *codes) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= words) return;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) w |= static_cast<uint32_t>(q[i * 8 + j] & 15) << code_shift(j);
    codes[i] = w;
}

// One wave per group of a row: the group's extremes, then its codes.  Lane l
// holds words l of the group (16 words at most); a word is eight weights.
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t *W, int64_t N, int64_t K, int64_t G, int group,
                                                       uint32_t *codes, void *scales, int scales_f32, uint8_t *zeros) {
    const int lane = threadIdx.x & 63;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (idx >= N * G) return;
    const int64_t n = idx / G, k = (idx % G) * group + lane * 8;
    const bool live = lane * 8 < group && k < K;
    float w[8], lo = 0.f, hi = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = live ? bf16_bits_to_f32(W[n * K + k + j]) : 0.f;
        lo = fminf(lo, w[j]);
        hi = fmaxf(hi, w[j]);
    }
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, h, 64));
        hi = fmaxf(hi, __shfl_xor(hi, h, 64));
    }
    float s = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
    if (!scales_f32) s = bf16_bits_to_f32(f32_to_bf16_bits(s));
    const float z = !zeros ? 8.f : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
    if (lane == 0) {
        if (scales_f32)
            static_cast<float *>(scales)[idx] = s;
        else
            static_cast<uint16_t *>(scales)[idx] = f32_to_bf16_bits(s);
        if (zeros) zeros[idx] = static_cast<uint8_t>(z);
    }
    if (!live) return;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float c = s > 0.f ? fminf(fmaxf(rintf(w[j] / s) + z, 0.f), 15.f) : z;
        word |= static_cast<uint32_t>(c) << code_shift(j);
    }
    codes[(n * K + k) / 8] = word;
}

#ifndef __HIP_DEVICE_COMPILE__
static bool grid_for(int64_t items, int64_t per, unsigned *grid) {
    const int64_t g = (items + per - 1) / per;
    if (g <= 0 || g > 0x7fffffff) return false;
    *grid = static_cast<unsigned>(g);
    return true;
}

hipError_t launch_quant(const QuantArgs &a, hipStream_t st) {
    unsigned grid;
    if (!grid_for(a.M * a.N, 4, &grid)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(quant_rows_kernel, dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_pack_codes(const uint8_t *q, int64_t N, int64_t K, uint32_t *codes, hipStream_t st) {
    unsigned grid;
    if (!grid_for(N * K / 8, 256, &grid)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(pack_codes_kernel, dim3(grid), dim3(256), 0, st, q, N * K / 8, codes);
    return hipGetLastError();
}

hipError_t launch_quantize(const uint16_t *W, int64_t N, int64_t K, int group, uint32_t *codes, void *scales,
                           int scales_f32, uint8_t *zeros, hipStream_t st) {
    const int64_t G = (K + group - 1) / group;
    unsigned grid;
    if (!grid_for(N * G, 4, &grid)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(quantize_kernel, dim3(grid), dim3(256), 0, st, W, N, K, G, group, codes, scales, scales_f32,
                       zeros);
    return hipGetLastError();
}
#endif

}  // namespace proj
