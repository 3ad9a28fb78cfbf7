// int8.hip -- projection of 8-bit integers with a scale for each token and
// each output, and the making of such integers from bf16 rows.
//
//     Y[m, n] = epilogue(x_scales[m] w_scales[n] sum_k X[m, k] W[n, k] (+ bias[n]))
//
// The sum is exact (32-bit integers); it meets the scales in 64-bit floating
// point, so that their product neither overflows nor vanishes on its way and
// the result before bias and GELU is the rounded one.
#include "layer.hpp"

namespace proj {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------ rows to integers
//
// scale = max |x| / 127 and q = rint(127 x / max |x|). With x = X 2^a and max |x| =
// A 2^b, X and A integers below 2^8, the quotient is n + 1/2 exactly or off it by
// 1 / (A 2^(b - a)) or more, 2^-16 of its size. So x times the fp32 quotient
// 127 / max |x|, which is off by 2^-23, rounded to 19 bits, is n + 1/2 exactly where
// the quotient is and on the same side of it where it is not: q is the exact one
// without a division for each element.
struct RowScale {
    float up, per, scale;  // x * up * per is the quotient; up is 1 unless the row is very small
    __device__ __forceinline__ explicit RowScale(uint32_t top) {  // bits of max |x|
        const float most = __uint_as_float(top << 16);
        up = most < 0x1p-64f ? 0x1p64f : 1.f;
        const bool numbers = top < 0x7f80u;  // neither infinity nor NaN
        per = top == 0 || !numbers ? 0.f : 127.f / (most * up);
        scale = numbers ? most / 127.f : __builtin_nanf("");
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t bits) const {  // the integer's byte
        const float y = __uint_as_float(bits << 16) * up * per;
        const float z = __uint_as_float((__float_as_uint(y) + 16u) & ~31u);
        // the integer nearest to z in the low bits; a NaN's place (its row's scale is NaN) is 0
        return per == 0.f ? 0u : __float_as_uint(z + 0x1.8p23f) & 0xffu;
    }
};

// Largest |x| of eight, as bits, two at a time.
__device__ __forceinline__ u16x2 most8(u16x2 top, u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    return top;
}

// One workgroup to a row, one element at a time.
__global__ __launch_bounds__(256) void quantize_rows_kernel(RowsArgs a) {
    __shared__ uint32_t peak[4];
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const uint16_t *x = a.X + m * a.stride;
        uint32_t top = 0;
        for (int64_t k = threadIdx.x; k < a.K; k += 256) top = max(top, static_cast<uint32_t>(x[k] & 0x7fff));
        for (int h = 32; h >= 1; h >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), h, 64)));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) peak[threadIdx.x >> 6] = top;
        __syncthreads();
        const RowScale s(max(max(peak[0], peak[1]), max(peak[2], peak[3])));
        for (int64_t k = threadIdx.x; k < a.q_stride; k += 256)
            a.q[m * a.q_stride + k] = static_cast<int8_t>(k < a.K ? s(x[k]) : 0u);
        if (threadIdx.x == 0) a.scales[m] = s.scale;
    }
}

// ------------------------------------------------------------------- product

__device__ __forceinline__ i32x4 mfma16x16x64(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// One output before bias and GELU.
__device__ __forceinline__ float scaled(int32_t sum, float xs, float ws) {
    return static_cast<float>(static_cast<double>(sum) * (static_cast<double>(xs) * ws));
}

// 16 x 16 outputs to a wave, operands straight from memory.
__global__ __launch_bounds__(256) void int_wave_kernel(IntArgs a) {
    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
    const int64_t tn = (a.N + 15) / 16, tiles = tn * ((a.M + 15) / 16);
    for (int64_t tile = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); tile < tiles;
         tile += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t m = tile / tn * 16 + c16, n = tile % tn * 16 + c16;
        const int8_t *x = a.X + (m < a.M ? m : a.M - 1) * a.K, *w = a.W + (n < a.N ? n : a.N - 1) * a.K;
        i32x4 acc = {0, 0, 0, 0};
        for (int64_t k = 0; k < a.K; k += 64) {
            i32x4 xv = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
            if (k + 16 * g < a.K) {
                xv = *reinterpret_cast<const i32x4 *>(x + k + 16 * g);
                wv = *reinterpret_cast<const i32x4 *>(w + k + 16 * g);
            }
            acc = mfma16x16x64(wv, xv, acc);
        }
        if (m >= a.M) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t col = tile % tn * 16 + 4 * g + r;
            if (col >= a.N) continue;
            const float b = (a.epi & 1) ? bf16_bits_to_f32(a.bias[col]) : 0.f;
            const float s = a.K > 0 ? scaled(acc[r], a.x_scales[m], a.w_scales[col]) : 0.f;
            store_out(a.Y, a.out, m * a.N + col, apply_epilogue(s, a.epi, b));
        }
    }
}

#ifndef __HIP_DEVICE_COMPILE__
hipError_t launch_quantize_rows(const RowsArgs &a, hipStream_t st) {
    const int64_t most = most_groups(256);
    hipLaunchKernelGGL(quantize_rows_kernel, dim3(static_cast<unsigned>(a.M < most ? a.M : most)), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_int(const IntArgs &a, hipStream_t st) {
    const int64_t tiles = (a.N + 15) / 16 * ((a.M + 15) / 16), most = most_groups(256), groups = (tiles + 3) / 4;
    hipLaunchKernelGGL(int_wave_kernel, dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(256), 0, st, a);
    return hipGetLastError();
}
#endif

}  // namespace proj
