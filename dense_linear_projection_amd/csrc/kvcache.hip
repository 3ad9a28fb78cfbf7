// kvcache.hip -- rotary positions and the storing of keys and values into a
// paged key-value cache.
#include "decode.hpp"

namespace proj {

// fp32 -> e4m3 bits (to nearest even), clamped to the largest finite value
// first: the conversion itself has no infinity to saturate to.  NaN stays.
__device__ __forceinline__ uint8_t f32_to_fp8_bits(float v) {
    const float c = v > 448.f ? 448.f : v < -448.f ? -448.f : v;
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xff);
}

// Element d of head h of one qkv row, rotated where it belongs to a rotated
// pair: `cs` is the position's row of the table.
__device__ __forceinline__ float rotated(const AppendArgs &a, const uint16_t *x, const float *cs, int d) {
    const float v = bf16_bits_to_f32(x[d]);
    if (d >= a.rot) return v;
    const int half = a.rot / 2;
    const int j = a.interleaved ? d >> 1 : d < half ? d : d - half;
    const bool second = a.interleaved ? (d & 1) != 0 : d >= half;
    const int partner = a.interleaved ? d ^ 1 : second ? d - half : d + half;
    const float u = bf16_bits_to_f32(x[partner]), c = cs[j], s = cs[half + j];
    return second ? v * c + u * s : v * c - u * s;
}

// One workgroup per token, a thread per element.
__global__ __launch_bounds__(256) void append_rows_kernel(AppendArgs a) {
    const int64_t t = blockIdx.x;
    const int D = a.c.dim, Hq = a.q_heads, Hkv = a.c.heads;
    const uint16_t *row = a.qkv + t * a.stride;
    const int64_t pos = a.positions[t], slot = a.slots[t];
    const bool known = a.rot == 0 || (pos >= 0 && pos < a.rope_rows);
    const float *cs = a.rope + (known ? pos : 0) * a.rot;
    if (a.q_out)
        for (int e = threadIdx.x; e < Hq * D; e += 256) {
            const float v = known ? rotated(a, row + e / D * D, cs, e % D) : __builtin_nanf("");
            a.q_out[t * Hq * D + e] = f32_to_bf16_bits(v);
        }
    const int64_t page = slot >> a.c.page_shift, place = slot & ((int64_t{1} << a.c.page_shift) - 1);
    if (!known || slot < 0 || page >= a.c.pages) return;
    for (int e = threadIdx.x; e < 2 * Hkv * D; e += 256) {
        const bool is_v = e >= Hkv * D;
        const int h = e / D - (is_v ? Hkv : 0), d = e % D;
        const uint16_t *x = row + static_cast<int64_t>(Hq) * D + e / D * D;
        const float v = is_v ? bf16_bits_to_f32(x[d]) : rotated(a, x, cs, d);
        const int64_t to = is_v ? page * a.c.vp + h * a.c.vh + place * a.c.vt + d
                                : page * a.c.kp + h * a.c.kh + place * a.c.kt + d;
        void *base = is_v ? a.c.v : a.c.k;
        if (a.c.fp8)
            static_cast<uint8_t *>(base)[to] = f32_to_fp8_bits(v / (is_v ? a.c.v_scale : a.c.k_scale));
        else
            static_cast<uint16_t *>(base)[to] = f32_to_bf16_bits(v);
    }
}

#ifndef __HIP_DEVICE_COMPILE__
hipError_t launch_append(const AppendArgs &a, hipStream_t st) {
    if (a.T > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(append_rows_kernel, dim3(static_cast<unsigned>(a.T)), dim3(256), 0, st, a);
    return hipGetLastError();
}
#endif

}  // namespace proj
