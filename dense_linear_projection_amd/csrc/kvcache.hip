// kvcache.hip -- the paged key-value cache of a decoding step: rotary
// positions and the storing of keys and values (append), and attention of
// one new token for each sequence over its pages (attend).
#include "decode.hpp"

namespace proj {

// fp32 -> e4m3 bits (to nearest even), clamped to the largest finite value
// first: the conversion itself has no infinity to saturate to.  NaN stays.
__device__ __forceinline__ uint8_t f32_to_fp8_bits(float v) {
    const float c = v > 448.f ? 448.f : v < -448.f ? -448.f : v;
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false) & 0xff);
}

__device__ __forceinline__ float fp8_bits_to_f32(uint8_t b) {
    return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(b), 0);
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

__device__ __forceinline__ float cache_value(const CacheArgs &c, const void *base, int64_t i) {
    return c.fp8 ? fp8_bits_to_f32(static_cast<const uint8_t *>(base)[i])
                 : bf16_bits_to_f32(static_cast<const uint16_t *>(base)[i]);
}

// One workgroup per sequence and query head.  Wave w takes tokens w, w + 4,
// ... with its lanes over the head's elements, and keeps the running maximum
// and sum of a softmax; the four waves join at the end.
__global__ __launch_bounds__(256) void attend_rows_kernel(AttendArgs a) {
    constexpr int PER = 4;  // elements of a head to a lane: up to 256
    __shared__ float part[4][64 * PER], top[4], sum[4];
    __shared__ int wrong;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = a.c.dim;
    const int64_t b = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads, h = hq / (a.q_heads / a.c.heads);
    const int64_t n = a.lengths[b];
    if (threadIdx.x == 0) wrong = n < 0 || n > a.max_len;
    __syncthreads();
    const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    const int64_t last = wrong ? first : n;
    float q[PER], o[PER], m = -__builtin_inff(), l = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int d = lane + 64 * i;
        q[i] = d < D ? bf16_bits_to_f32(a.q[b * a.q_stride + hq * D + d]) : 0.f;
        o[i] = 0.f;
    }
    for (int64_t t = first + wave; t < last; t += 4) {
        const int64_t page = a.tables[b * a.table_stride + (t >> a.c.page_shift)];
        const int64_t place = t & ((int64_t{1} << a.c.page_shift) - 1);
        if (page < 0 || page >= a.c.pages) {
            wrong = 1;
            break;
        }
        const int64_t ki = page * a.c.kp + h * a.c.kh + place * a.c.kt, vi = page * a.c.vp + h * a.c.vh + place * a.c.vt;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < D) s = __builtin_fmaf(q[i], cache_value(a.c, a.c.k, ki + lane + 64 * i), s);
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1) s += __shfl_xor(s, x, 64);
        s *= a.scale * a.c.k_scale;
        // a maximum of -infinity (every logit so far) leaves weights of zero
        const float mn = fmaxf(m, s), base = mn == -__builtin_inff() ? 0.f : mn;
        const float old = m == mn ? 1.f : expf(m - base), p = expf(s - base);
        m = mn;
        l = l * old + p;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < D)
                o[i] = __builtin_fmaf(p, cache_value(a.c, a.c.v, vi + lane + 64 * i), o[i] * old);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) part[wave][lane + 64 * i] = o[i];
    if (lane == 0) {
        top[wave] = m;
        sum[wave] = l;
    }
    __syncthreads();
    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    float f[4], all = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[w] = sum[w] == 0.f ? 0.f : expf(top[w] - mx);
        all += f[w] * sum[w];
    }
    const int d = threadIdx.x;
    const float nan = __builtin_nanf("");
    if (d < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v += f[w] == 0.f ? 0.f : f[w] * part[w][d];
        v = all == 0.f ? 0.f : v / all * a.c.v_scale;
        store_out(a.out, a.out_dtype, (b * a.q_heads + hq) * D + d, wrong ? nan : v);
    }
    if (d == 0 && a.lse) a.lse[b * a.q_heads + hq] = wrong ? nan : mx + logf(all);
}

#ifndef __HIP_DEVICE_COMPILE__
hipError_t launch_append(const AppendArgs &a, hipStream_t st) {
    if (a.T > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(append_rows_kernel, dim3(static_cast<unsigned>(a.T)), dim3(256), 0, st, a);
    return hipGetLastError();
}

bool attend_dim(int dim) {
    return dim == 64 || dim == 80 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

hipError_t launch_attend(const AttendArgs &a, hipStream_t st) {
    const int64_t grid = a.B * a.q_heads;
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(attend_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, a);
    return hipGetLastError();
}
#endif

}  // namespace proj
