// decode.hpp -- launchers of the decoding operators: 4-bit weights
// (quant.hip) and the paged key-value cache (kvcache.hip, attend.hip).
#pragma once

#include "common.hpp"

namespace proj {

// Workgroups that one launch may have: HIP takes less than 2^32 threads and 2^31 workgroups.
constexpr int64_t most_groups(int threads) {
    return 0xffffffffll / threads < 0x7fffffff ? 0xffffffffll / threads : 0x7fffffff;
}

// One call of the 4-bit projection.
struct QuantArgs {
    const uint16_t *X;      // bf16 [M, K]
    const uint32_t *codes;  // [N, K / 8]
    const void *scales;     // bf16 or fp32 [N, G]
    const uint8_t *zeros;   // [N, G] or nullptr (8)
    const uint16_t *bias;   // bf16 [N] or nullptr
    void *Y;                // fp32 / bf16 [M, N]
    int64_t M, N, K, G;     // G = ceil(K / group)
    int group, scales_f32, epi, out;
    float *ws;              // split-K partials
    size_t ws_bytes;
    int cus;
    int vec_scales = 0;     // set by the launcher: scales and zeros start at 16-byte boundaries
};
hipError_t launch_quant(const QuantArgs &a, hipStream_t st);

// q [N][K], one code to a byte -> words of eight.
hipError_t launch_pack_codes(const uint8_t *q, int64_t N, int64_t K, uint32_t *codes, hipStream_t st);

// bf16 W [N][K] -> codes, scales and (where not null) zeros.
hipError_t launch_quantize(const uint16_t *W, int64_t N, int64_t K, int group, uint32_t *codes, void *scales,
                           int scales_f32, uint8_t *zeros, hipStream_t st);

// The cache as kernels see it (strides in elements: page, head, token).
struct CacheArgs {
    void *k, *v;
    int64_t kp, kh, kt, vp, vh, vt;
    int64_t pages;
    int fp8, heads, dim, page_shift;
    float k_scale, v_scale;
};

struct AppendArgs {
    CacheArgs c;
    const uint16_t *qkv;
    int64_t stride, T;
    int q_heads, rot, interleaved;
    const float *rope;
    int64_t rope_rows;
    const int32_t *positions;
    const int64_t *slots;
    uint16_t *q_out;
};
hipError_t launch_append(const AppendArgs &a, hipStream_t st);

struct AttendArgs {
    CacheArgs c;
    const uint16_t *q;
    int64_t q_stride, B;
    int q_heads;
    const int32_t *tables;
    int64_t table_stride;
    const int32_t *lengths;
    int64_t max_len, window;
    float scale;
    void *out;
    int out_dtype;
    float *lse;
    float *ws;
    size_t ws_bytes;
    int cus;
    uint32_t *counters = nullptr;  // zero between calls
    int ncounters = 0;
    // set by the launcher: tokens of a part, parts of the longest sequence,
    // chunks of a key-value head's query heads, whether a sequence's last
    // workgroup to finish joins its parts, whether a part's heads go to one die
    int64_t part = 0;
    int parts = 0, chunks = 0, join = 0, by_die = 0;
};
hipError_t launch_attend(const AttendArgs &a, hipStream_t st);
bool attend_dim(int dim);  // whether a kernel for this head size is built

}  // namespace proj
