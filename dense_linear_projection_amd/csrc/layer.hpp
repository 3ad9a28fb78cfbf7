// layer.hpp -- launchers of a decoding layer's operators in 8-bit integers
// (int8.hip) and of attention over a prefix that a batch shares (prefix.hip).
#pragma once

#include "decode.hpp"

namespace proj {

// bf16 rows -> 8-bit integers and a scale for each.
struct RowsArgs {
    const uint16_t *X;  // bf16 [M, K], rows `stride` elements apart
    int64_t stride, M, K;
    int8_t *q;          // [M, q_stride], zero behind K
    int64_t q_stride;
    float *scales;      // [M]
};
hipError_t launch_quantize_rows(const RowsArgs &a, hipStream_t st);

// One product of 8-bit integers. K is a multiple of 16, at most kIntMaxK.
struct IntArgs {
    const int8_t *X, *W;              // [M, K], [N, K]
    const float *x_scales, *w_scales; // [M], [N]
    const uint16_t *bias;             // bf16 [N] or nullptr
    void *Y;                          // fp32 / bf16 [M, N], rows `row` elements apart
    int64_t M, N, K, row;
    int epi, out;
    int32_t *ws;                      // sums of a split K
    size_t ws_bytes;
    int cus;
    uint32_t *counters;               // ncounters of them, zero between calls
    int ncounters;
    const uint16_t *rows = nullptr;   // fused: the tokens in bf16 [M, rows_k], rows_stride elements apart, instead of X
    int64_t rows_stride = 0, rows_k = 0;
};
// the largest K whose sum of products of 8-bit integers, each at most 2^14, stays below 2^31
constexpr int64_t kIntMaxK = (int64_t{1} << 17) - 16;
hipError_t launch_int(const IntArgs &a, hipStream_t st);
// Whether the product takes so few tokens (K rounded up) in bf16, and that product: `rows` instead of X and x_scales.
bool int_fuses(int64_t M, int64_t N, int64_t K);
hipError_t launch_int_fused(const IntArgs &a, hipStream_t st);

// Attention of one new token for each sequence behind a shared prefix: `a` with
// a.prefix tokens in the pages of `pages`. hipErrorOutOfMemory (and nothing
// launched) where the workspace does not hold two parts of one sequence.
struct PrefixArgs {
    AttendArgs a;
    const int32_t *pages;
    // set by the launcher: tokens of a part, groups of rows that one workgroup takes
    int64_t part = 0;
    int chunks = 0;
    // and what makes a logit of <q, k>: to_logit up, down one over up
    float to_logit = 1.f, up = 1.f, down = 1.f;
};
hipError_t launch_attend_shared(const PrefixArgs &p, hipStream_t st);

}  // namespace proj
