// quant.hip -- projection with 4-bit weights and group scales, and the
// layout and making of such weights.
//
//     Y[m, n] = sum_g s[n, g] * (sum_{k in g} X[m, k] c[n, k] - z[n, g] sum_{k in g} X[m, k])
#include <type_traits>

#include "decode.hpp"
#include "kernels.hpp"

namespace proj {

// For what lies in LDS beside the copies' targets: the compiler takes accesses through types of
// their own (float, HIP's float2) for possible readers of any copy, and waits for all of them.
typedef float __attribute__((may_alias)) f32_any;
typedef uint16_t __attribute__((may_alias)) u16_any;

// Bit position of code j of a word of eight.
__host__ __device__ constexpr int code_shift(int j) { return 4 * (j / 2) + 16 * (j % 2); }

__device__ __forceinline__ float group_scale(const QuantArgs &a, int64_t i) {
    return a.scales_f32 ? static_cast<const float *>(a.scales)[i]
                        : bf16_bits_to_f32(static_cast<const uint16_t *>(a.scales)[i]);
}

constexpr float kLargest = 0x1.fffffep127f;

// Words w0 .. w1 - 1 of one output by the definition, x times s (c - z).  The
// kernels below put this in the place of a sum that is not finite: they take
// a group's scale, the matrix cores also 16 + z times its sum of x, after the
// sum over x c, so that an infinite x and sums beyond the largest number give
// NaN or infinity where the definition has infinity or a number.  One lane's
// work, since such an X is a fault or an extreme: K = N = 8192 with an infinity in
// one of 16 rows 420 us instead of 13, in each of 1024 rows 50 ms instead of 0.16
// (a NaN ends the walk: 0.2).
__device__ __forceinline__ float quant_by_definition(int64_t m, int64_t n, int64_t w0, int64_t w1) {
    // The call's arguments (every kernel's first), read again: kept for this, they would take registers from the loops.
    auto kernarg = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(kernarg));
    const QuantArgs &a = *(const QuantArgs *)kernarg;
    const int64_t words = a.K / 8;
    float acc = 0.f;
#pragma unroll 1
    for (int64_t w = w0; w < w1 && acc == acc; ++w) {  // NaN stays
        const uint32_t word = a.codes[n * words + w];
        const int64_t g = n * a.G + w * 8 / a.group;
        const float z = a.zeros ? static_cast<float>(a.zeros[g]) : 8.f, s = group_scale(a, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = static_cast<float>((word >> code_shift(j)) & 15u);
            acc = __builtin_fmaf(bf16_bits_to_f32(a.X[m * a.K + w * 8 + j]), s * (c - z), acc);
        }
    }
    return acc;
}

// Any K (a multiple of 8), alignment and number of outputs: one wave per
// output, lane l taking words l, l + 64, ... of the row.  A word lies within
// one group.  A launch that cannot have a wave for every output goes round.
// Bound by reading X two bytes at a time and the codes again for every row:
// K = N = 8192 26 us for one row, 280 for 16, 16 ms for 1024.
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t words = a.K / 8, outputs = a.M * a.N;
    for (int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); idx < outputs;
         idx += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t m = idx / a.N, n = idx % a.N;
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
            if (!(fabsf(acc) <= kLargest)) acc = quant_by_definition(m, n, 0, words);
            const float b = (a.epi & 1) ? bf16_bits_to_f32(a.bias[n]) : 0.f;
            store_out(a.Y, a.out, idx, apply_epilogue(acc, a.epi, b));
        }
    }
}

// ------------------------------------------------ on the matrix cores
//
// Both kernels below take K in steps of 128 and multiply X by the codes
// themselves, in bf16 and therefore exactly: a code c becomes 16 + c, which is
// the code's four bits put into the bf16 pattern of 16.0 (a shift and an
// and-or for two codes), and
//     sum_k x (c - z) = sum_k x (16 + c) - (16 + z) sum_k x
// is had by starting the matrix product's accumulator at -(16 + z) sum_k x.
// The sums of x come from a product with constant columns.  At a group's end
// its fp32 sum is scaled and added: nothing is rounded below fp32.
//
// A lane reads 16 bytes of a column's codes: words 4 g .. 4 g + 3 of the
// step's sixteen (g = lane / 16).  One product of 32 k takes a word from each
// g, and which words meet in one product only matters across a group's end:
// as loaded they are 4 g + r (r = 0..3), which is right for groups of 128;
// exchanging rows of lanes makes it the same half of the step (groups of 64)
// or the same quarter (groups of 32).  X is read in the same order.

// An offset past every resource made here (they are below 2^31 bytes): a load there gives zero.
constexpr uint32_t kOutside = 0x80000000u;

// Which of a step's sixteen words (and chunks of 8 x) lane group g holds in register r.
template <int GROUP>
__device__ __forceinline__ int word_of(int r, int g) {
    if (GROUP == 128) return 4 * g + r;
    if (GROUP == 64) return (r & 1) + 8 * (r >> 1) + 4 * (g & 1) + 2 * (g >> 1);
    return 4 * r + g;
}

template <int GROUP>
__device__ __forceinline__ u32x4 arrange(u32x4 w) {
    if constexpr (GROUP <= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        w = u32x4{a[0], b[0], a[1], b[1]};
        if constexpr (GROUP == 32) {
            const auto c = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
            const auto d = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
            w = u32x4{c[0], c[1], d[0], d[1]};
        }
    }
    return w;
}

// Eight codes -> 16 + code in bf16.  The two constants are kept in registers
// (their values hidden from the compiler) so that and-then-or is one
// instruction, which takes no literal: 8 instructions a word instead of 12.
struct Widen {
    uint32_t mask, sixteen;
    __device__ __forceinline__ Widen() {
        asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
        asm("v_mov_b32 %0, 0x41804180" : "=v"(sixteen));
    }
    __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
        return __builtin_bit_cast(bf16x8, u32x4{((w << 3) & mask) | sixteen, ((w >> 1) & mask) | sixteen,
                                                ((w >> 5) & mask) | sixteen, ((w >> 9) & mask) | sixteen});
    }
};

// How a row ends: kWhole at a step's end (K a multiple of 128), kWords
// anywhere (K a multiple of 8), also within a lane's 16 bytes of codes, which
// are then four loads, so that none straddles its resource's end.
enum Edge { kWhole = 0, kWords = 1 };

// Words 4 g .. 4 g + 3 of a step of one column; past the resource's end zero.
template <int EDGE>
__device__ __forceinline__ u32x4 load_words(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t step) {
    if constexpr (EDGE == kWhole) {
        return __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off), static_cast<int>(step), 0);
    } else {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(off + 4 * i), static_cast<int>(step), 0);
        return w;
    }
}

// Up to 32 token rows (16 MT): bound by reading the codes once, at the
// smallest sizes by the latency of doing so.  A workgroup owns 16 NT columns;
// its waves take steps in turn (two neighbouring ones at a time where there
// are enough: 128 contiguous bytes of a column) with no barrier, and add up
// through LDS at the end.  Nothing is split over workgroups, so there is one
// launch and no workspace.  Neighbouring lanes read neighbouring 16 bytes
// (the cache takes a load whose lanes do not lie in runs one lane at a time:
// 64 cycles instead of 16), DEPTH steps ahead, into registers, and pass them on
// to the lanes that need them through a piece of LDS of the wave's own.  The
// columns' scales lie in LDS as fp32 and their zero points (8 where none are
// given) as bytes, `span` steps at a time.  M = 16, K = N = 8192: 12.9 us, of
// which about 5 are launch, first reads and end, the rest 4.3 TB/s; M = 1, N = 1024:
// 7.4 us.
template <int MT, int NT, int WAVES, int DEPTH, int GROUP, int EDGE>
__global__ __launch_bounds__(WAVES * 64) void quant_wave_kernel(QuantArgs a, int span) {
    constexpr int GP = 128 / GROUP, PER = 4 / GP;  // groups of a step, registers of a group
    constexpr int COLS = 16 * NT, THREADS = WAVES * 64;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * COLS;
    const int cols = a.N - n0 < COLS ? static_cast<int>(a.N - n0) : COLS;
    const int M = static_cast<int>(a.M), steps = static_cast<int>((a.K + 127) / 128);
    const uint32_t words = static_cast<uint32_t>(a.K / 8);
    const uint32_t wbytes = static_cast<uint32_t>(cols) * words * 4u, xbytes = static_cast<uint32_t>(M) * words * 16u;

    const Widen widen;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bf16x8 minus = __builtin_bit_cast(bf16x8, u32x4{0xbf80bf80u, 0xbf80bf80u, 0xbf80bf80u, 0xbf80bf80u});
    // byte offsets of a lane's codes (column lane / 4, piece lane % 4) and X (row
    // lane / 16 of four, chunk lane % 16); columns and rows past the end lie
    // outside the resources
    constexpr int XI = 4 * MT;  // loads of X a step
    uint32_t woff[NT], xoff[XI];
#pragma unroll
    for (int t = 0; t < NT; ++t) woff[t] = ((16u * t + lane / 4) * words + 4u * (lane % 4)) * 4u;
#pragma unroll
    for (int i = 0; i < XI; ++i) xoff[i] = ((4u * i + lane / 16) * words + c16) * 16u;
    // the wave's own LDS: its codes, then X with chunk c of row m at c ^ m % 16
    char *own = lds + wave * (NT * 1024 + MT * 4096);
    char *scales = lds + WAVES * (NT * 1024 + MT * 4096);

    for (int from = 0; from < steps; from += span) {
        const int count = steps - from < span ? steps - from : span;
        const int pair = count >= 4 * WAVES ? 1 : 0;
        auto step_of = [&](int i) { return ((wave + WAVES * (i >> pair)) << pair) + (i & pair); };
        u32x4 w[DEPTH][NT], x[DEPTH][XI];
        // steps past the end are read from empty resources: zeros
        auto fetch = [&](int slot, int i) {
            const int at = step_of(i);
            const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(a.codes + n0 * words, at < count ? wbytes : 0u);
            const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.X, at < count ? xbytes : 0u);
            const uint32_t word = static_cast<uint32_t>(from + at) * 16u;
            // in a row's last step, if it is short, the lanes' own offsets must show where the end is
            const bool inside = EDGE == kWhole || word + 16 <= words;
            const uint32_t by_lane = inside ? 0u : word, by_step = inside ? word : 0u;
            const uint32_t past = EDGE == kWhole || word + c16 < words ? 0u : kOutside;
#pragma unroll
            for (int t = 0; t < NT; ++t) w[slot][t] = load_words<EDGE>(rw, woff[t] + by_lane * 4u, by_step * 4u);
#pragma unroll
            for (int j = 0; j < XI; ++j)
                x[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(
                    rx, static_cast<int>((xoff[j] + by_lane * 16u) | past), static_cast<int>(by_step * 16u), 0);
        };
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) fetch(d, d);

        // scales [column][group], rows an odd number of words apart, and behind them the zero points
        const int groups = count * GP, row = groups | 1, zrow = ((groups + 3) / 4 | 1) * 4;
        float *sc = reinterpret_cast<float *>(scales);
        uint8_t *zc = reinterpret_cast<uint8_t *>(sc + COLS * row);
        if (from > 0) __syncthreads();
        const int64_t G = a.G, first = static_cast<int64_t>(from) * GP;
        const int valid = G - first < groups ? static_cast<int>(G - first) : groups;
        // a wave's lanes over `per` units of a row (a power of two) and 64 / per rows
        auto over = [&](int units, auto &&f) {
            const int shift = units >= 64 ? 6 : 32 - __builtin_clz(static_cast<unsigned>(units - 1 | 1));
            const int rows = 64 >> shift;
#pragma unroll 4
            for (int n = wave * rows + (lane >> shift); n < COLS; n += WAVES * rows)
                for (int i = lane & ((1 << shift) - 1); i < units; i += 1 << shift) f(n, i);
        };
        const int vec = a.scales_f32 ? 4 : 8;
        if (G % 16 == 0 && first % 16 == 0 && valid % 16 == 0 && a.vec_scales) {
            over(valid / vec, [&](int n, int i) {
                u32x4 v = {0u, 0u, 0u, 0u};
                const int64_t at = (n0 + n) * G + first + i * vec;
                if (n < cols) v = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.scales) + at * (16 / vec));
                float *to = sc + n * row + i * vec;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (a.scales_f32) {
                        to[e] = __uint_as_float(v[e]);
                    } else {
                        to[2 * e] = __uint_as_float(v[e] << 16);
                        to[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
                    }
                }
            });
            over(valid / 16, [&](int n, int i) {
                u32x4 v = {0x08080808u, 0x08080808u, 0x08080808u, 0x08080808u};
                if (n < cols && a.zeros) v = *reinterpret_cast<const u32x4 *>(a.zeros + (n0 + n) * G + first + i * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t *>(zc + n * zrow + i * 16 + 4 * e) = v[e];
            });
        } else {
            over(groups, [&](int n, int i) {
                const bool ok = n < cols && i < valid;
                const int64_t at = (n0 + n) * G + first + i;
                sc[n * row + i] = ok ? group_scale(a, at) : 0.f;
                zc[n * zrow + i] = ok && a.zeros ? a.zeros[at] : 8;
            });
        }
        __syncthreads();

        for (int i0 = 0; step_of(i0) < count; i0 += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                const int at = step_of(i0 + d);
                if (at >= count) break;
#pragma unroll
                for (int t = 0; t < NT; ++t) *reinterpret_cast<u32x4 *>(own + t * 1024 + lane * 16) = w[d][t];
#pragma unroll
                for (int j = 0; j < XI; ++j) {
                    const int r = 4 * j + lane / 16;
                    *reinterpret_cast<u32x4 *>(own + NT * 1024 + r * 256 + ((c16 ^ (r & 15)) << 4)) = x[d][j];
                }
                fetch(d, i0 + d + DEPTH);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
                bf16x8 xv[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        xv[m][r] = *reinterpret_cast<const bf16x8 *>(own + NT * 1024 + (16 * m + c16) * 256 +
                                                                     ((word_of<GROUP>(r, g) ^ c16) << 4));
                u32x4 wv[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    wv[t] = arrange<GROUP>(*reinterpret_cast<const u32x4 *>(own + t * 1024 + c16 * 64 + g * 16));
#pragma unroll
                for (int q = 0; q < GP; ++q) {
                    f32x4 minus_x[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        minus_x[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int r = q * PER; r < (q + 1) * PER; ++r) minus_x[m] = mfma16x16x32(xv[m][r], minus, minus_x[m]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int gi = at * GP + q;
                        const float s = sc[(16 * t + c16) * row + gi];
                        // no branch on a.zeros here: the compiler leaves too few wait states between a
                        // matrix product and its result's use behind the join of two branches
                        const float z = 16.f + static_cast<float>(zc[(16 * t + c16) * zrow + gi]);
                        f32x4 p[MT];
#pragma unroll
                        for (int m = 0; m < MT; ++m) p[m] = minus_x[m] * z;
#pragma unroll
                        for (int r = q * PER; r < (q + 1) * PER; ++r) {
                            const bf16x8 wf = widen(wv[t][r]);
#pragma unroll
                            for (int m = 0; m < MT; ++m) p[m] = mfma16x16x32(xv[m][r], wf, p[m]);
                        }
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[m][t][v] = __builtin_fmaf(s, p[m][v], acc[m][t][v]);
                        // done here: moved to the step's end, the products of all its groups would be held at once
#pragma unroll
                        for (int m = 0; m < MT; ++m) asm volatile("" : "+v"(acc[m][t]));
                    }
                }
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            }
        }
    }

    // add the waves' sums, 16 rows at a time, over their pieces of LDS (1 KB for each tile of columns); those
    // that are not finite are marked and done again at the end, where their code is not in the way
    float *red = reinterpret_cast<float *>(lds);
    constexpr int EACH = (16 * COLS + THREADS - 1) / THREADS;  // outputs of a thread of 16 rows
    static_assert(MT * EACH <= 32, "a bit to a sum");
    uint32_t again = 0;
    auto put = [&](int m, int n, float y) {
        const float b = (a.epi & 1) ? bf16_bits_to_f32(a.bias[n0 + n]) : 0.f;
        store_out(a.Y, a.out, m * a.N + n0 + n, apply_epilogue(y, a.epi, b));
    };
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[(wave * 16 + 4 * g + v) * COLS + 16 * t + c16] = acc[i][t][v];
        __syncthreads();
        const int rows = M - 16 * i < 16 ? M - 16 * i : 16;
        for (int e = tid, k = 0; e < rows * COLS; e += THREADS, ++k) {
            const int m = e / COLS, n = e % COLS;
            if (n >= cols) continue;
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) y += red[(w * 16 + m) * COLS + n];
            if (fabsf(y) <= kLargest)
                put(16 * i + m, n, y);
            else
                again |= 1u << (i * EACH + k);
        }
    }
    if (!__any(again != 0)) return;
    for (; again != 0; again &= again - 1) {
        const int bit = __builtin_ctz(again), e = tid + bit % EACH * THREADS, m = bit / EACH * 16 + e / COLS, n = e % COLS;
        put(m, n, quant_by_definition(m, n0 + n, 0, words));
    }
}

template <int MT, int NT, int WM, int WN, int GROUP>
struct TileCfg {
    static constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = WM * WN;
    static constexpr int GP = 128 / GROUP, PER = 4 / GP;
    static constexpr int RING = 3;                      // steps in LDS
    static constexpr int STAGE = BM * 256;              // bytes of a step's X
    static constexpr int NX = STAGE / 1024 / WAVES;     // copies of a wave
    static constexpr int WSTAGE = BN * 64;              // bytes of a step's codes
    static constexpr int NW = WSTAGE / 1024 / WAVES;    // copies of a wave
    static constexpr int SI = (BN * GP + WAVES * 64 - 1) / (WAVES * 64);  // scales of a thread
    static constexpr int SCALES = GP * BN;              // a float and a bf16 each
    static constexpr int SUMS = GP * BM;                // floats
    static constexpr int LDS = RING * (STAGE + WSTAGE) + 2 * (SCALES * 6 + SUMS * 4);
    static_assert(LDS <= 160 << 10, "a compute unit's LDS");
    static_assert(STAGE % (1024 * WAVES) == 0 && WSTAGE % (1024 * WAVES) == 0, "copies divide evenly over the waves");
};

// More rows: tiles of BM rows by BN columns, 16 MT x 16 NT to a wave.  X and
// the codes go through rings of three steps in LDS, filled by copies that pass
// no register (16-byte chunk c of X's row m at c ^ m % 16, so that the 16 rows
// of a fragment fall on different banks); codes are widened in the registers
// of the waves that use them.  In step s the workgroup multiplies step s,
// adds up the x of step s + 1 (one 16-row tile to a wave), puts down the scales
// of s + 1, reads its X fragments of s + 1, and fetches the codes of s + 2 and
// the scales and X of s + 3; one barrier a step publishes all of it.  Loads
// complete in order, so whatever is used a step after its issue makes all that
// was issued before it wait: everything is used two steps after.  M = 1024,
// K = N = 8192, groups of 128, no zero points: 143 us (960 TFLOP/s; 180 where the
// clock is low); without the memory operations the loop takes 108, its matrix
// operations alone 98.  M = 64, N = 28672, groups of 64, zero points: 73 us, with
// vector instructions in 39% of a SIMD's cycles and matrix ones in 19%: few waves
// (1.3 to a SIMD) that wait.  The 128 x 256 tile's registers hold what the
// first needs; with zero points or ragged rows 2 to 104 are spilled, and each
// reload waits for all copies (times at launch_tile).
template <int MT, int NT, int WM, int WN, int GROUP, bool ZEROS, bool F32, int EDGE>
__global__ __launch_bounds__(WM *WN * 64, 2) void quant_tile_kernel(QuantArgs a, int splits) {
    using C = TileCfg<MT, NT, WM, WN, GROUP>;
    constexpr int GP = C::GP, PER = C::PER, THREADS = C::WAVES * 64;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char *wlds = lds + C::RING * C::STAGE;
    float *sums = reinterpret_cast<float *>(wlds + C::RING * C::WSTAGE);
    f32_any *sc = sums + 2 * C::SUMS;                              // scales [group][column]
    u16_any *zc = reinterpret_cast<u16_any *>(sc + 2 * C::SCALES);  // 16 + zero point, in bf16
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave % WM, wn = wave / WM;

    // Workgroup ids go round the eight dies in turn; each die takes a
    // contiguous run of tiles, rows fastest, so that the codes of a column
    // block are fetched by one die.
    const uint32_t mb = static_cast<uint32_t>((a.M + C::BM - 1) / C::BM), total = gridDim.x;
    const uint32_t die = blockIdx.x % 8, share = total / 8, more = total % 8;
    uint32_t id = die * share + (die < more ? die : more) + blockIdx.x / 8;
    const int split = static_cast<int>(id % static_cast<uint32_t>(splits));
    id /= static_cast<uint32_t>(splits);
    const int64_t m0 = static_cast<int64_t>(id % mb) * C::BM, n0 = static_cast<int64_t>(id / mb) * C::BN;
    const int rows = a.M - m0 < C::BM ? static_cast<int>(a.M - m0) : C::BM;
    const int cols = a.N - n0 < C::BN ? static_cast<int>(a.N - n0) : C::BN;
    const int steps = static_cast<int>((a.K + 127) / 128);
    const int first = static_cast<int>(static_cast<int64_t>(steps) * split / splits);
    const int count = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / splits) - first;
    const uint32_t words = static_cast<uint32_t>(a.K / 8);

    // Byte offsets of a lane's copies of X (block j * WAVES + wave of a stage is
    // four rows of 16 chunks), codes and scales.  Rows and columns past the
    // end lie outside the resources; steps past the end (which are issued all
    // the same, so that every step waits for the same count) use empty ones.
    // A step moves a scalar offset, which the bounds may not include: only in
    // a row's last step, if it is short, do lanes work out theirs.
    const uint32_t xbytes = static_cast<uint32_t>(rows) * words * 16u, wbytes = static_cast<uint32_t>(cols) * words * 4u;
    const uint32_t G = static_cast<uint32_t>(a.G), sbytes = static_cast<uint32_t>(cols) * G;
    constexpr uint32_t size = F32 ? 4 : 2;
    const char *scale0 = static_cast<const char *>(a.scales) + n0 * a.G * size;
    const uint8_t *zero0 = ZEROS ? a.zeros + n0 * a.G : nullptr;
    uint32_t xoff[C::NX], woff[C::NW], soff[C::SI];
#pragma unroll
    for (int j = 0; j < C::NX; ++j) {
        const uint32_t r = static_cast<uint32_t>((j * C::WAVES + wave) * 4 + lane / 16);
        xoff[j] = (r * words + (static_cast<uint32_t>(c16) ^ (r & 15))) * 16u;
    }
#pragma unroll
    for (int j = 0; j < C::NW; ++j)
        woff[j] = (static_cast<uint32_t>((j * C::WAVES + wave) * 16 + lane / 4) * words + lane % 4 * 4u) * 4u;
#pragma unroll
    for (int i = 0; i < C::SI; ++i) {
        const uint32_t e = i * THREADS + tid;
        soff[i] = e / GP * G + e % GP;
    }
    auto copy_x = [&](int s, int j) {
        char *to = lds + (s % C::RING) * C::STAGE + (j * C::WAVES + wave) * 1024;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(a.X + m0 * a.K, s < count ? xbytes : 0u);
        const uint32_t word = static_cast<uint32_t>(first + s) * 16u;
        if (EDGE == kWhole || word + 16 <= words) {
            dma16_buf(r, xoff[j], word * 16u, to);
        } else {
            const uint32_t row = static_cast<uint32_t>((j * C::WAVES + wave) * 4 + lane / 16);
            const bool in = word + (static_cast<uint32_t>(c16) ^ (row & 15)) < words;  // past the row: zeros
            dma16_buf(r, in ? xoff[j] + word * 16u : kOutside, 0, to);
        }
    };
    // codes: block j * WAVES + wave of a step is 16 columns of 64 bytes
    auto copy_w = [&](int s, int j) {
        char *to = wlds + (s % C::RING) * C::WSTAGE + (j * C::WAVES + wave) * 1024;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(a.codes + n0 * words, s < count ? wbytes : 0u);
        const uint32_t word = static_cast<uint32_t>(first + s) * 16u;
        if constexpr (EDGE == kWhole) {
            dma16_buf(r, woff[j], word * 4u, to);
        } else {
            // four bytes to a lane, so that none straddles the resource's end
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t col = (j * C::WAVES + wave) * 16u + 4u * i + lane / 16;
                dma4_buf(r, (col * words + word + c16) * 4u, 0, to + i * 256);
            }
        }
    };
    // scales and zero points as they are in memory: converting them waits for them
    // (in their own types: so does widening them)
    std::conditional_t<F32, uint32_t, uint16_t> sv[2][C::SI];
    uint8_t zv[2][C::SI];
    auto load_scales = [&](int s, int odd) {
        const uint32_t at = static_cast<uint32_t>(first + s) * GP;
        const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(scale0, s < count ? sbytes * size : 0u);
        const __amdgpu_buffer_rsrc_t rz = buffer_rsrc(zero0, s < count ? sbytes : 0u);
#pragma unroll
        for (int i = 0; i < C::SI; ++i) {
            const uint32_t e = i * THREADS + tid;
            const uint32_t off = EDGE == kWhole || GP == 1 || at + e % GP < G ? soff[i] + at : kOutside / 4;
            if constexpr (F32)
                sv[odd][i] = __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(off * 4u), 0, 0);
            else
                sv[odd][i] = __builtin_amdgcn_raw_buffer_load_b16(rs, static_cast<int>(off * 2u), 0, 0);
            if (ZEROS) zv[odd][i] = __builtin_amdgcn_raw_buffer_load_b8(rz, static_cast<int>(off), 0, 0);
        }
    };
    auto put_scales = [&](int s, int odd) {
#pragma unroll
        for (int i = 0; i < C::SI; ++i) {
            const int e = i * THREADS + tid, to = (s & 1) * C::SCALES + e % GP * C::BN + e / GP;
            if (e >= C::SCALES) continue;
            if constexpr (F32)
                sc[to] = __uint_as_float(sv[odd][i]);
            else
                sc[to] = bf16_bits_to_f32(sv[odd][i]);
            if (ZEROS) zc[to] = f32_to_bf16_bits(16.f + static_cast<float>(zv[odd][i]));
        }
    };
    // LDS offsets of a lane's fragments within a 16-row tile
    int xaddr[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) xaddr[r] = c16 * 256 + ((word_of<GROUP>(r, g) ^ c16) << 4);
    auto fragment = [&](int s, int tile, int r) {
        return *reinterpret_cast<const bf16x8 *>(lds + (s % C::RING) * C::STAGE + tile * 4096 + xaddr[r]);
    };
    // -sum x (times 24, 16 and the zero point of 8, where there are no zeros
    // given) of a step's groups, one 16-row tile to a wave: read, add, put down
    const uint32_t unit = ZEROS ? 0xbf80bf80u : 0xc1c0c1c0u;
    const bf16x8 minus = __builtin_bit_cast(bf16x8, u32x4{unit, unit, unit, unit});
    const int sum_tile = wave % (C::BM / 16);
    bf16x8 sx[4];
    f32x4 sum_x[GP];
    auto read_x = [&](int s) {
#pragma unroll
        for (int r = 0; r < 4; ++r) sx[r] = fragment(s, sum_tile, r);
    };
    auto add_x = [&]() {
#pragma unroll
        for (int q = 0; q < GP; ++q) {
            sum_x[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = q * PER; r < (q + 1) * PER; ++r) sum_x[q] = mfma16x16x32(sx[r], minus, sum_x[q]);
        }
    };
    auto put_sums = [&](int s) {
        if (c16 == 0)
#pragma unroll
            for (int q = 0; q < GP; ++q)
                *reinterpret_cast<f32x4 *>(sums + (s & 1) * C::SUMS + q * C::BM + 16 * sum_tile + 4 * g) = sum_x[q];
    };

    const Widen widen;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Per step a wave issues NX + NW copies (and loads of scales); waiting
    // until that many are left therefore has those issued two steps ago done
    // and leaves the last step's in flight.
    constexpr int COPIES = C::NX + C::NW * (EDGE == kWords ? 4 : 1);
    load_scales(0, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < C::NX; ++j) copy_x(s, j);
    put_scales(0, 0);
    load_scales(1, 1);
    load_scales(2, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int j = 0; j < C::NW; ++j) copy_w(s, j);
        if (s == 0)
#pragma unroll
            for (int j = 0; j < C::NX; ++j) copy_x(2, j);
    }
    wait_vm<COPIES>();
    __syncthreads();
    // X fragments of the step, each replaced by the next step's after its last use
    bf16x8 xf[4][MT];
    auto load_x = [&](int s, int r) {
#pragma unroll
        for (int i = 0; i < MT; ++i) xf[r][i] = fragment(s, wm * MT + i, r);
    };
#pragma unroll
    for (int r = 0; r < 4; ++r) load_x(0, r);
    read_x(0);
    add_x();
    put_sums(0);

    auto step = [&](int s, auto parity) {
        constexpr int odd = decltype(parity)::value;
        wait_vm<COPIES>();
        lds_wait_all();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int column = (s & 1) * C::SCALES + wn * NT * 16 + c16;
        const float *xs = sums + (s & 1) * C::SUMS + wm * MT * 16 + 4 * g;
        u32x4 w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            w[t] = arrange<GROUP>(*reinterpret_cast<const u32x4 *>(wlds + (s % C::RING) * C::WSTAGE +
                                                                   (wn * NT + t) * 1024 + c16 * 64 + g * 16));
#pragma unroll
        for (int q = 0; q < GP; ++q) {
            f32x4 cs[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) cs[i] = *reinterpret_cast<const f32x4 *>(xs + q * C::BM + 16 * i);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float scale = sc[column + q * C::BN + 16 * t];
                const float zero = ZEROS ? bf16_bits_to_f32(zc[column + q * C::BN + 16 * t]) : 0.f;
                f32x4 p[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) p[i] = ZEROS ? cs[i] * zero : cs[i];
#pragma unroll
                for (int r = q * PER; r < (q + 1) * PER; ++r) {
                    const bf16x8 wf = widen(w[t][r]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) p[i] = mfma16x16x32(xf[r][i], wf, p[i]);
                    if (t == NT - 1) load_x(s + 1, r);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][t][v] = __builtin_fmaf(scale, p[i][v], acc[i][t][v]);
                // done here: moved to the step's end, the products of all its groups would be held at once
#pragma unroll
                for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[i][t]));

                // What the coming steps need, a little after each tile: all
                // waves are at the same place of a step, and issued together
                // these stand in line for the memory pipeline while the matrix
                // cores wait.
                constexpr int H = GP * NT;
                const int h = q * NT + t;
                if (q == 0)
#pragma unroll
                    for (int j = t * C::NX / NT; j < (t + 1) * C::NX / NT; ++j) copy_x(s + 3, j);
                if (q == 0)
#pragma unroll
                    for (int j = t * C::NW / NT; j < (t + 1) * C::NW / NT; ++j) copy_w(s + 2, j);
                if (h == 0) read_x(s + 1);
                if (h == 1) {
                    add_x();
                    put_scales(s + 1, odd ^ 1);
                }
                if (h == (H > 2 ? 2 : 1)) {
                    load_scales(s + 3, odd ^ 1);
                    put_sums(s + 1);
                }
            }
        }
    };
    for (int s = 0; s < count; s += 2) {
        step(s, std::integral_constant<int, 0>());
        if (s + 1 < count) step(s + 1, std::integral_constant<int, 1>());
    }
    wait_vm<0>();

    // Sums that are not finite are marked, and done again one after the other:
    // in place, their code would be there once for every sum.  The lane's place
    // is worked out again, so that it takes no registers in the loop.
    int l = static_cast<int>(__lane_id());
    asm volatile("" : "+v"(l));
    const int row0 = wm * MT * 16 + 4 * (l >> 4), col0 = wn * NT * 16 + (l & 15);
    auto put = [&](int r, int col, float sum, float b) {
        const int64_t at = (m0 + r) * a.N + n0 + col;
        if (splits > 1)
            a.ws[split * a.M * a.N + at] = sum;
        else
            store_out(a.Y, a.out, at, apply_epilogue(sum, a.epi, b));
    };
    const bool biased = (a.epi & 1) && splits == 1;
    uint64_t again = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = col0 + 16 * t;
        if (col >= cols) continue;
        const float b = biased ? bf16_bits_to_f32(a.bias[n0 + col]) : 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int r = row0 + 16 * i + v;
                if (r >= rows) continue;
                if (fabsf(acc[i][t][v]) <= kLargest)
                    put(r, col, acc[i][t][v], b);
                else
                    again |= uint64_t{1} << ((t * MT + i) * 4 + v);
            }
    }
    static_assert(NT * MT * 4 <= 64, "a bit to a sum");
    const int64_t w0 = static_cast<int64_t>(first) * 16, w1 = w0 + static_cast<int64_t>(count) * 16;
    if (!__any(again != 0)) return;
    for (; again != 0; again &= again - 1) {
        const int bit = __builtin_ctzll(again), v = bit & 3, i = (bit >> 2) % MT, t = (bit >> 2) / MT;
        const int r = row0 + 16 * i + v, col = col0 + 16 * t;
        put(r, col, quant_by_definition(m0 + r, n0 + col, w0, w1 < words ? w1 : words),
            biased ? bf16_bits_to_f32(a.bias[n0 + col]) : 0.f);
    }
}

// A word to a thread; bound by bytes: 8192 x 8192 20 us, 5.1 TB/s.
__global__ __launch_bounds__(256) void pack_codes_kernel(const uint8_t *q, int64_t words, uint32_t *codes) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) w |= static_cast<uint32_t>(q[i * 8 + j] & 15) << code_shift(j);
        codes[i] = w;
    }
}

// One wave per group of a row: the group's extremes, then its codes.  Lane l
// holds words l of the group (16 words at most); a word is eight weights.
// Weights are registered once: 8192 x 8192 takes 269 us with groups of 128, 519 of
// 64, 1001 of 32, bound by the waves, of whose lanes 16, 8 or 4 hold weights.
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t *W, int64_t N, int64_t K, int64_t G, int group,
                                                       uint32_t *codes, void *scales, int scales_f32, uint8_t *zeros) {
    const int lane = threadIdx.x & 63;
    for (int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); idx < N * G;
         idx += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t n = idx / G, k = (idx % G) * group + lane * 8;
        const bool live = lane * 8 < group && k < K;
        float w[8], lo = 0.f, hi = 0.f;
        bool finite = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = live ? bf16_bits_to_f32(W[n * K + k + j]) : 0.f;
            lo = fminf(lo, w[j]);
            hi = fmaxf(hi, w[j]);
            finite = finite && fabsf(w[j]) <= kLargest;
        }
#pragma unroll
        for (int h = 32; h >= 1; h >>= 1) {
            lo = fminf(lo, __shfl_xor(lo, h, 64));
            hi = fmaxf(hi, __shfl_xor(hi, h, 64));
        }
        const float range = hi - lo;  // past the largest float for weights at both its ends
        float s = !zeros ? fmaxf(hi, -lo) / 7.f : range <= kLargest ? range / 15.f : hi / 15.f - lo / 15.f;
        if (!scales_f32) s = bf16_bits_to_f32(f32_to_bf16_bits(s));
        if (__any(!finite)) s = __builtin_nanf("");  // the extremes above leave a NaN out
        const float z = !zeros ? 8.f : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
        if (lane == 0) {
            if (scales_f32)
                static_cast<float *>(scales)[idx] = s;
            else
                static_cast<uint16_t *>(scales)[idx] = f32_to_bf16_bits(s);
            if (zeros) zeros[idx] = static_cast<uint8_t>(z);
        }
        if (!live) continue;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = s > 0.f ? fminf(fmaxf(rintf(w[j] / s) + z, 0.f), 15.f) : z;
            word |= static_cast<uint32_t>(c) << code_shift(j);
        }
        codes[(n * K + k) / 8] = word;
    }
}

// Instantiated here: the launchers below are compiled for the host only.
#define PROJ_QUANT_TILE(G, Z, F, E)                                                         \
    template __global__ void quant_tile_kernel<4, 2, 1, 4, G, Z, F, E>(QuantArgs, int);     \
    template __global__ void quant_tile_kernel<4, 4, 2, 4, G, Z, F, E>(QuantArgs, int);
#define PROJ_QUANT_EDGE(G, E)                                                               \
    template __global__ void quant_wave_kernel<1, 1, 8, 4, G, E>(QuantArgs, int);           \
    template __global__ void quant_wave_kernel<1, 2, 8, 3, G, E>(QuantArgs, int);           \
    template __global__ void quant_wave_kernel<1, 4, 4, 3, G, E>(QuantArgs, int);           \
    template __global__ void quant_wave_kernel<2, 2, 8, 2, G, E>(QuantArgs, int);           \
    PROJ_QUANT_TILE(G, true, true, E)                                                       \
    PROJ_QUANT_TILE(G, true, false, E)                                                      \
    PROJ_QUANT_TILE(G, false, true, E)                                                      \
    PROJ_QUANT_TILE(G, false, false, E)
#define PROJ_QUANT_GROUP(G)    \
    PROJ_QUANT_EDGE(G, kWhole) \
    PROJ_QUANT_EDGE(G, kWords)
PROJ_QUANT_GROUP(32)
PROJ_QUANT_GROUP(64)
PROJ_QUANT_GROUP(128)

#ifndef __HIP_DEVICE_COMPILE__
// Workgroups of 256 threads for kernels that go round where these are too few.
static dim3 grid_for(int64_t items, int64_t per) {
    const int64_t g = (items + per - 1) / per;
    return dim3(static_cast<unsigned>(g < most_groups(256) ? g : most_groups(256)));
}

static hipError_t launch_rows(const QuantArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(quant_rows_kernel, grid_for(a.M * a.N, 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int MT, int NT, int WAVES, int DEPTH, int GROUP, int EDGE>
static hipError_t run_wave(const QuantArgs &a, hipStream_t st) {
    constexpr int gp = 128 / GROUP, cols = 16 * NT;
    const int64_t groups_n = (a.N + cols - 1) / cols;
    if (groups_n > most_groups(WAVES * 64)) return launch_rows(a, st);
    // the waves' own pieces, and the scales of as many steps as fit into 44 KB
    // beside them: 5 bytes a group, rows padded
    constexpr int pieces = WAVES * (NT * 1024 + MT * 4096);
    const int64_t steps = (a.K + 127) / 128;
    int64_t span = (((44 << 10) / cols - 16) / 5 - 1) / gp;
    if (span >= 16) span = span / 16 * 16;  // a later span starts at a multiple of 16 groups
    if (span > steps) span = steps;
    const int64_t groups = span * gp;
    int64_t lds = pieces + cols * ((groups | 1) * 4 + ((groups + 3) / 4 | 1) * 4);
    auto kernel = quant_wave_kernel<MT, NT, WAVES, DEPTH, GROUP, EDGE>;
    if (lds > (64 << 10)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups_n)), dim3(WAVES * 64), static_cast<unsigned>(lds), st, a,
                       static_cast<int>(span));
    return hipGetLastError();
}

template <int GROUP, int EDGE>
static hipError_t launch_wave(const QuantArgs &a, hipStream_t st) {
    // Columns to a workgroup, by how many there are to a compute unit (M = 16,
    // K = 8192; us with 16, 32 and 64 columns): N = 4096 9.2, 10.4, 19.0; N = 8192
    // 16.4, 13.1, 20.0; N = 28672 59.1, 46.3, 38.3.  With 32 rows 32 columns are
    // best throughout (N = 28672: 67.0, with 64 70.2).
    const int64_t cus = a.cus;
    if (a.M > 16) return run_wave<2, 2, 8, 2, GROUP, EDGE>(a, st);
    if (a.N <= 16 * cus) return run_wave<1, 1, 8, 4, GROUP, EDGE>(a, st);
    if (a.N <= 64 * cus) return run_wave<1, 2, 8, 3, GROUP, EDGE>(a, st);
    return run_wave<1, 4, 4, 3, GROUP, EDGE>(a, st);
}

template <int MT, int NT, int WM, int WN, int GROUP, bool ZEROS, int EDGE>
static hipError_t run_tile(const QuantArgs &a, hipStream_t st) {
    using C = TileCfg<MT, NT, WM, WN, GROUP>;
    const int64_t tiles = ((a.M + C::BM - 1) / C::BM) * ((a.N + C::BN - 1) / C::BN), steps = (a.K + 127) / 128;
    // split K where the tiles leave compute units idle, in runs of four steps at
    // least (M = 64, K = 8192, N = 28672, 224 tiles: 100, 82, 91, 90 us with 1 to 4
    // splits; M = 64, K = 8192, N = 512, runs of at least 2, 4, 8, 16 steps: 18.5,
    // 16.5, 18.0, 24.1 us)
    int64_t splits = tiles >= a.cus ? 1 : 2 * a.cus / tiles;
    if (splits > steps / 4) splits = steps / 4;
    const int64_t room = static_cast<int64_t>(a.ws_bytes / 4) / (a.M * a.N);
    if (splits > room) splits = room;
    if (splits < 1) splits = 1;
    if (tiles * splits > most_groups(C::WAVES * 64)) return launch_rows(a, st);
    auto kernel = a.scales_f32 ? quant_tile_kernel<MT, NT, WM, WN, GROUP, ZEROS, true, EDGE>
                               : quant_tile_kernel<MT, NT, WM, WN, GROUP, ZEROS, false, EDGE>;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       C::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tiles * splits)), dim3(C::WAVES * 64), C::LDS, st, a,
                       static_cast<int>(splits));
    e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    Args r{};
    r.M = a.M, r.N = a.N, r.K = a.K;
    r.epi = a.epi, r.out = a.out;
    r.bias = a.bias;
    r.Y = a.Y;
    r.ws = a.ws;
    return launch_splitk_reduce(r, static_cast<int>(splits), st);
}

template <int GROUP, bool ZEROS, int EDGE>
static hipError_t launch_tile(const QuantArgs &a, hipStream_t st) {
    // large tiles once there are enough of them (K = 8192, N = 8192; us with 128 x 256
    // and with 64 x 128 tiles; groups of 128, no zero points): M = 256 71, 58;
    // M = 512 107, 96; M = 1024 159, 196.  The rule is that combination's: M = 1024
    // with groups of 64 175, 221, with zero points and groups of 128 170, 223, of 64
    // 349, 252, of 32 729, 305; K = 8160 with zero points and groups of 128 280, 254
    if (((a.M + 127) / 128) * ((a.N + 255) / 256) * 2 > a.cus) return run_tile<4, 4, 2, 4, GROUP, ZEROS, EDGE>(a, st);
    return run_tile<4, 2, 1, 4, GROUP, ZEROS, EDGE>(a, st);
}

template <int GROUP, int EDGE>
static hipError_t launch_group(const QuantArgs &a, hipStream_t st) {
    // up to 32 rows without tiles (K = 8192; us without and with): M = 24 N = 8192
    // 15.8, 21.2; M = 32 N = 28672 67, 74; M = 32 N = 2048 13.4, 12.0
    if (a.M <= 32) return launch_wave<GROUP, EDGE>(a, st);
    return a.zeros ? launch_tile<GROUP, true, EDGE>(a, st) : launch_tile<GROUP, false, EDGE>(a, st);
}

template <int GROUP>
static hipError_t launch_edge(const QuantArgs &a, hipStream_t st) {
    return a.K % 128 == 0 ? launch_group<GROUP, kWhole>(a, st) : launch_group<GROUP, kWords>(a, st);
}

hipError_t launch_quant(const QuantArgs &args, hipStream_t st) {
    QuantArgs a = args;
    a.vec_scales = (reinterpret_cast<uintptr_t>(a.scales) | reinterpret_cast<uintptr_t>(a.zeros)) % 16 == 0;
    // the matrix-core kernels read X in 16-byte chunks, and address a tile's
    // codes (at most 256 columns) and rows of X (128) with 32 bits
    if (a.K > 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.K < (int64_t{1} << 23)) {
        switch (a.group) {
            case 32: return launch_edge<32>(a, st);
            case 64: return launch_edge<64>(a, st);
            case 128: return launch_edge<128>(a, st);
        }
    }
    return launch_rows(a, st);
}

hipError_t launch_pack_codes(const uint8_t *q, int64_t N, int64_t K, uint32_t *codes, hipStream_t st) {
    hipLaunchKernelGGL(pack_codes_kernel, grid_for(N * K / 8, 256), dim3(256), 0, st, q, N * K / 8, codes);
    return hipGetLastError();
}

hipError_t launch_quantize(const uint16_t *W, int64_t N, int64_t K, int group, uint32_t *codes, void *scales,
                           int scales_f32, uint8_t *zeros, hipStream_t st) {
    const int64_t G = (K + group - 1) / group;
    hipLaunchKernelGGL(quantize_kernel, grid_for(N * G, 4), dim3(256), 0, st, W, N, K, G, group, codes, scales, scales_f32,
                       zeros);
    return hipGetLastError();
}
#endif

}  // namespace proj
