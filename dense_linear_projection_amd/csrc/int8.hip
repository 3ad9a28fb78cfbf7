// int8.hip -- projection of 8-bit integers with a scale for each token and
// each output, and the making of such integers from bf16 rows.
//
//     Y[m, n] = epilogue(x_scales[m] w_scales[n] sum_k X[m, k] W[n, k] (+ bias[n]))
//
// The sum is exact (32-bit integers); it meets the scales in 64-bit floating
// point, so that their product neither overflows nor vanishes on its way and
// the result before bias and GELU is the rounded one.
#include <type_traits>

#include "layer.hpp"

namespace proj {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;
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
    // eight elements' integers, in order. Where the row has no integers (zeros, or a NaN in it) they are 0.
    __device__ __forceinline__ u32x2 operator()(u32x4 x) const {
        uint32_t n[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = __uint_as_float(e % 2 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16) * up * per;
            // 19 bits of y, and the nearest integer in the low bits of a number of 2^23
            n[e] = __float_as_uint(__uint_as_float((__float_as_uint(y) + 16u) & ~31u) + 0x1.8p23f);
        }
        u32x2 q = {0u, 0u};
        if (per != 0.f)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[4 * h + 3], n[4 * h + 2], 0x0c0c0400u),
                                             __builtin_amdgcn_perm(n[4 * h + 1], n[4 * h], 0x0c0c0400u), 0x05040100u);
        return q;
    }
};

// Largest |x| of eight, as bits, two at a time.
__device__ __forceinline__ u16x2 most8(u16x2 top, u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    return top;
}

// Elements 8 c .. 8 c + 7 of a row, zeros behind its end.
template <bool ONCE = true>
__device__ __forceinline__ u32x4 row_chunk(const uint16_t *x, int64_t c, int64_t K, bool vec) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(x + 8 * c);
    if (vec && 8 * c + 8 <= K) return ONCE ? __builtin_nontemporal_load(p) : *p;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (8 * c < K)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * c + e < K) w[e / 2] |= static_cast<uint32_t>(x[8 * c + e]) << (16 * (e % 2));
    return w;
}

// LANES threads to a row, 256 to a workgroup. The row's R chunks of a thread stay in
// registers between its largest element and its integers (R = 0: longer rows, read
// twice). vec: rows start at 16-byte boundaries. Bound by bytes: 4096 rows of 8192 21.4 us,
// 4.7 TB/s; up to 16 rows 4 us, latency.
template <int LANES, int R>
__global__ __launch_bounds__(256) void quantize_rows_kernel(RowsArgs a, int vec) {
    constexpr int ROWS = 256 / LANES;
    __shared__ uint32_t peak[4];
    const int t = threadIdx.x % LANES;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * ROWS; m0 < a.M; m0 += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t m = m0 + threadIdx.x / LANES;
        const bool there = m < a.M;
        const uint16_t *x = a.X + (there ? m : a.M - 1) * a.stride;
        u16x2 top2 = {0, 0};
        u32x4 w[R > 0 ? R : 1];
        if constexpr (R > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) w[r] = row_chunk(x, r * LANES + t, a.K, vec != 0);
#pragma unroll
            for (int r = 0; r < R; ++r) top2 = most8(top2, w[r]);
        } else {
            for (int64_t c = t; 8 * c < a.K; c += LANES) top2 = most8(top2, row_chunk(x, c, a.K, vec != 0));
        }
        uint32_t top = max(top2[0], top2[1]);
#pragma unroll
        for (int h = 32; h >= 1; h >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), h, 64)));
        if constexpr (LANES == 256) {
            __syncthreads();  // the row before is done with
            if ((threadIdx.x & 63) == 0) peak[threadIdx.x >> 6] = top;
            __syncthreads();
            top = max(max(peak[0], peak[1]), max(peak[2], peak[3]));
        }
        if (!there) continue;
        const RowScale s(top);
        int8_t *q = a.q + m * a.q_stride;
        if constexpr (R > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (8 * (r * LANES + t) < a.q_stride) *reinterpret_cast<u32x2 *>(q + 8 * (r * LANES + t)) = s(w[r]);
            for (int64_t c = R * LANES + t; 8 * c < a.q_stride; c += LANES) *reinterpret_cast<u32x2 *>(q + 8 * c) = u32x2{0u, 0u};
        } else {
            for (int64_t c = t; 8 * c < a.q_stride; c += LANES) *reinterpret_cast<u32x2 *>(q + 8 * c) = s(row_chunk(x, c, a.K, vec != 0));
        }
        if (t == 0) a.scales[m] = s.scale;
    }
}

#define PROJ_ROWS_VARIANTS(X) X(64, 1) X(64, 2) X(256, 1) X(256, 2) X(256, 4) X(256, 8) X(256, 0)
#define PROJ_ROWS_INST(LANES, R) template __global__ void quantize_rows_kernel<LANES, R>(RowsArgs, int);
PROJ_ROWS_VARIANTS(PROJ_ROWS_INST)

// ------------------------------------------------------------------- product

__device__ __forceinline__ i32x4 mfma16x16x64(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// One output before bias and GELU.
__device__ __forceinline__ float scaled(int32_t sum, float xs, float ws) {
    return static_cast<float>(static_cast<double>(sum) * (static_cast<double>(xs) * ws));
}

// Bias and GELU of scaled sums. One GELU for every kernel, so that which of them runs does not show in the result.
template <int N>
__device__ __forceinline__ void finish(float (&v)[N], int epi, const float (&bias)[N]) {
    if (epi & 1)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += bias[e];
    if (epi & 2)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = gelu_tanh_fast(v[e]);
}

// Four outputs of one token, before bias and GELU scaled already, written where they are there.
__device__ __forceinline__ void write4(const IntArgs &a, int64_t m, int64_t n, const int32_t (&sum)[4], float xs) {
    float v[4], bias[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t col = n + r < a.N ? n + r : a.N - 1;
        v[r] = scaled(sum[r], xs, a.w_scales[col]);
        bias[r] = (a.epi & 1) ? bf16_bits_to_f32(a.bias[col]) : 0.f;
    }
    finish(v, a.epi, bias);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (n + r < a.N) store_out(a.Y, a.out, m * a.row + n + r, v[r]);
}

// An offset past every resource made here (they are below 2^31 bytes): a load there gives zero.
constexpr uint32_t kOutside = 0x80000000u;

// Few tokens: bound by reading W once. A workgroup has 16 MT tokens and 16 NT
// outputs and walks its share of K in stages of KC bytes, D - 1 of them on
// their way into an LDS ring (global-to-LDS copies of 1 KB, whole runs of KC bytes of
// a row) while one is multiplied; wave w takes the 64-byte steps w, w + WAVES, ...
// of a stage for the whole tile, and the waves' sums meet in LDS at the end.
// 16-byte chunk c of LDS row r lies at position c ^ (r % 16): the 16 rows of a
// fragment fall on different banks. W is read past the caches (non-temporal), X
// stays in them. With S > 1 splits of K the last workgroup of a tile to
// finish adds the others' sums, which lie in the workspace. 16 tokens, K = N = 8192
// 13.3 us, 5.1 TB/s; 64, N = 28672 46 us, the same rate.
//
// FUSED: very few tokens come as bf16 rows, and every workgroup makes them integers
// itself, in LDS, while its first stages of W are on their way: their bytes are few
// beside W's, and a launch less counts more (one token, K8192 N1024: 8.6 us a call
// against 10.5).
constexpr int kFusedRows = 4, kFusedK = 8192;  // rows whose chunks a workgroup's registers hold

template <int MT, int NT, int WAVES, int KC, int D, bool FUSED = false>
struct IntStreamCfg {
    static constexpr int NR = 16 * NT, MR = 16 * MT, CPR = KC / 16, RPI = 1024 / KC;
    static constexpr int STAGE = (NR + (FUSED ? 0 : MR)) * KC;
    static constexpr int PERW = STAGE / 1024 / WAVES;    // copies of a wave in a stage
    static constexpr int E = MT * NT * 256;              // outputs of a tile
    static constexpr int RED = WAVES * E * 4;
    static constexpr int LDS = D * STAGE > RED ? D * STAGE : RED;
    static_assert(STAGE % (1024 * WAVES) == 0 && CPR >= 16 && KC / 64 >= WAVES && (KC / 64) % WAVES == 0, "stage");
    static_assert(PERW * (D - 2) <= 63 && LDS <= 160 * 1024, "ring");
};

template <int MT, int NT, int WAVES, int KC, int D, bool FUSED>
__global__ __launch_bounds__(WAVES * 64) void int_stream_kernel(IntArgs a, uint32_t splits) {
    using C = IntStreamCfg<MT, NT, WAVES, KC, D, FUSED>;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    __shared__ __attribute__((aligned(16))) char made[FUSED ? kFusedRows * kFusedK : 16];
    __shared__ uint32_t peak[FUSED ? kFusedRows * WAVES : 1];
    __shared__ float made_scale[FUSED ? kFusedRows : 1];
    const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t tiles_n = static_cast<uint32_t>((a.N + C::NR - 1) / C::NR);
    uint32_t tile = blockIdx.x, split = 0;
    if (splits > 1) {
        tile = blockIdx.x / splits;
        split = blockIdx.x - tile * splits;
    }
    uint32_t tm = 0, tn = tile;
    if (a.M > C::MR) {
        tm = tile / tiles_n;
        tn = tile - tm * tiles_n;
    }
    const int64_t m0 = static_cast<int64_t>(tm) * C::MR, n0 = static_cast<int64_t>(tn) * C::NR;
    const int K = static_cast<int>(a.K), T = (K + KC - 1) / KC;
    const int first = static_cast<int>(static_cast<uint32_t>(T) * split / splits);
    const int nst = static_cast<int>(static_cast<uint32_t>(T) * (split + 1) / splits) - first;
    // Workgroups begin at different places of K: rows lie a power of two apart, and walking in step would
    // gather all reads on few memory channels.
    const int turn = nst > 0 ? static_cast<int>(tn * 7u % static_cast<uint32_t>(nst)) : 0;

    const int64_t rows_w = a.N - n0 < C::NR ? a.N - n0 : C::NR, rows_x = a.M - m0 < C::MR ? a.M - m0 : C::MR;
    const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(a.W + n0 * a.K, static_cast<uint32_t>(rows_w * a.K));
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(a.X + m0 * a.K, FUSED ? 0u : static_cast<uint32_t>(rows_x * a.K));
    const __amdgpu_buffer_rsrc_t none = buffer_rsrc(a.W, 0);
    uint32_t voff[C::PERW];
    int chunk[C::PERW];
#pragma unroll
    for (int j = 0; j < C::PERW; ++j) {
        const int row = (wave + j * WAVES) * C::RPI + lane / C::CPR;
        chunk[j] = ((lane % C::CPR) ^ (row & 15)) * 16;
        voff[j] = static_cast<uint32_t>((row < C::NR ? row : row - C::NR) * K + chunk[j]);
    }
    auto issue = [&](int i) {
        char *slot = lds + (i % D) * C::STAGE;
        int stage = i + turn;
        stage = (stage >= nst ? stage - nst : stage) + first;
        const bool live = i < nst, tail = stage == T - 1 && K % KC != 0;
#pragma unroll
        for (int j = 0; j < C::PERW; ++j) {
            const bool is_w = (wave + j * WAVES) * C::RPI < C::NR;  // wave-uniform
            // behind K lies the next row
            const uint32_t v = tail && stage * KC + chunk[j] >= K ? kOutside : voff[j];
            char *to = slot + (wave + j * WAVES) * 1024;
            if (is_w)
                dma16_buf_nt(live ? rw : none, v, static_cast<uint32_t>(stage * KC), to);
            else
                dma16_buf(live ? rx : none, v, static_cast<uint32_t>(stage * KC), to);
        }
    };
    i32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    constexpr int R = kFusedK / 8 / (WAVES * 64);
    u32x4 row[FUSED ? kFusedRows : 1][R];  // asked for ahead of the copies: loads complete in order
    if constexpr (FUSED) {
        const bool vec = a.rows_stride % 8 == 0 && reinterpret_cast<uintptr_t>(a.rows) % 16 == 0;
#pragma unroll
        for (int m = 0; m < kFusedRows; ++m)
            if (m < a.M)
#pragma unroll
                for (int r = 0; r < R; ++r) row[m][r] = row_chunk<false>(a.rows + m * a.rows_stride, r * WAVES * 64 + tid, a.rows_k, vec);
    }
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i);
    if constexpr (FUSED) {
#pragma unroll
        for (int m = 0; m < kFusedRows; ++m)
            if (m < a.M) {
                u16x2 top2 = {0, 0};
#pragma unroll
                for (int r = 0; r < R; ++r) top2 = most8(top2, row[m][r]);
                uint32_t top = max(top2[0], top2[1]);
#pragma unroll
                for (int h = 32; h >= 1; h >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), h, 64)));
                if (lane == 0) peak[m * WAVES + wave] = top;
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();  // the copies need not have landed
        asm volatile("" ::: "memory");
#pragma unroll
        for (int m = 0; m < kFusedRows; ++m)
            if (m < a.M) {
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) top = max(top, peak[m * WAVES + w]);
                const RowScale s(top);
                if (tid == 0) made_scale[m] = s.scale;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (8 * (r * WAVES * 64 + tid) < K) *reinterpret_cast<u32x2 *>(made + m * K + 8 * (r * WAVES * 64 + tid)) = s(row[m][r]);
            }
    }
    for (int i = 0; i < nst; ++i) {
        wait_vm<C::PERW *(D - 2)>();  // this wave's copies of stage i have landed
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();  // everyone's have, and the slot of stage i - 1 is free
        asm volatile("" ::: "memory");
        issue(i + D - 1);
        const char *slot = lds + (i % D) * C::STAGE;
#pragma unroll
        for (int s = 0; s < KC / 64 / WAVES; ++s) {
            const int c = (wave + s * WAVES) * 4 + g;
            i32x4 xf[MT], wf[NT];
            if constexpr (FUSED) {
                int stage = i + turn;
                stage = (stage >= nst ? stage - nst : stage) + first;
                const int k = stage * KC + 16 * c;
                xf[0] = i32x4{0, 0, 0, 0};
                if (c16 < rows_x && k < K) xf[0] = *reinterpret_cast<const i32x4 *>(made + c16 * K + k);
            } else {
#pragma unroll
                for (int t = 0; t < MT; ++t) xf[t] = *reinterpret_cast<const i32x4 *>(slot + (C::NR + t * 16 + c16) * KC + ((c ^ c16) << 4));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) wf[t] = *reinterpret_cast<const i32x4 *>(slot + (t * 16 + c16) * KC + ((c ^ c16) << 4));
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int u = 0; u < NT; ++u) acc[t][u] = mfma16x16x64(wf[u], xf[t], acc[t][u]);
        }
    }
    wait_vm<0>();
    __syncthreads();

    // The waves' sums, four outputs (columns 4 g ..) of a token (row c16) at a time
    i32x4 *red = reinterpret_cast<i32x4 *>(lds);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) red[(wave * MT * NT + t * NT + u) * 64 + lane] = acc[t][u];
    __syncthreads();
    constexpr int Q = (C::E / 4 + WAVES * 64 - 1) / (WAVES * 64);
    i32x4 sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = tid + q * WAVES * 64;
        if (e >= C::E / 4) break;
        sum[q] = red[e];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum[q] += red[w * (C::E / 4) + e];
    }
    if (splits > 1) {
        // Sums go past the dies' own caches, in both directions, so that waiting for the stores is all the order needed.
        int &is_last = *reinterpret_cast<int *>(lds);  // the sums there are in registers
        uint64_t *mine = reinterpret_cast<uint64_t *>(a.ws) + (static_cast<int64_t>(tile) * splits + split) * (C::E / 2);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = tid + q * WAVES * 64;
            if (e >= C::E / 4) break;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                __hip_atomic_store(mine + 2 * e + x, static_cast<uint64_t>(static_cast<uint32_t>(sum[q][2 * x + 1])) << 32 |
                                                         static_cast<uint32_t>(sum[q][2 * x]),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            is_last = __hip_atomic_fetch_add(a.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == splits;
            if (is_last) __hip_atomic_store(a.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!is_last) return;
        const uint64_t *all = reinterpret_cast<const uint64_t *>(a.ws) + static_cast<int64_t>(tile) * splits * (C::E / 2);
        for (uint32_t p = 0; p < splits; ++p) {
            if (p == split) continue;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int e = tid + q * WAVES * 64;
                if (e >= C::E / 4) break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint64_t v = __hip_atomic_load(all + p * (C::E / 2) + 2 * e + x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    sum[q][2 * x] += static_cast<int32_t>(static_cast<uint32_t>(v));
                    sum[q][2 * x + 1] += static_cast<int32_t>(static_cast<uint32_t>(v >> 32));
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = tid + q * WAVES * 64;
        if (e >= C::E / 4) break;
        const int t = e / 64 / NT, u = e / 64 % NT, ln = e % 64;
        const int64_t m = m0 + t * 16 + ln % 16, n = n0 + u * 16 + 4 * (ln / 16);
        if (m >= a.M || n >= a.N) continue;
        const int32_t v[4] = {sum[q][0], sum[q][1], sum[q][2], sum[q][3]};
        write4(a, m, n, v, FUSED ? made_scale[m] : a.x_scales[m]);
    }
}

// Many tokens: bound by the matrix cores. One workgroup to a compute unit walks
// BM x BN tiles; its eight waves (WM x WN of them over the tile, wave w and w + 4 on one
// SIMD) are two groups that take turns: while one multiplies, the other reads its
// fragments from LDS and issues its share of the copies. K goes in ranges of 128
// bytes, whose halves (X rows, W rows) lie in a ring of five LDS slots filled by
// global-to-LDS copies two ranges ahead; the ring runs on across tiles, so the next
// tile's first ranges are on their way while this one is finished.
//   * LDS rows are 128 bytes, the 16-byte chunk c of a row at position c ^ swizzle, so
//     that the 16 rows of a fragment fall on different banks: for X bits 1..3 of the row,
//     for W, whose fragments take rows 8 q + 4 j + t (q, t = 0..3) of a pair of blocks, bits
//     1, 3 and 4. So a lane's results are eight consecutive outputs of one token.
//   * group 0 reads step p of a range in one phase and multiplies in the next, group 1
//     one phase later; a barrier stands between phases, and a range's copies are waited
//     for just before the barrier that opens its first.
// 4096 tokens, K = N = 8192 in 256 x 256 tiles 203 us, 2.7e15 operations a second (the
// library's product 238): the matrix cores work in 65% of the cycles, at 1.9 GHz.
__device__ __forceinline__ int swizzle_x(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swizzle_w(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

// Barrier without a memory fence (the waits are explicit), which nothing moves across.
__device__ __forceinline__ void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

template <int BM, int BN, int WM, int WN>
struct IntTileCfg {
    static constexpr int SLOTS = 5, SLOT = (BM > BN ? BM : BN) * 128;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    static constexpr int NCA = BM / 64, NCB = BN / 64;  // copies of a wave in a range, each of eight rows
    static constexpr int LDS = SLOTS * SLOT;
    static constexpr int GROUP = 4;                     // tile rows that are walked together
    static_assert(WM * WN == 8 && TM % 16 == 0 && TN % 32 == 0 && BM % 64 == 0 && BN % 64 == 0 && LDS <= 160 * 1024, "tile");
};

template <int BM, int BN, int WM, int WN, int OCC>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2 * OCC, 2 * OCC))) void int_tile_kernel(IntArgs a) {
    using C = IntTileCfg<BM, BN, WM, WN>;
    constexpr int FM = C::FM, FN = C::FN, SLOT = C::SLOT;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, fr = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), grp = wave >> 2, wg = wave & 3;
    const int wm = wave / WN, wn = wave % WN;
    const int K = static_cast<int>(a.K), KH = (K + 127) / 128;
    const uint32_t tiles_m = static_cast<uint32_t>((a.M + BM - 1) / BM), tiles_n = static_cast<uint32_t>((a.N + BN - 1) / BN);
    const uint32_t tiles = tiles_m * tiles_n;
    // Tile of an item: ids go round the eight dies, whose items are neighbours, in groups of tile rows,
    // so that operands are shared in a die's L2.
    auto origin = [&](uint32_t item, int64_t &m0, int64_t &n0) {
        const uint32_t at = tiles % 8 == 0 ? item % 8 * (tiles / 8) + item / 8 : item;
        const uint32_t per = C::GROUP * tiles_n, gr = at / per, in = at - gr * per, first = gr * C::GROUP;
        const uint32_t rows = tiles_m - first < C::GROUP ? tiles_m - first : C::GROUP;
        const uint32_t ni = in / rows;
        m0 = static_cast<int64_t>(first + in - ni * rows) * BM;
        n0 = static_cast<int64_t>(ni) * BN;
    };
    auto resources = [&](uint32_t item, __amdgpu_buffer_rsrc_t &rx, __amdgpu_buffer_rsrc_t &rw) {
        if (item >= tiles) {
            rx = rw = buffer_rsrc(a.X, 0);
            return;
        }
        int64_t m0, n0;
        origin(item, m0, n0);
        rx = buffer_rsrc(a.X + m0 * a.K, static_cast<uint32_t>((a.M - m0 < BM ? a.M - m0 : BM) * a.K));
        rw = buffer_rsrc(a.W + n0 * a.K, static_cast<uint32_t>((a.N - n0 < BN ? a.N - n0 : BN) * a.K));
    };
    const int drow = lane >> 3;
    uint32_t xoff[C::NCA], woff[C::NCB];
#pragma unroll
    for (int j = 0; j < C::NCA; ++j) {
        const int row = (grp * (BM / 16) + wg + 4 * j) * 8 + drow;
        xoff[j] = static_cast<uint32_t>(row * K + ((lane & 7) ^ swizzle_x(row)) * 16);
    }
#pragma unroll
    for (int j = 0; j < C::NCB; ++j) {
        const int row = (grp * (BN / 16) + wg + 4 * j) * 8 + drow;
        woff[j] = static_cast<uint32_t>(row * K + ((lane & 7) ^ swizzle_w(row)) * 16);
    }
    auto copy_x = [&](__amdgpu_buffer_rsrc_t r, int T, int slot) {
        if (T == KH - 1 && K % 128 != 0) {  // behind K lies the next row: zeros instead, here, so that W's do not matter
#pragma unroll
            for (int j = 0; j < C::NCA; ++j) {
                const int row = (grp * (BM / 16) + wg + 4 * j) * 8 + drow;
                const uint32_t v = T * 128 + ((lane & 7) ^ swizzle_x(row)) * 16 < K ? xoff[j] : kOutside;
                dma16_buf(r, v, static_cast<uint32_t>(T * 128), lds + slot * SLOT + (grp * (BM / 16) + wg + 4 * j) * 1024);
            }
        } else {
#pragma unroll
            for (int j = 0; j < C::NCA; ++j)
                dma16_buf(r, xoff[j], static_cast<uint32_t>(T * 128), lds + slot * SLOT + (grp * (BM / 16) + wg + 4 * j) * 1024);
        }
    };
    auto copy_w = [&](__amdgpu_buffer_rsrc_t r, int T, int slot) {
#pragma unroll
        for (int j = 0; j < C::NCB; ++j)
            dma16_buf(r, woff[j], static_cast<uint32_t>(T * 128), lds + slot * SLOT + (grp * (BN / 16) + wg + 4 * j) * 1024);
    };
    auto next = [](int slot, int d) { return slot + d >= C::SLOTS ? slot + d - C::SLOTS : slot + d; };
    const int sx = swizzle_x(fr);  // the fragments' first rows are multiples of 16
    auto frag_x = [&](const char *base, int i, int p) {
        return *reinterpret_cast<const i32x4 *>(base + (wm * C::TM + i * 16 + fr) * 128 + (((4 * p + fg) ^ sx) << 4));
    };
    auto frag_w = [&](const char *base, int j, int p) {
        const int row = wn * C::TN + (j >> 1) * 32 + 8 * (fr >> 2) + 4 * (j & 1) + (fr & 3);
        return *reinterpret_cast<const i32x4 *>(base + row * 128 + (((4 * p + fg) ^ swizzle_w(row)) << 4));
    };

    uint32_t item = blockIdx.x;
    __amdgpu_buffer_rsrc_t cx, cw, nx, nw;
    resources(item, cx, cw);
    int s0 = 0;  // slot of the current range's X; its W follows, then the next range's X
    copy_x(cx, 0, 0);
    copy_w(cw, 0, 1);
    copy_x(cx, 1, 2);
    resources(item + gridDim.x, nx, nw);
    wait_vm<C::NCA>();
    barrier_only();
    for (; item < tiles; item += gridDim.x) {
        i32x4 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        auto walk = [&](auto group) {
            constexpr int GRP = decltype(group)::value;
            if (GRP == 1) barrier_only();
            i32x4 xf[FM], wf[FN];
            for (int T = 0; T < KH; ++T) {
                const char *xs = lds + s0 * SLOT, *ws = lds + next(s0, 1) * SLOT;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int i = 0; i < FM; ++i) xf[i] = frag_x(xs, i, p);
#pragma unroll
                    for (int j = 0; j < FN; ++j) wf[j] = frag_w(ws, j, p);
                    if (p == 0) {  // W of the next range, this tile's or the next tile's first
                        if (T + 1 < KH)
                            copy_w(cw, T + 1, next(s0, 3));
                        else
                            copy_w(nw, 0, next(s0, 3));
                    } else {       // X of the one after that
                        if (T + 2 < KH)
                            copy_x(cx, T + 2, next(s0, 4));
                        else
                            copy_x(nx, T + 2 - KH, next(s0, 4));
                    }
                    if (GRP == 1 && p == 1) {
                        wait_vm<C::NCA>();  // the next range has landed (this wave's part)
                        lds_wait_all();     // the next phase refills the slot of X
                    }
                    barrier_only();
                    lds_wait_all();
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j] = mfma16x16x64(wf[j], xf[i], acc[i][j]);
                    if (GRP == 0 && p == 1) wait_vm<C::NCA>();
                    barrier_only();
                }
                s0 = next(s0, 2);
            }
            if (GRP == 0) barrier_only();
        };
        if (grp == 0)
            walk(std::integral_constant<int, 0>{});
        else
            walk(std::integral_constant<int, 1>{});

        int64_t m0, n0;
        origin(item, m0, n0);
        m0 += wm * C::TM + fr;
        n0 += wn * C::TN + 8 * fg;
        // eight consecutive outputs of a token: acc[i][2 j][0 ..], acc[i][2 j + 1][0 ..]
        const bool whole = a.row % 8 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
        float xs[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) xs[i] = a.x_scales[m0 + 16 * i < a.M ? m0 + 16 * i : a.M - 1];
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) {
            const int64_t n = n0 + 32 * j;
            float ws[8], bias[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t col = n + e < a.N ? n + e : a.N - 1;
                ws[e] = a.w_scales[col];
                bias[e] = (a.epi & 1) ? bf16_bits_to_f32(a.bias[col]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int64_t m = m0 + 16 * i;
                if (m >= a.M || n >= a.N) continue;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = scaled(acc[i][2 * j + e / 4][e % 4], xs[i], ws[e]);
                finish(v, a.epi, bias);
                if (whole && n + 8 <= a.N && a.out == OUT_BF16) {
                    u32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = f32_to_bf16_bits(v[2 * e]) | static_cast<uint32_t>(f32_to_bf16_bits(v[2 * e + 1])) << 16;
                    __builtin_nontemporal_store(y, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.Y) + m * a.row + n));
                } else if (whole && n + 8 <= a.N) {
                    f32x4 *y = reinterpret_cast<f32x4 *>(static_cast<float *>(a.Y) + m * a.row + n);
                    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, y);
                    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, y + 1);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (n + e < a.N) store_out(a.Y, a.out, m * a.row + n + e, v[e]);
                }
            }
        }
        cx = nx;
        cw = nw;
        resources(item + 2 * gridDim.x, nx, nw);
    }
    wait_vm<0>();  // the copies for the tile after the last (empty resources) still write LDS
}

#define PROJ_INT_TILE_VARIANTS(X) X(256, 256, 4, 2, 1) X(256, 128, 4, 2, 1) X(128, 128, 4, 2, 2)
#define PROJ_INT_TILE_INST(BM, BN, WM, WN, OCC) template __global__ void int_tile_kernel<BM, BN, WM, WN, OCC>(IntArgs);
PROJ_INT_TILE_VARIANTS(PROJ_INT_TILE_INST)

// K = 0: the sum is empty.
__global__ __launch_bounds__(256) void int_empty_kernel(IntArgs a) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < a.M * a.N; i += static_cast<int64_t>(gridDim.x) * 256) {
        float v[1] = {0.f};
        const float bias[1] = {(a.epi & 1) ? bf16_bits_to_f32(a.bias[i % a.N]) : 0.f};
        finish(v, a.epi, bias);
        store_out(a.Y, a.out, i, v[0]);
    }
}

#define PROJ_INT_STREAM_VARIANTS(X)                                                                       \
    X(1, 1, 8, 512, 5) X(1, 2, 8, 512, 5) X(1, 4, 4, 256, 7) X(2, 2, 8, 512, 4) X(2, 4, 4, 256, 6)        \
    X(4, 2, 4, 256, 6) X(4, 4, 4, 256, 4) X(4, 7, 4, 256, 3) X(6, 2, 4, 256, 5) X(6, 4, 4, 256, 3)        \
    X(8, 2, 4, 256, 4) X(8, 4, 4, 256, 3)
#define PROJ_INT_STREAM_INST(MT, NT, WV, KC, D) template __global__ void int_stream_kernel<MT, NT, WV, KC, D, false>(IntArgs, uint32_t);
PROJ_INT_STREAM_VARIANTS(PROJ_INT_STREAM_INST)
template __global__ void int_stream_kernel<1, 1, 8, 512, 5, true>(IntArgs, uint32_t);
template __global__ void int_stream_kernel<1, 2, 8, 512, 5, true>(IntArgs, uint32_t);

#ifndef __HIP_DEVICE_COMPILE__
template <int LANES, int R>
static hipError_t launch_rows(const RowsArgs &a, hipStream_t st) {
    const int64_t groups = (a.M + 256 / LANES - 1) / (256 / LANES), most = most_groups(256);
    const int vec = a.stride % 8 == 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0;
    hipLaunchKernelGGL((quantize_rows_kernel<LANES, R>), dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(256), 0, st, a,
                       vec);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(const RowsArgs &a, hipStream_t st) {
    if (a.K <= 512) return launch_rows<64, 1>(a, st);
    if (a.K <= 1024) return launch_rows<64, 2>(a, st);
    if (a.K <= 2048) return launch_rows<256, 1>(a, st);
    if (a.K <= 4096) return launch_rows<256, 2>(a, st);
    if (a.K <= 8192) return launch_rows<256, 4>(a, st);
    return a.K <= 16384 ? launch_rows<256, 8>(a, st) : launch_rows<256, 0>(a, st);
}

// How far K is split: while there are fewer tiles than compute units, in shares of 4096 at least (one token, K8192
// N1024: two of them 7.4 us, four 7.7, one 7.5; 16 tokens, K16384 N512: 8.2, 9.3, 10.6), as far as the workspace
// holds the sums.
static int64_t stream_splits(const IntArgs &a, int mt, int nt) {
    const int64_t tiles = (a.N + 16 * nt - 1) / (16 * nt) * ((a.M + 16 * mt - 1) / (16 * mt));
    int64_t splits = a.cus / tiles;
    if (splits > a.K / 4096) splits = a.K / 4096;
    const int64_t room = static_cast<int64_t>(a.ws_bytes / (mt * nt * 1024)) / tiles;
    if (splits > room) splits = room;
    return tiles > a.ncounters || splits < 1 ? 1 : splits;
}

template <int MT, int NT, int WAVES, int KC, int D, bool FUSED = false>
static hipError_t launch_int_stream(const IntArgs &a, hipStream_t st) {
    const int64_t tiles = (a.N + 16 * NT - 1) / (16 * NT) * ((a.M + 16 * MT - 1) / (16 * MT)), splits = stream_splits(a, MT, NT);
    hipLaunchKernelGGL((int_stream_kernel<MT, NT, WAVES, KC, D, FUSED>), dim3(static_cast<unsigned>(tiles * splits)), dim3(WAVES * 64), 0, st, a,
                       static_cast<uint32_t>(splits));
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int OCC>
static hipError_t launch_int_tile(const IntArgs &a, hipStream_t st) {
    const int64_t tiles = (a.M + BM - 1) / BM * ((a.N + BN - 1) / BN), most = OCC * static_cast<int64_t>(a.cus);
    hipLaunchKernelGGL((int_tile_kernel<BM, BN, WM, WN, OCC>), dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(512), 0,
                       st, a);
    return hipGetLastError();
}

bool int_fuses(int64_t M, int64_t N, int64_t K) {
    return K > 0 && M <= kFusedRows && K <= kFusedK && (N + 15) / 16 <= most_groups(256);
}

hipError_t launch_int_fused(const IntArgs &a, hipStream_t st) {
    return (a.N + 31) / 32 >= a.cus ? launch_int_stream<1, 2, 8, 512, 5, true>(a, st) : launch_int_stream<1, 1, 8, 512, 5, true>(a, st);
}

hipError_t launch_int(const IntArgs &a, hipStream_t st) {
    const int64_t most = most_groups(256);
    if (a.K == 0) {
        const int64_t groups = (a.M * a.N + 255) / 256;
        hipLaunchKernelGGL(int_empty_kernel, dim3(static_cast<unsigned>(groups < most ? groups : most)), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    // more tiles than one launch can have workgroups for, however small they are: rows, then columns, in pieces
    if ((a.M + 15) / 16 * ((a.N + 15) / 16) > most) {
        IntArgs x = a, y = a;
        const int64_t size = a.out == OUT_F32 ? 4 : 2;
        if (a.M > 16) {
            x.M = (a.M / 2 + 15) / 16 * 16;
            y.M = a.M - x.M;
            y.X = a.X + x.M * a.K;
            y.x_scales = a.x_scales + x.M;
            y.Y = static_cast<char *>(a.Y) + x.M * a.row * size;
        } else {
            x.N = (a.N / 2 + 15) / 16 * 16;
            y.N = a.N - x.N;
            y.W = a.W + x.N * a.K;
            y.w_scales = a.w_scales + x.N;
            y.bias = a.bias ? a.bias + x.N : nullptr;
            y.Y = static_cast<char *>(a.Y) + x.N * size;
        }
        const hipError_t e = launch_int(x, st);
        return e != hipSuccess ? e : launch_int(y, st);
    }
    // The kernel that is expected to be done first. Its time goes in rounds of one workgroup to a compute unit, each
    // of a part that does not depend on K and one that does; in units of 0.15 us, K = 8192: streaming 40 and one for
    // each row of X or W that a workgroup reads, a join of splits 10 and 4 for 256 outputs (M128 N8192 in 128 x 32 30 us,
    // M64 N28672 in 64 x 112 48, M64 N8192 in 64 x 32 20.5, in two splits of 64 x 64 27.8), tiles 20
    // and 380 (128 x 128; two of them to a unit 513), 420 (256 x 128), 540 (256 x 256) (M1024 N8192 in 256 x 128
    // 70 us, the others 80 and 84; M512 N28672 in 256 x 256 117, the others 141 and 157).
    const double deep = static_cast<double>(a.K) / 8192;
    hipError_t (*best)(const IntArgs &, hipStream_t) = nullptr;
    double least = 0;
    auto offer = [&](double cost, hipError_t (*launch)(const IntArgs &, hipStream_t)) {
        if (!best || cost < least) {
            best = launch;
            least = cost;
        }
    };
    auto rounds = [&](int bm, int bn, int64_t units) { return ((a.M + bm - 1) / bm * ((a.N + bn - 1) / bn) + units - 1) / units; };
    const int64_t cus = a.cus;
    if (a.K > 128) {  // tiles look two ranges of K ahead
        const int64_t r = rounds(128, 128, cus);
        offer(r == 1 ? 20 + 380 * deep : (r + 1) / 2 * (20 + 513 * deep), launch_int_tile<128, 128, 4, 2, 2>);
        offer(rounds(256, 128, cus) * (20 + 420 * deep), launch_int_tile<256, 128, 4, 2, 1>);
        offer(rounds(256, 256, cus) * (20 + 540 * deep), launch_int_tile<256, 256, 4, 2, 1>);
    }
#define PROJ_INT_STREAM_OFFER(MT, NT, WV, KC, D)                                                                  \
    if (const int64_t r = rounds(16 * MT, 16 * NT, cus), s = stream_splits(a, MT, NT); r * cus <= most - cus) \
        offer(r * (40 + (s > 1 ? 10 + 4 * MT * NT : 0) + 16 * (MT + NT) * deep / s), launch_int_stream<MT, NT, WV, KC, D>);
    PROJ_INT_STREAM_VARIANTS(PROJ_INT_STREAM_OFFER)
    return best ? best(a, st) : hipErrorInvalidValue;
}
#endif

}  // namespace proj
