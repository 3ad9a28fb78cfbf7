// prefix.hip -- attention of one new token for each sequence of a batch whose
// first tokens are the same pages for all: the shared tokens' part.
//
// For a key-value head, the rows of all sequences and query heads that read it
// (B * per of them) meet each shared token once, as a product of two matrices,
//     w[t][r] = scale <q[r], k[t]>,  m = max_t w,  l = sum_t exp(w - m),
//     o[r][:] = sum_t exp(w[t][r] - m) v[t][:],
// in parts of the prefix that join with the parts of each sequence's own tokens
// (attend.hip). A row sees the tokens lo <= t < hi of the prefix, by its
// sequence's length and window.
//
// A workgroup is four waves on (key-value head, part, group of 128 rows), 32 rows to
// a wave. Keys and values go into LDS in bf16 whatever the cache's type, 64 tokens
// to a step, those of the next steps on their way while this one is computed. Waves
// without rows only copy: with 8 rows in all, four waves on different tokens, each with
// a part of its own, took 87 us a call for 65536 tokens where these took 68.
//   * w: v_mfma_f32_32x32x16_bf16 with A = 32 tokens of K and B = 32 rows of q,
//     held for the whole call. A lane of the result has row l % 32 and tokens
//     8 (v / 4) + 4 (l / 32) + v % 4. The sums start at minus the row's running
//     maximum, so what comes out is w - m without a subtraction.
//   * o: A = V transposed (32 elements of the head x 16 tokens), B = the
//     probabilities as they lie: slot 4 y + i of lane half h is token
//     16 s + 8 y + 4 h + i of step s. V follows by being read in that order with
//     LDS's transposing loads.
//   * vector instructions and matrix ones take about the same time here, so the
//     former are what counts. Logits stay in units of <q, k>, and the scale comes in
//     the exponent; the maximum moves only when a logit passes it by more than 5
//     (a factor of 148); the sign of the scale is put into q. Where the scale in base 2
//     passes the range of a float, differences from the maximum are first multiplied by
//     a power of two.
//   * in LDS, tokens lie in sixteens, within those the 16-byte chunks of a token in
//     fours: a lane copies chunks of one token only, whose address it works out
//     once, and every read below has its place in its offset. Position
//     (c % 4) ^ (token / 4 % 4) of a four holds chunk c: 16 tokens at one chunk, and
//     four chunks of 4 tokens, fall on different banks.
//   * a probability enters as three bf16 terms, which together are its 24 bits, whatever
//     the results' type, as in attend.hip. Two are faster (a call of 256 sequences behind
//     32768 tokens 502 us instead of 586, of 64 behind 8192 80 instead of 84.5), but a few
//     of a thousand bf16 results are then not the fp32 ones rounded.
// 256 sequences of 64 query heads behind 32768 tokens (8 heads of 128, bf16) 480 to 524 us
// for the prefix, 0.52 to 0.57e15 operations a second of the formula's; the matrix cores
// work in 58% of the cycles, vector instructions issue in 52%. Every token of the prefix is
// read, whatever lengths and a window leave of it.
#include <cmath>
#include <type_traits>

#include "layer.hpp"
#include "parts.hpp"

namespace proj {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

namespace {

constexpr int kTerms = 3;  // bf16 terms of a probability
constexpr float kLowest = -0x1.fffffep127f;
constexpr float kLog2e = 1.4426950408889634f;

// Four e4m3 bytes -> bf16, exact; two 32-bit words of pairs.
__device__ __forceinline__ u32x2 fp8x4_to_bf16(uint32_t w) {
    u32x2 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    return r;
}

// Two floats -> their bf16 halves, lo first: cut, or rounded to nearest even.
__device__ __forceinline__ uint32_t cut2(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
    typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

template <int D>
struct PrefixCfg {
    static constexpr int SUB = 2, TOK = 32 * SUB;         // tiles of 32 tokens of a step, its tokens
    static constexpr int U = TOK / 64;                    // of them copied by a lane
    static constexpr int NC = D / 8, CH = (NC + 3) / 4;   // 16-byte chunks of a token, fours of them
    static constexpr int KS = D / 16, DT = CH;            // steps of the first product, tiles of the second
    static constexpr int TILE = TOK * CH * 64;            // bytes of a step's keys (or values)
    static constexpr int UT = D / 16, UI = (UT + 3) / 4;  // 16-byte loads of a token in 8 bits, of a lane
    static_assert(4 * TILE <= 128 * 1024, "two steps in LDS");
};

}  // namespace

template <int D, bool FP8>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void prefix_kernel(PrefixArgs p) {
    using C = PrefixCfg<D>;
    const AttendArgs &a = p.a;
    __shared__ __attribute__((aligned(16))) char lds[4 * C::TILE];
    __shared__ int bad[4];  // a page of the step is outside the cache; by step % 4
    __shared__ uint32_t again[4];  // rows of each wave whose sums are not finite
    static_assert(4 * C::TILE >= rows_again_lds(D), "room for rows_again");

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // workgroup -> (head, part, group of rows): those of one head and part read
    // the same keys and values and go to one die, ids going round the eight dies
    const uint32_t chunks = static_cast<uint32_t>(p.chunks), die = blockIdx.x % 8, local = blockIdx.x / 8;
    const uint32_t pair = local / chunks * 8 + die, chunk = local % chunks;
    const uint32_t parts = static_cast<uint32_t>(a.prefix_parts);
    if (pair >= static_cast<uint32_t>(a.c.heads) * parts) return;
    const int h = static_cast<int>(pair / parts), part = static_cast<int>(pair % parts);
    const int per = a.q_heads / a.c.heads;
    const int64_t first = part * p.part, last = a.prefix < first + p.part ? a.prefix : first + p.part;
    const int tokens = static_cast<int>(last - first), steps = (tokens + C::TOK - 1) / C::TOK;

    // this lane's row, and the tokens that it sees, counted from the part's first
    const int64_t rows = a.B * per, r = (static_cast<int64_t>(chunk) * 4 + wave) * 32 + c32;
    const int64_t rr = r < rows ? r : rows - 1, b = rr / per, hq = rr % per;
    const int64_t n = a.lengths[b];
    int lo = 0, hi = 0;
    if (n > 0 && n <= a.max_len && r < rows) {
        const int64_t low = a.window > 0 && n > a.window ? n - a.window : 0;
        lo = static_cast<int>((low < first ? first : low < last ? low : last) - first);
        hi = static_cast<int>((n < first ? first : n < last ? n : last) - first);
    }
    const bool none = hi <= lo;  // a row that sees nothing here: computed with the others, and dropped
    // logits are to_logit up <q, k>, q with the scale's sign (and 0 times it, with the scale 1, for a scale of zero)
    const float to_logit = p.to_logit, c = to_logit * kLog2e, enough = 5.f / to_logit;
    const bool far = p.up != 1.f;
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 q[C::KS];
#pragma unroll
    for (int i = 0; i < C::KS; ++i) {
        u32x4 w = __builtin_bit_cast(u32x4, load16(a.q + b * a.q_stride + (static_cast<int64_t>(h) * per + hq) * D + 16 * i + 8 * half));
        w ^= flip;
        q[i] = __builtin_bit_cast(bf16x8, w);
    }
    if (__builtin_expect(a.scale == 0.f, 0))
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
            u32x4 w = __builtin_bit_cast(u32x4, q[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e)  // NaN where infinite or no number
                w[e] = ((w[e] & 0x7f80u) == 0x7f80u ? 0x7fc0u : 0u) | ((w[e] & 0x7f800000u) == 0x7f800000u ? 0x7fc00000u : 0u);
            q[i] = __builtin_bit_cast(bf16x8, w);
        }
    f32x16 o[C::DT], negm;  // negm: minus the running maximum, from which a sum starts
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        negm[v] = 0.f;
#pragma unroll
        for (int i = 0; i < C::DT; ++i) o[i][v] = 0.f;
    }
    // the maximum moves for a logit this far above it: any, before the first
    float above = -__builtin_inff(), l = 0.f;

    const int64_t kb_bytes = h * a.c.kh, vb_bytes = h * a.c.vh;
    constexpr int SIZE = FP8 ? 1 : 2;
    const char *kb = static_cast<const char *>(a.c.k) + kb_bytes * SIZE, *vb = static_cast<const char *>(a.c.v) + vb_bytes * SIZE;
    const int64_t place_mask = (int64_t{1} << a.c.page_shift) - 1;
    u32x4 kr[C::U][C::UI], vr[C::U][C::UI];  // 8-bit keys and values on their way
    int32_t kpage[C::U], vpage[C::U];        // pages of the lane's tokens of the steps that are copied next

    // the lane's token of a step (behind the part's end: its last, masked later)
    auto token = [&](int step, int u) -> int64_t {
        const int t = step * C::TOK + (wave * C::U + u) * 16 + lane / 4;
        return first + (t < tokens ? t : tokens - 1);
    };
    auto find_pages = [&](int step, int32_t (&page)[C::U]) {
#pragma unroll
        for (int u = 0; u < C::U; ++u) page[u] = p.pages[token(step, u) >> a.c.page_shift];
    };
    // Starts the copies of a step's keys or values, whose pages are known; nothing is read through a wrong one.
    auto copy = [&](int step, const int32_t (&page)[C::U], const char *from, int64_t page_stride, int64_t token_stride, char *to,
                    u32x4 (&reg)[C::U][C::UI]) {
#pragma unroll
        for (int u = 0; u < C::U; ++u) {
            const bool ok = page[u] >= 0 && page[u] < a.c.pages;
            if (!ok) bad[step % 4] = 1;
            const char *at = from + ((ok ? page[u] : 0) * page_stride + (token(step, u) & place_mask) * token_stride) * SIZE;
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < C::UI; ++i) {
                    const int x = lane % 4 + 4 * i < C::UT ? lane % 4 + 4 * i : C::UT - 1;
                    reg[u][i] = *reinterpret_cast<const u32x4 *>(at + 16 * x);
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::CH; ++i) {
                    int x = 4 * i + ((lane % 4) ^ (lane >> 4));
                    if (C::NC % 4 != 0 && x >= C::NC) x = C::NC - 1;
                    dma16(at + 16 * x, to + ((wave * C::U + u) * C::CH + i) * 1024);
                }
            }
        }
    };
    auto copy_k = [&](int step) { copy(step, kpage, kb, a.c.kp, a.c.kt, lds + (step & 1) * 2 * C::TILE, kr); };
    auto copy_v = [&](int step) { copy(step, vpage, vb, a.c.vp, a.c.vt, lds + (step & 1) * 2 * C::TILE + C::TILE, vr); };
    // and ends them: 8-bit ones are widened on their way into LDS
    auto land = [&](const u32x4 (&reg)[C::U][C::UI], char *to) {
        if constexpr (FP8) {
#pragma unroll
            for (int u = 0; u < C::U; ++u)
#pragma unroll
                for (int i = 0; i < C::UI; ++i)
                    if (C::UT % 4 == 0 || lane % 4 + 4 * i < C::UT)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = 2 * (lane % 4 + 4 * i) + e;
                            const u32x2 w0 = fp8x4_to_bf16(reg[u][i][2 * e]), w1 = fp8x4_to_bf16(reg[u][i][2 * e + 1]);
                            *reinterpret_cast<u32x4 *>(to + ((wave * C::U + u) * C::CH + ch / 4) * 1024 + lane / 4 * 64 +
                                                       ((ch % 4) ^ (lane >> 4)) * 16) = u32x4{w0[0], w0[1], w1[0], w1[1]};
                        }
        }
    };
    auto land_k = [&](int step) { land(kr, lds + (step & 1) * 2 * C::TILE); };
    auto land_v = [&](int step) { land(vr, lds + (step & 1) * 2 * C::TILE + C::TILE); };
    // The page of step + 1's tokens serves its values now and served its keys a step ago.
    auto next_pages = [&](int step) {
#pragma unroll
        for (int u = 0; u < C::U; ++u) vpage[u] = kpage[u];
        if (step < steps) find_pages(step, kpage);
    };

    // where this lane's pieces lie: chunk 2 i + half of token c32 (i even, i odd), and 4 elements of a V row for
    // each of two rows eight apart
    int kat[2], vat[2];
    // Zero, hidden from the compiler: where it knows the reads' places it keeps many of them in registers, 85 more
    // than there are.
    int row0 = 0;
    asm volatile("" : "+s"(row0));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        kat[x] = ((row0 + c32) / 16 * C::CH) * 1024 + c16 * 64 + (((2 * x + half) ^ (c16 / 4)) * 16);
        const int row = 8 * x + 4 * half + c16 / 4, ch = 2 * ((lane >> 4) & 1) + (c16 & 3) / 2;
        vat[x] = (row0 / 16 * C::CH) * 1024 + row * 64 + ((ch ^ (row / 4 % 4)) * 16) + (c16 & 1) * 8;
    }

    // Sums of a step, started at minus the maximum.
    f32x16 s[C::SUB];
    auto multiply = [&](const char *kt) {
#pragma unroll
        for (int x = 0; x < C::SUB; ++x) {
#pragma unroll
            for (int i = 0; i < C::KS; ++i) {
                const bf16x8 k = *reinterpret_cast<const bf16x8 *>(kt + kat[i % 2] + x * 2 * C::CH * 1024 + i / 2 * 1024);
                s[x] = mfma32x32x16(k, q[i], i == 0 ? negm : s[x]);
            }
        }
    };
    const bool idle = __all(none);  // the wave only copies
    if (a.c.pages == 0) {  // no memory: whatever a row sees is outside the cache
        above = none ? above : 0.f;
        l = none ? 0.f : __builtin_nanf("");
    } else if (steps > 0) {
        if (tid < 4) bad[tid] = 0;
        __syncthreads();
        find_pages(0, kpage);
        copy_k(0);
        next_pages(1);
        copy_v(0);
        land_k(0);
        if (steps > 1) copy_k(1);
        next_pages(2);
        land_v(0);
        if (steps > 1) land_k(1);
        wait_vm<0>();
        __syncthreads();
        if (!idle) multiply(lds);
        __syncthreads();  // the keys of the step after next go where these are
    }
    // In a step: the copies of the next one's values and the keys of the one after it start, the sums become
    // probabilities, and matrix operations follow all together, this step's values and the next one's keys: so one
    // wave of a SIMD has its vector instructions while the other has these.
    for (int step = 0; step < steps && a.c.pages > 0; ++step) {
        const bool any_bad = bad[step % 4] != 0;
        if (tid == 0) bad[(step + 3) % 4] = 0;  // read a step ago, written in the next
        if (step + 1 < steps) copy_v(step + 1);
        if (step + 2 < steps) copy_k(step + 2);
        next_pages(step + 3);
        const int t0 = step * C::TOK + row0;
        if (!idle) {
            const bool whole = __all((lo <= t0 && hi >= t0 + 32 * C::SUB) || none) && t0 + 32 * C::SUB <= tokens && !any_bad && !far;
            if (!whole) {
                if (far)
#pragma unroll
                    for (int x = 0; x < C::SUB; ++x) s[x] *= p.up;
#pragma unroll
                for (int x = 0; x < C::SUB; ++x)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int t = t0 + 32 * x + 8 * (v / 4) + 4 * half + v % 4;
                        if (t < lo || t >= hi) {
                            s[x][v] = -__builtin_inff();
                        } else if (any_bad) {
                            const int32_t pg = p.pages[(first + t) >> a.c.page_shift];
                            if (pg < 0 || pg >= a.c.pages) s[x][v] = __builtin_nanf("");
                        }
                    }
            }
            float most = s[0][0];
#pragma unroll
            for (int x = 0; x < C::SUB; ++x)
#pragma unroll
                for (int v = 0; v < 16; ++v) most = fmaxf(most, s[x][v]);
            if (__any(most > above)) {
                most = fmaxf(most, __shfl_xor(most, 32, 64));
                const bool moves = most > above;
                const float by = moves ? most : 0.f, f = above < 0.f ? 1.f : __builtin_amdgcn_exp2f(-by * c);
                if (moves) above = enough;
                l *= f;
#pragma unroll
                for (int i = 0; i < C::DT; ++i) o[i] *= f;
                negm -= by * p.down;
#pragma unroll
                for (int x = 0; x < C::SUB; ++x) s[x] -= by;
            }
            bf16x8 prob[C::SUB][kTerms][2];
#pragma unroll
            for (int x = 0; x < C::SUB; ++x) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t bits[kTerms][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float p0 = __builtin_amdgcn_exp2f(s[x][8 * y + 2 * i] * c), p1 = __builtin_amdgcn_exp2f(s[x][8 * y + 2 * i + 1] * c);
                        l += p0;
                        l += p1;
#pragma unroll
                        for (int k = 0; k < kTerms; ++k) {
                            if (k + 1 == kTerms) {
                                bits[k][i] = round2(p0, p1);
                            } else {
                                bits[k][i] = cut2(p0, p1);
                                p0 -= __uint_as_float(__float_as_uint(p0) & 0xffff0000u);
                                p1 -= __uint_as_float(__float_as_uint(p1) & 0xffff0000u);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kTerms; ++k)
                        prob[x][k][y] = __builtin_bit_cast(bf16x8, u32x4{bits[k][0], bits[k][1], bits[k][2], bits[k][3]});
                }
            }
            const char *vt = lds + (step & 1) * 2 * C::TILE + C::TILE;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < C::SUB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int i = 0; i < C::DT; ++i) {
                        s16x4 z[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            z[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (__attribute__((address_space(3))) s16x4 *)(vt + vat[j] + (2 * x + y) * C::CH * 1024 + i * 1024));
                        const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(z[0], z[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                        for (int k = 0; k < kTerms; ++k) o[i] = mfma32x32x16(v, prob[x][k][y], o[i]);
                    }
            // the last step's are of no use, but a branch would part the matrix operations
            multiply(lds + ((step + 1) & 1) * 2 * C::TILE);
            // LDS reads eight ahead of the operations that need them
            constexpr int READS = C::SUB * (4 * C::DT + C::KS), PRODUCTS = C::SUB * (2 * C::DT * kTerms + C::KS), AHEAD = 8;
            __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
            for (int i = 0; i < READS - AHEAD; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS - READS + AHEAD, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // an 8-bit step's keys go where this step's were: every wave has multiplied those a step ago
        if (step + 1 < steps) land_v(step + 1);
        if (step + 2 < steps) land_k(step + 2);
        wait_vm<0>();
        __syncthreads();
    }
    l += __shfl_xor(l, 32, 64);
    const float top = -negm[0];

    // A sum that is not finite though its probabilities are: a value met a
    // probability of zero (a token that another row sees) or a vanished term, or
    // sums passed the largest float. Such rows are worked out again, below.
    float check = 0.f;
#pragma unroll
    for (int i = 0; i < C::DT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            if (32 * i + 8 * (v / 4) + 4 * half < D) check += o[i][v] * 0.f;
    check += __shfl_xor(check, 32, 64);
    const uint64_t marks = __ballot(!(check == 0.f) && l == l && !none);  // infinity times 0 is NaN
    if (lane == 0) again[wave] = static_cast<uint32_t>(marks);

    float m = above < 0.f ? kLowest : top * p.up * to_logit;
    if (none) {
        m = kLowest;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < C::DT; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[i][v] = 0.f;
    }
    auto part_of = [&](int64_t b, int64_t hq) {
        return a.ws + ((b * a.q_heads + static_cast<int64_t>(h) * per + hq) * (a.parts + a.prefix_parts) + a.parts + part) * (D + 4);
    };
    if (r < rows) {
        float *to = part_of(b, hq);
#pragma unroll
        for (int i = 0; i < C::DT; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int d = 32 * i + 8 * y + 4 * half;
                if (d < D) *reinterpret_cast<f32x4 *>(to + d) = f32x4{o[i][4 * y], o[i][4 * y + 1], o[i][4 * y + 2], o[i][4 * y + 3]};
            }
        if (half == 0) *reinterpret_cast<u32x2 *>(to + D) = u32x2{__float_as_uint(m), __float_as_uint(l)};
    }
    __syncthreads();
    if ((again[0] | again[1] | again[2] | again[3]) == 0) return;
    wait_vm<0>();  // what is stored again has been stored
    rows_again<D, FP8>(
        a.c, p.pages, h, static_cast<double>(a.scale) * a.c.k_scale, again, 4, lds,
        [&](int x) {
            const int64_t at = static_cast<int64_t>(chunk) * 128 + x, bx = at / per, nx = a.lengths[bx];
            const int64_t low = a.window > 0 && nx > a.window ? nx - a.window : 0;
            return RowAgain{a.q + bx * a.q_stride + (static_cast<int64_t>(h) * per + at % per) * D, low > first ? low : first,
                            nx < last ? nx : last};
        },
        [&](int x, int d, const RowMean &y) {
            const int64_t at = static_cast<int64_t>(chunk) * 128 + x;
            float *to = part_of(at / per, at % per);
            to[d] = y.mean;
            if (d < 2) to[D + d] = d == 0 ? y.most : -y.total;
        });
}

#define PROJ_PREFIX_INST(D)                                       \
    template __global__ void prefix_kernel<D, false>(PrefixArgs); \
    template __global__ void prefix_kernel<D, true>(PrefixArgs);
PROJ_PREFIX_INST(64)
PROJ_PREFIX_INST(80)
PROJ_PREFIX_INST(96)
PROJ_PREFIX_INST(128)
PROJ_PREFIX_INST(192)
PROJ_PREFIX_INST(256)

#ifndef __HIP_DEVICE_COMPILE__
template <int D>
static hipError_t enqueue_prefix(const PrefixArgs &p, int64_t grid, hipStream_t st) {
    auto kernel = p.a.c.fp8 ? prefix_kernel<D, true> : prefix_kernel<D, false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int D>
static hipError_t launch_shared_dim(PrefixArgs p, hipStream_t st) {
    AttendArgs &a = p.a;
    const int per = a.q_heads / a.c.heads;
    const int64_t rows = a.B * per, longest = a.max_len > a.prefix ? a.max_len - a.prefix : 0;
    a.chunks = attend_chunks(a);
    const int64_t own_rows = a.B * a.c.heads * a.chunks, most = most_groups(256);
    // room for parts of a row: at least one of its own and one of the prefix
    const int64_t held = static_cast<int64_t>(a.ws_bytes / (sizeof(float) * (D + 4))) / (a.B * a.q_heads);
    p.chunks = static_cast<int>((rows + 127) / 128);
    if (held < 2 || own_rows > most - 7 * a.c.heads * a.chunks || a.B * a.q_heads > most ||
        (static_cast<int64_t>(a.c.heads) + 7) * p.chunks > most) {
        if (a.B == 1) return hipErrorOutOfMemory;
        PrefixArgs x = p;
        x.a.B = a.B / 2;
        const hipError_t e = launch_shared_dim<D>(x, st);
        if (e != hipSuccess) return e;
        x.a = attend_rest(a, x.a.B);
        return launch_shared_dim<D>(x, st);
    }
    // parts of the prefix: two workgroups to a compute unit, none shorter than 128 tokens
    const int64_t pairs = static_cast<int64_t>(a.c.heads) * p.chunks;
    int64_t parts = (2 * static_cast<int64_t>(a.cus) + pairs - 1) / pairs;
    if (parts > (a.prefix + 127) / 128) parts = (a.prefix + 127) / 128;
    if (parts > held - 1) parts = held - 1;
    if (parts < 1) parts = 1;
    p.part = ((a.prefix + parts - 1) / parts + 127) / 128 * 128;
    parts = a.prefix > p.part ? (a.prefix + p.part - 1) / p.part : 1;
    a.prefix_parts = static_cast<int>(parts);
    if (longest > 0) {
        const int64_t room = held - a.prefix_parts, most_parts = (most - 7 * a.c.heads * a.chunks) / own_rows;
        plan_attend(a, longest, room < most_parts ? room : most_parts);
    }
    const int64_t grid = (static_cast<int64_t>(a.c.heads) * parts + 7) / 8 * 8 * p.chunks;
    hipError_t e = enqueue_prefix<D>(p, grid, st);
    if (e == hipSuccess && longest > 0) e = launch_attend_parts(a, st);
    return e != hipSuccess ? e : launch_attend_join(a, st);
}

hipError_t launch_attend_shared(const PrefixArgs &args, hipStream_t st) {
    PrefixArgs p = args;
    // The scales' product, exact in 64 bits, as a float and (where that or its base-2 form may pass the ends of the
    // range) a power of two. Below 2^-240 every finite logit is 0 beside the others, and so it is with that.
    const double f = std::fabs(static_cast<double>(p.a.scale)) * p.a.c.k_scale;
    if (p.a.scale == 0.f) {
        p.to_logit = 1.f;
    } else if (f > 0x1p-100 && f < 0x1p100) {
        p.to_logit = static_cast<float>(f);
    } else {
        const int e = std::ilogb(f) > 120 ? 120 : std::ilogb(f) < -120 ? -120 : std::ilogb(f);
        p.up = std::ldexp(1.f, e);
        p.down = std::ldexp(1.f, -e);
        p.to_logit = static_cast<float>((f < 0x1p-240 ? 0x1p-240 : f) * p.down);
    }
    switch (p.a.c.dim) {
        case 64: return launch_shared_dim<64>(p, st);
        case 80: return launch_shared_dim<80>(p, st);
        case 96: return launch_shared_dim<96>(p, st);
        case 128: return launch_shared_dim<128>(p, st);
        case 192: return launch_shared_dim<192>(p, st);
        case 256: return launch_shared_dim<256>(p, st);
    }
    return hipErrorInvalidValue;
}
#endif

}  // namespace proj
