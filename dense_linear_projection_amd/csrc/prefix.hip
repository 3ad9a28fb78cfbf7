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
// A workgroup is four waves on (key-value head, part, group of rows), WQ of them
// along the rows (32 to a wave) and 4 / WQ along the tokens. Tiles of keys and
// values go through registers into LDS, in bf16 whatever the cache's type, those
// of the next step on their way while this one is computed.
//   * w: v_mfma_f32_32x32x16_bf16 with A = 32 tokens of K and B = 32 rows of q,
//     held for the whole call. A lane of the result has row l % 32 and tokens
//     8 (v / 4) + 4 (l / 32) + v % 4.
//   * o: A = V transposed (32 elements of the head x 16 tokens), B = the
//     probabilities as they lie: slot 4 y + i of lane half h is token
//     16 s + 8 y + 4 h + i of step s. V follows by being read in that order with
//     LDS's transposing loads.
#include <type_traits>

#include "layer.hpp"

namespace proj {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

namespace {

constexpr int kPages = 2048;  // tokens whose pages are staged at once
constexpr float kLowest = -0x1.fffffep127f;
constexpr float kLog2e = 1.4426950408889634f;

// Four e4m3 bytes -> bf16, exact; two 32-bit words of pairs.
__device__ __forceinline__ u32x2 fp8x4_to_bf16(uint32_t w) {
    u32x2 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    return r;
}

__device__ __forceinline__ float exp_above(float x, float most) { return __builtin_amdgcn_exp2f((x - most) * kLog2e); }

// Two floats -> their bf16 halves, lo first: cut, or rounded to nearest even.
__device__ __forceinline__ uint32_t cut2(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
    typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

template <int D, bool FP8, int WQ>
struct PrefixCfg {
    static constexpr int WT = 4 / WQ;                       // waves along the tokens
    static constexpr int SUB = WT == 1 ? 2 : 1;             // tiles of 32 tokens of a wave in a step
    static constexpr int TOK = 32 * WT * SUB;               // tokens of a step
    static constexpr int ROW = 2 * D;                       // bytes of a token in LDS
    static constexpr int NC = ROW / 16;                     // its 16-byte chunks
    static constexpr int UNITS = TOK * D * (FP8 ? 1 : 2) / 16;  // 16-byte loads of a step's keys (or values)
    static constexpr int PER = (UNITS + 255) / 256;         // of them to a thread
    static constexpr int UR = D * (FP8 ? 1 : 2) / 16;       // of them to a token
    static constexpr int TILE = TOK * ROW;
    static constexpr int BUFS = 4 * TILE <= (D <= 128 && WQ > 1 ? 80 : 152) * 1024 ? 2 : 1;
    static constexpr int LDS = BUFS * 2 * TILE;
    static constexpr int KS = D / 16, DT = (D + 31) / 32;
    static constexpr int PERIOD = ROW % 256 == 0 ? 1 : ROW % 128 == 0 ? 2 : ROW % 64 == 0 ? 4 : 8;
    // Where chunk c of row r lies, turned by the row. K: one chunk of 16 rows falls on different banks;
    // V: four chunks of four rows do.
    static __device__ __forceinline__ int place_k(int c, int r) { return (c + r / PERIOD) % NC; }
    static __device__ __forceinline__ int place_v(int c, int r) { return (c + 4 * (r / PERIOD)) % NC; }
};

}  // namespace

template <int D, bool FP8, int WQ, int TERMS>
__global__ __launch_bounds__(256, D <= 128 && WQ > 1 ? 2 : 1) void prefix_kernel(PrefixArgs p) {
    using C = PrefixCfg<D, FP8, WQ>;
    const AttendArgs &a = p.a;
    __shared__ __attribute__((aligned(16))) char lds[C::LDS];
    __shared__ uint32_t pages[kPages + 2];
    __shared__ int bad;  // a page of the chunk is outside the cache

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31, c16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wq = wave % WQ, wt = wave / WQ;
    // workgroup -> (head, part, group of rows): those of one head and part read
    // the same keys and values and go to one die, ids going round the eight dies
    const uint32_t chunks = static_cast<uint32_t>(p.chunks), die = blockIdx.x % 8, local = blockIdx.x / 8;
    const uint32_t pair = local / chunks * 8 + die, chunk = local % chunks;
    const uint32_t parts = static_cast<uint32_t>(a.prefix_parts / C::WT);
    if (pair >= static_cast<uint32_t>(a.c.heads) * parts) return;
    const int h = static_cast<int>(pair / parts), part = static_cast<int>(pair % parts);
    const int per = a.q_heads / a.c.heads;
    const int64_t first = part * p.part, last = a.prefix < first + p.part ? a.prefix : first + p.part;

    // this lane's row, and the tokens that it sees, counted from the part's first
    const int64_t rows = a.B * per, r = (static_cast<int64_t>(chunk) * WQ + wq) * 32 + c32;
    const int64_t rr = r < rows ? r : rows - 1, b = rr / per, hq = rr % per;
    const int64_t n = a.lengths[b];
    int lo = 0, hi = 0;
    if (n > 0 && n <= a.max_len && r < rows) {
        const int64_t low = a.window > 0 && n > a.window ? n - a.window : 0;
        lo = static_cast<int>((low < first ? first : low < last ? low : last) - first);
        hi = static_cast<int>((n < first ? first : n < last ? n : last) - first);
    }
    const bool none = hi <= lo;  // a row that sees nothing here: computed with the others, and dropped
    bf16x8 q[C::KS];
#pragma unroll
    for (int i = 0; i < C::KS; ++i)
        q[i] = load16(a.q + b * a.q_stride + (static_cast<int64_t>(h) * per + hq) * D + 16 * i + 8 * half);
    f32x16 o[C::DT];
#pragma unroll
    for (int i = 0; i < C::DT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[i][v] = 0.f;
    float m = kLowest, l = 0.f;

    const char *kb = static_cast<const char *>(a.c.k) + h * a.c.kh * (FP8 ? 1 : 2);
    const char *vb = static_cast<const char *>(a.c.v) + h * a.c.vh * (FP8 ? 1 : 2);
    const int64_t place_mask = (int64_t{1} << a.c.page_shift) - 1;
    const float to_logit = a.scale * a.c.k_scale;
    u32x4 kr[C::PER], vr[C::PER];

    for (int64_t base = first; base < last; base += kPages) {
        const int64_t end = last < base + kPages ? last : base + kPages;
        const int64_t page0 = base >> a.c.page_shift;
        const int npages = static_cast<int>(((end - 1) >> a.c.page_shift) - page0) + 1;
        const int left = static_cast<int>(end - base), in_page = static_cast<int>(base & place_mask);
        const int steps = (left + C::TOK - 1) / C::TOK;
        __syncthreads();  // the chunk before is done with
        if (tid == 0) bad = 0;
        __syncthreads();
        for (int i = tid; i < npages; i += 256) {
            const int32_t page = p.pages[page0 + i];
            const bool ok = page >= 0 && page < a.c.pages;
            pages[i] = ok ? static_cast<uint32_t>(page) : ~0u;
            if (!ok) bad = 1;
        }
        __syncthreads();
        const bool any_bad = bad != 0;

        // the step's keys and values into registers; nothing is read through a wrong page
        auto load = [&](int step) {
#pragma unroll
            for (int i = 0; i < C::PER; ++i) {
                const int id = i * 256 + tid < C::UNITS ? i * 256 + tid : C::UNITS - 1;
                const int t = step * C::TOK + id / C::UR, at = in_page + (t < left ? t : left - 1);
                const uint32_t page = pages[at >> a.c.page_shift];
                const int64_t place = at & static_cast<int>(place_mask);
                const int64_t ke = static_cast<int64_t>(page) * a.c.kp + place * a.c.kt;
                const int64_t ve = static_cast<int64_t>(page) * a.c.vp + place * a.c.vt;
                kr[i] = vr[i] = u32x4{0u, 0u, 0u, 0u};
                if (page != ~0u) {
                    kr[i] = *reinterpret_cast<const u32x4 *>(kb + (FP8 ? ke : 2 * ke) + id % C::UR * 16);
                    vr[i] = *reinterpret_cast<const u32x4 *>(vb + (FP8 ? ve : 2 * ve) + id % C::UR * 16);
                }
            }
        };
        // and from there into LDS; values past the end are zero there: zero times NaN is not
        auto store = [&](int step, char *kt, char *vt) {
#pragma unroll
            for (int i = 0; i < C::PER; ++i) {
                const int id = i * 256 + tid, row = id / C::UR, u = id % C::UR;
                if (C::UNITS % 256 != 0 && id >= C::UNITS) break;
                if (step * C::TOK + row >= left) vr[i] = u32x4{0u, 0u, 0u, 0u};
                if constexpr (FP8) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const u32x2 k0 = fp8x4_to_bf16(kr[i][2 * x]), k1 = fp8x4_to_bf16(kr[i][2 * x + 1]);
                        const u32x2 v0 = fp8x4_to_bf16(vr[i][2 * x]), v1 = fp8x4_to_bf16(vr[i][2 * x + 1]);
                        *reinterpret_cast<u32x4 *>(kt + row * C::ROW + C::place_k(2 * u + x, row) * 16) = u32x4{k0[0], k0[1], k1[0], k1[1]};
                        *reinterpret_cast<u32x4 *>(vt + row * C::ROW + C::place_v(2 * u + x, row) * 16) = u32x4{v0[0], v0[1], v1[0], v1[1]};
                    }
                } else {
                    *reinterpret_cast<u32x4 *>(kt + row * C::ROW + C::place_k(u, row) * 16) = kr[i];
                    *reinterpret_cast<u32x4 *>(vt + row * C::ROW + C::place_v(u, row) * 16) = vr[i];
                }
            }
        };

        load(0);
        for (int step = 0; step < steps; ++step) {
            char *kt = lds + (step % C::BUFS) * 2 * C::TILE, *vt = kt + C::TILE;
            if (C::BUFS == 1) __syncthreads();  // the step before is done with
            store(step, kt, vt);
            if (step + 1 < steps) load(step + 1);
            __syncthreads();
#pragma unroll
            for (int sub = 0; sub < C::SUB; ++sub) {
                const int row0 = (wt * C::SUB + sub) * 32;                         // the tile in LDS
                const int t0 = static_cast<int>(base - first) + step * C::TOK + row0;  // and in the part
                const int tiles_end = static_cast<int>(base - first) + left;
                if (__all(hi <= t0 || lo >= t0 + 32)) continue;  // no row of the wave sees it
                f32x16 s;
#pragma unroll
                for (int v = 0; v < 16; ++v) s[v] = 0.f;
#pragma unroll
                for (int i = 0; i < C::KS; ++i) {
                    const int row = row0 + c32;
                    const bf16x8 k = *reinterpret_cast<const bf16x8 *>(kt + row * C::ROW + C::place_k(2 * i + half, row) * 16);
                    s = mfma32x32x16(k, q[i], s);
                }
                float w[16], most = kLowest;
                const bool whole = __all((lo <= t0 && hi >= t0 + 32) || none) && t0 + 32 <= tiles_end && !any_bad;
#pragma unroll
                for (int v = 0; v < 16; ++v) w[v] = s[v] * to_logit;
                if (!whole) {
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int t = t0 + 8 * (v / 4) + 4 * half + v % 4;
                        if (t < lo || t >= hi || t >= tiles_end)
                            w[v] = -__builtin_inff();
                        else if (any_bad && pages[(in_page + t - static_cast<int>(base - first)) >> a.c.page_shift] == ~0u)
                            w[v] = __builtin_nanf("");
                    }
                }
#pragma unroll
                for (int v = 0; v < 16; ++v) most = fmaxf(most, w[v]);
                if (__any(most > m + 5.f)) {
                    most = fmaxf(fmaxf(most, __shfl_xor(most, 32, 64)), m);
                    const float f = exp_above(m, most);
                    m = most;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < C::DT; ++i) o[i] *= f;
                }
                bf16x8 prob[TERMS][2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t bits[TERMS][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float p0 = exp_above(w[8 * x + 2 * i], m), p1 = exp_above(w[8 * x + 2 * i + 1], m);
                        l += p0 + p1;
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) {
                            if (k + 1 == TERMS) {
                                bits[k][i] = round2(p0, p1);
                            } else {
                                bits[k][i] = cut2(p0, p1);
                                p0 -= __uint_as_float(__float_as_uint(p0) & 0xffff0000u);
                                p1 -= __uint_as_float(__float_as_uint(p1) & 0xffff0000u);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < TERMS; ++k)
                        prob[k][x] = __builtin_bit_cast(bf16x8, u32x4{bits[k][0], bits[k][1], bits[k][2], bits[k][3]});
                }
#pragma unroll
                for (int i = 0; i < C::DT; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s16x4 y[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int row = row0 + 16 * x + 8 * j + 4 * half + c16 / 4;
                            const int chunk_v = 4 * i + 2 * ((lane >> 4) & 1) + (c16 & 3) / 2;  // past the head: any other's
                            y[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (__attribute__((address_space(3))) s16x4 *)(vt + row * C::ROW + C::place_v(chunk_v, row) * 16 + (c16 & 1) * 8));
                        }
                        const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) o[i] = mfma32x32x16(v, prob[k][x], o[i]);
                    }
            }
        }
    }
    l += __shfl_xor(l, 32, 64);

    // A sum that is not finite though its probabilities are: a value met a
    // probability of zero (a token that another row sees) or a vanished term.
    // Such rows are worked out again from the definition, a token at a time,
    // taking nothing from where the probability is zero.
    float check = 0.f;
#pragma unroll
    for (int i = 0; i < C::DT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            if (32 * i + 8 * (v / 4) + 4 * half < D) check += o[i][v] * 0.f;
    check += __shfl_xor(check, 32, 64);  // a row's two lanes go together: they exchange halves of its logits
    const bool again = !(check == 0.f) && l == l && !none;  // infinity times 0 is NaN
    if (__any(again)) {
        if (again)
#pragma unroll
            for (int i = 0; i < C::DT; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) o[i][v] = 0.f;
#pragma unroll 1
        for (int64_t t = first; t < last; ++t) {
            const int at = static_cast<int>(t - first);
            if (C::WT > 1 && at % kPages / 32 % C::WT != wt) continue;  // another wave's token
            const int32_t page = p.pages[t >> a.c.page_shift];
            if (page < 0 || page >= a.c.pages) continue;  // those that see it are NaN already
            const int64_t ke = page * a.c.kp + (t & place_mask) * a.c.kt, ve = page * a.c.vp + (t & place_mask) * a.c.vt;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < C::KS; ++i) {
                const u32x4 qb = __builtin_bit_cast(u32x4, q[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t x = ke + 16 * i + 8 * half + e;
                    const float k = FP8 ? __builtin_amdgcn_cvt_f32_fp8(reinterpret_cast<const uint8_t *>(kb)[x], 0)
                                        : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(kb)[x]);
                    dot = __builtin_fmaf(k, __uint_as_float(e % 2 ? qb[e / 2] & 0xffff0000u : qb[e / 2] << 16), dot);
                }
            }
            dot += __shfl_xor(dot, 32, 64);
            const float prob = at >= lo && at < hi ? exp_above(dot * to_logit, m) : 0.f;
            if (!again || prob == 0.f) continue;
#pragma unroll
            for (int i = 0; i < C::DT; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int d = 32 * i + 8 * (v / 4) + 4 * half + v % 4;
                    if (d >= D) continue;
                    const float x = FP8 ? __builtin_amdgcn_cvt_f32_fp8(reinterpret_cast<const uint8_t *>(vb)[ve + d], 0)
                                        : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(vb)[ve + d]);
                    o[i][v] = __builtin_fmaf(prob, x, o[i][v]);
                }
        }
    }

    if (none) {
        m = kLowest;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < C::DT; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[i][v] = 0.f;
    }
    if (r >= rows) return;
    const int64_t row = b * a.q_heads + static_cast<int64_t>(h) * per + hq;
    float *to = a.ws + (row * (a.parts + a.prefix_parts) + a.parts + part * C::WT + wt) * (D + 4);
#pragma unroll
    for (int i = 0; i < C::DT; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int d = 32 * i + 8 * y + 4 * half;
            if (d < D) *reinterpret_cast<f32x4 *>(to + d) = f32x4{o[i][4 * y], o[i][4 * y + 1], o[i][4 * y + 2], o[i][4 * y + 3]};
        }
    if (half == 0) *reinterpret_cast<u32x2 *>(to + D) = u32x2{__float_as_uint(m), __float_as_uint(l)};
}

#define PROJ_PREFIX_WQ(D, WQ)                                              \
    template __global__ void prefix_kernel<D, false, WQ, 2>(PrefixArgs); \
    template __global__ void prefix_kernel<D, false, WQ, 3>(PrefixArgs); \
    template __global__ void prefix_kernel<D, true, WQ, 2>(PrefixArgs);  \
    template __global__ void prefix_kernel<D, true, WQ, 3>(PrefixArgs);
#define PROJ_PREFIX_INST(D) \
    PROJ_PREFIX_WQ(D, 1)    \
    PROJ_PREFIX_WQ(D, 4)
PROJ_PREFIX_INST(64)
PROJ_PREFIX_INST(80)
PROJ_PREFIX_INST(96)
PROJ_PREFIX_INST(128)
PROJ_PREFIX_INST(192)
PROJ_PREFIX_INST(256)

#ifndef __HIP_DEVICE_COMPILE__
template <int D, int WQ>
static hipError_t enqueue_prefix(const PrefixArgs &p, int64_t grid, hipStream_t st) {
    auto kernel = p.a.c.fp8 ? (p.a.out_dtype == OUT_F32 ? prefix_kernel<D, true, WQ, 3> : prefix_kernel<D, true, WQ, 2>)
                            : (p.a.out_dtype == OUT_F32 ? prefix_kernel<D, false, WQ, 3> : prefix_kernel<D, false, WQ, 2>);
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
    // the four waves along the tokens where one has all the rows (each then has a part of its own)
    const int wq = rows <= 32 && held >= 5 ? 1 : 4, wt = 4 / wq;
    p.chunks = static_cast<int>((rows + 32 * wq - 1) / (32 * wq));
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
    // parts of the prefix: two workgroups to a compute unit, none shorter than 256 tokens
    const int64_t pairs = static_cast<int64_t>(a.c.heads) * p.chunks;
    int64_t parts = (2 * static_cast<int64_t>(a.cus) + pairs - 1) / pairs;
    if (parts > (a.prefix + 255) / 256) parts = (a.prefix + 255) / 256;
    if (parts > (held - 1) / wt) parts = (held - 1) / wt;
    if (parts < 1) parts = 1;
    p.part = ((a.prefix + parts - 1) / parts + 127) / 128 * 128;
    parts = a.prefix > p.part ? (a.prefix + p.part - 1) / p.part : 1;
    a.prefix_parts = static_cast<int>(parts * wt);
    if (longest > 0) {
        const int64_t room = held - a.prefix_parts, most_parts = (most - 7 * a.c.heads * a.chunks) / own_rows;
        plan_attend(a, longest, room < most_parts ? room : most_parts);
    }
    const int64_t grid = (static_cast<int64_t>(a.c.heads) * parts + 7) / 8 * 8 * p.chunks;
    hipError_t e = wq == 1 ? enqueue_prefix<D, 1>(p, grid, st) : enqueue_prefix<D, 4>(p, grid, st);
    if (e == hipSuccess && longest > 0) e = launch_attend_parts(a, st);
    return e != hipSuccess ? e : launch_attend_join(a, st);
}

hipError_t launch_attend_shared(const PrefixArgs &p, hipStream_t st) {
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
