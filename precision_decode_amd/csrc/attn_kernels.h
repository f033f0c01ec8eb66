// Device code of attention over a paged NVFP4 cache (nvfp4_attn.h says what it
// computes).  Not part of the C ABI.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane
// holds one query row: softmax runs along its own registers, the scores that
// leave the first product are, rounded, the B operand of the second, and the
// sums are rescaled by one number a lane.  e2m1 * e4m3 has at most 6 significant
// bits within 2^-10 .. 2688 and is exact in fp16, so K and V meet the fp16 matrix
// instructions as they are.  Q keeps its bits: a bf16 row is scaled by a power of
// two that brings its largest element to 2^14, where elements down to 2^-28 of it
// stay exact and what smaller ones lose lies below fp32's rounding of the sum.  P
// is exp2 of the scores minus the row's running maximum, times 2^8, rounded to
// fp16: 11 significant bits for every weight down to 2^-22 of the largest.
#ifndef NVFP4_ATTN_KERNELS_H
#define NVFP4_ATTN_KERNELS_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <utility>

#include "cache_kernels.h"
#include "device_common.h"

namespace nvfp4attn {

using nvfp4dev::f16x8;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kStep = 64;                  // cache tokens of a step: four runs of 16, each within one page
constexpr int kRun = 16;
constexpr float kWeightShift = 8.0f;       // P is scaled by 2^8
constexpr float kRescaleAt = 6.0f;         // growth of the maximum (log2) that rescales the sums: P stays below 2^14
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    CacheArgs c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_token, q_head, o_token, o_head;
    const int32_t *table, *lengths, *starts;
    int64_t table_stride;
    int32_t pages, table_width, batch, group, tokens, max_query, window, sinks, bf16;
    bool q_wide, o_wide;
    float scale;
    float *part, *ml;      // per workgroup two partial results: [rows][dp] sums, [rows][2] maximum and sum
    int64_t *prefix;       // [batch + 1] steps of the sequences before each
    int32_t groups;        // workgroups among which the steps are dealt out
};

struct Sequence {
    int len, first, n, computed;   // cache tokens, first query's row of Q, queries, queries that are computed
};

__device__ __forceinline__ int steps_of(int tokens) { return (tokens >> 6) + ((tokens & 63) != 0 ? 1 : 0); }

__device__ __forceinline__ Sequence sequence_of(const AttnArgs &a, int b) {
    Sequence s;
    const int most = a.table_width << a.c.page_log2;
    s.len = a.lengths[b];
    s.len = s.len < 0 ? 0 : s.len > most ? most : s.len;
    if (a.starts != nullptr) {
        int x = a.starts[b], y = a.starts[b + 1];
        x = x < 0 ? 0 : x > a.tokens ? a.tokens : x;
        y = y < x ? x : y > a.tokens ? a.tokens : y;
        s.first = x;
        s.n = y - x;
    } else {
        s.n = a.tokens / a.batch;
        s.first = b * s.n;
    }
    s.computed = s.n < a.max_query ? s.n : a.max_query;
    return s;
}

// The steps of the cache that a tile of query rows sees: `sinks` first ones, then
// those from `from` on, `count` in all.
struct Steps {
    int p_first, p_last;           // positions of the tile's first and last query (may be negative)
    int sinks, from, count;
    __device__ __forceinline__ int at(int i) const { return i < sinks ? i : from + (i - sinks); }
};

__device__ __forceinline__ Steps steps_for(const AttnArgs &a, const Sequence &s, int row0, int rows) {
    Steps w = {};
    const int last_row = s.computed * a.group - 1;
    if (row0 > last_row) return w;
    const int end_row = row0 + rows - 1 < last_row ? row0 + rows - 1 : last_row;
    w.p_first = s.len - s.n + row0 / a.group;
    w.p_last = s.len - s.n + end_row / a.group;
    if (w.p_last < 0) return w;
    const int hi = w.p_last + 1;
    int lo = 0;
    if (a.window > 0) {
        lo = (w.p_first > 0 ? w.p_first : 0) - a.window + 1;
        lo = lo > 0 ? lo : 0;
    }
    w.from = lo >> 6;
    const int sinks = steps_of(a.sinks < hi ? a.sinks : hi);
    w.sinks = sinks < w.from ? sinks : w.from;
    w.count = w.sinks + steps_of(hi) - w.from;
    return w;
}

__device__ __forceinline__ float xor16(float v, bool take_max) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float x = __builtin_bit_cast(float, static_cast<unsigned>(r[0])),
                y = __builtin_bit_cast(float, static_cast<unsigned>(r[1]));
    return take_max ? __builtin_fmaxf(x, y) : x + y;
}
__device__ __forceinline__ float xor32(float v, bool take_max) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float x = __builtin_bit_cast(float, static_cast<unsigned>(r[0])),
                y = __builtin_bit_cast(float, static_cast<unsigned>(r[1]));
    return take_max ? __builtin_fmaxf(x, y) : x + y;
}
// Maximum and sum over the four 16-lane rows, the same in each.
__device__ __forceinline__ float rows_max(float v) { return xor32(xor16(v, true), true); }
__device__ __forceinline__ float rows_sum(float v) { return xor32(xor16(v, false), false); }

// Lane N of each 16-lane row, to the whole row.
template <int N>
__device__ __forceinline__ f16x2 row_bcast(f16x2 v) {
    return nvfp4dev::halves(static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(nvfp4dev::bits(v)), 0x150 + N, 0xF, 0xF, false)));
}

__device__ __forceinline__ f16x2 e4m3_high_f16(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
}

// 8 E2M1 codes times pairs of fp16 scales.
__device__ __forceinline__ f16x8 decode8(uint32_t w, f16x2 s0, f16x2 s1, f16x2 s2, f16x2 s3) {
    const f16x2 a = nvfp4dev::e2m1x2_f16<0>(w) * s0, b = nvfp4dev::e2m1x2_f16<1>(w) * s1,
                c = nvfp4dev::e2m1x2_f16<2>(w) * s2, d = nvfp4dev::e2m1x2_f16<3>(w) * s3;
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Bytes of 4 x 4 turned: out word t holds byte t of each word.
__device__ __forceinline__ void turn_bytes(u32x4 w, uint32_t (&t)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    t[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    t[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    t[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    t[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// ---------------------------------------------------------------- the stream kernel
//
// A workgroup holds 16 R query rows of one sequence and kv head; its four waves
// take the steps of the cache in turn, each with running maxima, sums and outputs
// of its own that are joined at the end, so that waves never wait for each other
// within the loop.  A lane of A operand r = lane % 16 holds token 16 (r / 4) +
// 4 (r % 4) + t in score tile t: it then ends with the scores of 16 tokens of one
// run in the order in which the transposed LDS read hands out V's.
template <int NB, int R>
struct Stream {
    static constexpr int kDp = 16 * NB;
    static constexpr int kRows = 16 * R;
    static constexpr int kK = kDp / 32;            // 32-element slices of a row: words a lane holds of a token
    static constexpr int kChunks = kDp / 32;       // 16-byte pieces of a token's codes
    static constexpr int kLaneBlocks = NB / 4;     // scale blocks of a lane's slice of K
    static constexpr int kStage = kStep * kDp / 2; // a wave's V codes in LDS

    struct Buffers {
        __attribute__((aligned(16))) uint8_t v[kAttnWaves][kStage];
        __attribute__((aligned(16))) float o[kAttnWaves][kRows][20];   // one block of 16 outputs, rows padded
        float m[kAttnWaves][kRows], l[kAttnWaves][kRows];
    };

    struct Loads {                                 // a step on its way
        uint32_t k[4][kK];
        uint32_t ks[kLaneBlocks];
        u32x4 v[kChunks];
        u32x4 vs;
        int page[4];                               // of each run, -1 where nothing is visible
    };

    int lane, wave, r16, h;                        // r16 = lane % 16, h = lane / 16
    f16x8 q[R][kK];
    float c[R];                                    // scores to log2 units
    int pos[R];
    f32x4 acc[R][NB];
    float m[R], l[R];

    // The pages of step s as lane r16 / 4 sees them (its run's), -1 without one.
    __device__ __forceinline__ int entry(const AttnArgs &a, const int32_t *row, int len, int s) const {
        const int token = s * kStep + kRun * (r16 >> 2);
        int i = token >> a.c.page_log2;
        i = i < a.table_width ? i : a.table_width - 1;
        const int p = row[i];
        return token < len && p >= 0 && p < a.pages ? p : -1;
    }

    __device__ __forceinline__ void load(const AttnArgs &a, int kvh, int s, int e, Loads &x) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.page[i] = __builtin_amdgcn_readlane(e, 4 * i);
        const int ps = 1 << a.c.page_log2;
        const uint32_t page_codes = static_cast<uint32_t>(a.c.kv_heads) << a.c.page_log2;   // tokens of all heads
        const int tok0 = s * kStep;
        const int own = e < 0 ? 0 : e;
        // K: this lane's four tokens
        {
            const int off = ((tok0 + kRun * (r16 >> 2)) & (ps - 1)) + 4 * (r16 & 3);
            const uint64_t at = static_cast<uint64_t>(own) * page_codes + (static_cast<uint32_t>(kvh) << a.c.page_log2);
            const uint8_t *p = a.c.k_codes + (at + off) * (kDp / 2) + h * (kDp / 8);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if constexpr (kK % 4 == 0) {
#pragma unroll
                    for (int j = 0; j < kK; j += 4) {
                        const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + t * (kDp / 2) + 4 * j));
                        x.k[t][j] = w[0]; x.k[t][j + 1] = w[1]; x.k[t][j + 2] = w[2]; x.k[t][j + 3] = w[3];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kK; j += 2) {
                        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p + t * (kDp / 2) + 4 * j));
                        x.k[t][j] = w[0]; x.k[t][j + 1] = w[1];
                    }
                }
            }
            const uint8_t *sp = a.c.k_scales + at * NB + off;
#pragma unroll
            for (int j = 0; j < kLaneBlocks; ++j)
                x.ks[j] = *reinterpret_cast<const uint32_t *>(sp + ((h * kLaneBlocks + j) << a.c.page_log2));
        }
        // V: pieces of 16 bytes in memory order
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = i * kWave + lane, token = at / kChunks, piece = at % kChunks;
            const int run = token >> 4;
            int p = run == 0 ? x.page[0] : run == 1 ? x.page[1] : run == 2 ? x.page[2] : x.page[3];
            p = p < 0 ? 0 : p;
            const uint64_t base = static_cast<uint64_t>(p) * page_codes + (static_cast<uint32_t>(kvh) << a.c.page_log2);
            const uint8_t *vp = a.c.v_codes + (base + ((tok0 + token) & (ps - 1))) * (kDp / 2) + 16 * piece;
            x.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(vp));
        }
        // V's scales: lane r16 of run h takes block r16, 16 tokens
        {
            int p = h == 0 ? x.page[0] : h == 1 ? x.page[1] : h == 2 ? x.page[2] : x.page[3];
            p = p < 0 ? 0 : p;
            const uint64_t base = static_cast<uint64_t>(p) * page_codes + (static_cast<uint32_t>(kvh) << a.c.page_log2);
            const int b = r16 < NB ? r16 : NB - 1;
            x.vs = *reinterpret_cast<const u32x4 *>(a.c.v_scales + base * NB + (b << a.c.page_log2) +
                                                    ((tok0 + kRun * h) & (ps - 1)));
        }
    }

    static __device__ __forceinline__ int piece_at(int token, int piece) {
        // pieces change places so that 16 tokens' reads of one block fall on all banks
        const int f = kChunks == 2 ? (token >> 3) & 1 : kChunks == 4 ? (token >> 2) & 3
                      : kChunks == 6 ? (token >> 3) & 1 : (token >> 1) & 7;
        return token * (kDp / 2) + 16 * (piece ^ f);
    }

    template <int B>
    __device__ __forceinline__ void block(const uint8_t *stage, const f16x2 (&vs)[8], const f16x8 (&p)[R][2]) {
        typedef __attribute__((address_space(3))) i32x2 lds2;
        const int token = kRun * h + 4 * (r16 & 3) + (r16 >> 2);
        const uint8_t *at = stage + piece_at(token, B / 2) + 8 * (B % 2);
        const i32x2 w = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds2 *)at);
        f16x2 s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = row_bcast<B>(vs[i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f16x8 v = decode8(static_cast<uint32_t>(w[k]), s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]);
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][B] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[r][k], acc[r][B], 0, 0, 0);
        }
    }
    template <int... B>
    __device__ __forceinline__ void blocks(std::integer_sequence<int, B...>, const uint8_t *stage, const f16x2 (&vs)[8],
                                           const f16x8 (&p)[R][2]) {
        (block<B>(stage, vs, p), ...);
    }

    // Rows that see a token whose block of V is NaN: NaN there.  `bad` holds the
    // tokens (bits) of this lane's run and block.
    template <int B>
    __device__ __forceinline__ void poison_block(const AttnArgs &a, int tok0, uint32_t bad) {
        for (int run = 0; run < 4; ++run) {
            uint32_t bits = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(bad), kRun * run + B));
            while (bits != 0) {
                const int j = tok0 + kRun * run + __builtin_ctz(bits);
                bits &= bits - 1;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (visible(a, pos[r], j)) acc[r][B] = f32x4{1, 1, 1, 1} * __uint_as_float(0x7FC00000u);
            }
        }
    }
    template <int... B>
    __device__ __forceinline__ void poison(std::integer_sequence<int, B...>, const AttnArgs &a, int tok0, uint32_t bad) {
        (poison_block<B>(a, tok0, bad), ...);
    }

    static __device__ __forceinline__ bool visible(const AttnArgs &a, int p, int j) {
        return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
    }

    __device__ __forceinline__ void step(const AttnArgs &a, const Steps &w, int s, Loads &x, uint8_t *stage) {
        const int tok0 = s * kStep;
        const bool pages = (x.page[0] | x.page[1] | x.page[2] | x.page[3]) >= 0;
        const bool whole = pages && tok0 + kStep - 1 <= w.p_first &&
                           (a.window == 0 || tok0 > w.p_last - a.window || tok0 + kStep - 1 < a.sinks);
        // V's codes to LDS
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = i * kWave + lane;
            *reinterpret_cast<u32x4 *>(stage + piece_at(at / kChunks, at % kChunks)) = x.v[i];
        }
        wave_fence();

        // scores
        f32x4 sc[R][4];
        f16x2 ks[kLaneBlocks][2];
#pragma unroll
        for (int j = 0; j < kLaneBlocks; ++j) {
            ks[j][0] = nvfp4dev::e4m3x2_f16(x.ks[j]);
            ks[j][1] = e4m3_high_f16(x.ks[j]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int r = 0; r < R; ++r) sc[r][t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < kK; ++j) {
                const _Float16 sv = ks[j / 2][t / 2][t % 2];
                const f16x2 ss = {sv, sv};
                const f16x8 k = decode8(x.k[t][j], ss, ss, ss, ss);
#pragma unroll
                for (int r = 0; r < R; ++r) sc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[r][j], sc[r][t], 0, 0, 0);
            }
        }

        // V's scales, and which of its blocks are NaN
        uint32_t bad = 0;
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t nan = ((x.vs[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                // one bit a byte, to bits 4 i .. 4 i + 3
                bad |= ((nan >> 7) * 0x10204080u >> 28) << (4 * i);
                x.vs[i] &= ~((nan >> 7) * 0xFFu);
            }
        }
        uint32_t turned[4];
        turn_bytes(x.vs, turned);
        f16x2 vs[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vs[2 * t] = nvfp4dev::e4m3x2_f16(turned[t]);
            vs[2 * t + 1] = e4m3_high_f16(turned[t]);
        }

        // softmax: the row's maximum, weights, their sum
        f16x8 p[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t seen = 0xFFFFu;
            if (!whole) {
                seen = 0;
                const bool page = (h == 0 ? x.page[0] : h == 1 ? x.page[1] : h == 2 ? x.page[2] : x.page[3]) >= 0;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool v = page && visible(a, pos[r], tok0 + kRun * h + 4 * i + t);
                        seen |= (v ? 1u : 0u) << (4 * t + i);
                        sc[r][t][i] = v ? sc[r][t][i] : -__builtin_inff();
                    }
            }
            float top = sc[r][0][0];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, sc[r][t][i]);
            top = rows_max(top);
            top = top == -__builtin_inff() ? top : top * c[r];
            const bool grown = top > m[r] + kRescaleAt || (m[r] == -__builtin_inff() && top > m[r]);
            if (__any(grown)) {
                const float to = grown ? top : m[r];
                const float f = grown ? __builtin_amdgcn_exp2f(m[r] - to) : 1.0f;
                m[r] = to;
                l[r] *= f;
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[r][b] *= f;
            }
            const float shift = kWeightShift - (m[r] == -__builtin_inff() ? 0.0f : m[r]);
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][t][i], c[r], shift));
                    if (!whole) e = (seen >> (4 * t + i)) & 1u ? e : 0.0f;
                    sum += e;
                    p[r][t / 2][4 * (t % 2) + i] = static_cast<_Float16>(e);
                }
            l[r] += sum;
        }

        blocks(std::make_integer_sequence<int, NB>{}, stage, vs, p);
        if (!whole && __any(bad != 0)) poison(std::make_integer_sequence<int, NB>{}, a, tok0, bad);
        wave_fence();
    }

    // Query rows row0 .. of sequence s as B operands.
    __device__ __forceinline__ void load_queries(const AttnArgs &a, const Sequence &s, int kvh, int row0) {
        const int rows = s.computed * a.group;
        const float g = a.scale * (a.c.k_global != nullptr ? a.c.k_global[kvh] : 1.0f);
        const bool bf16 = a.bf16 != 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = row0 + 16 * r + r16;
            const int i = row / a.group, head = kvh * a.group + (row - i * a.group);
            pos[r] = -1;
            u32x4 raw[kK];
#pragma unroll
            for (int j = 0; j < kK; ++j) raw[j] = u32x4{0, 0, 0, 0};
            if (row < rows) {
                const int at = s.len - s.n + i;
                pos[r] = at < 0 ? -1 : at;
                const uint16_t *p = a.q + static_cast<int64_t>(s.first + i) * a.q_token + head * a.q_head;
#pragma unroll
                for (int j = 0; j < kK; ++j) {
                    const int e0 = h * (kDp / 4) + 8 * j;
                    if (e0 < a.c.head_dim) raw[j] = load8(p + e0, a.q_wide);
                }
            }
            float x[kK][8];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kK; ++j) {
                widen(raw[j], bf16, x[j]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t b = __float_as_uint(x[j][k]) & 0x7FFFFFFFu;
                    top = b > top ? b : top;
                }
            }
            // a power of two that brings the row's largest element to [2^14, 2^15), bf16 only
            float up = 1.0f, down = 1.0f;
            if (bf16) {
                // magnitudes as floats, infinities and NaN included, sort as their patterns do
                uint32_t all = top;
                const uint32_t t16 = static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 16, kWave));
                all = t16 > all ? t16 : all;
                const uint32_t t32 = static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 32, kWave));
                all = t32 > all ? t32 : all;
                int e = static_cast<int>(all >> 23) - 127;          // -127 (zero, subnormal) .. 128
                e = e < -100 ? -100 : e > 127 ? 127 : e;
                up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
                down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
            }
            const float sign = g < 0.0f ? -up : up;
            c[r] = __builtin_fabsf(g) * kLog2e * down;
#pragma unroll
            for (int j = 0; j < kK; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k) q[r][j][k] = static_cast<_Float16>(x[j][k] * sign);
        }
    }

    // Steps i0 .. i1 of the sequence's list for query rows row0 .., joined over the
    // waves and written: to `out`, or where `slot` >= 0 as a partial result.
    __device__ __forceinline__ void run(const AttnArgs &a, Buffers &buf, const Sequence &s, const Steps &w, int b, int kvh,
                                        int row0, int i0, int i1, int64_t slot) {
        lane = threadIdx.x & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        r16 = lane & 15;
        h = lane >> 4;
        const int32_t *row = a.table + static_cast<int64_t>(b) * a.table_stride;
        load_queries(a, s, kvh, row0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int k = 0; k < NB; ++k) acc[r][k] = f32x4{0, 0, 0, 0};
        }
        uint8_t *stage = buf.v[wave];
        int i = i0 + wave;
        if (i < i1) {
            Loads x;
            load(a, kvh, w.at(i), entry(a, row, s.len, w.at(i)), x);
            int next = i + kAttnWaves;
            int e = next < i1 ? entry(a, row, s.len, w.at(next)) : -1;
            for (;;) {
                Loads y;
                const bool more = next < i1;
                int after = -1;
                if (more) {
                    load(a, kvh, w.at(next), e, y);
                    if (next + kAttnWaves < i1) after = entry(a, row, s.len, w.at(next + kAttnWaves));
                }
                step(a, w, w.at(i), x, stage);
                if (!more) break;
                x = y;
                e = after;
                i = next;
                next += kAttnWaves;
            }
        }
        join(a, buf, s, kvh, row0, slot);
    }

    __device__ __forceinline__ void join(const AttnArgs &a, Buffers &buf, const Sequence &s, int kvh, int row0,
                                         int64_t slot) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = rows_sum(l[r]);
            if (h == 0) {
                buf.m[wave][16 * r + r16] = m[r];
                buf.l[wave][16 * r + r16] = sum;
            }
        }
        __syncthreads();
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = buf.m[0][16 * r + r16];
#pragma unroll
            for (int k = 1; k < kAttnWaves; ++k) top = __builtin_fmaxf(top, buf.m[k][16 * r + r16]);
            f[r] = m[r] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[r] - top);
        }
        const float g = a.c.v_global != nullptr ? a.c.v_global[kvh] : 1.0f;
        const bool bf16 = a.bf16 != 0;
        const int rows = s.computed * a.group;
        // this thread's row and four outputs of each block
        constexpr int kEach = kRows * 4;           // threads of a block of outputs
        const int my_row = threadIdx.x / 4 % kRows, my = threadIdx.x % 4;
        const bool busy = threadIdx.x < kEach;
        float top = -__builtin_inff(), total = 0.0f;
        if (busy) {
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k) top = __builtin_fmaxf(top, buf.m[k][my_row]);
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k) {
                const float mk = buf.m[k][my_row];
                total += buf.l[k][my_row] * (mk == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mk - top));
            }
            if (slot >= 0 && my == 0) {
                a.ml[(slot * kRows + my_row) * 2] = top;
                a.ml[(slot * kRows + my_row) * 2 + 1] = total;
            }
        }
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        const int global_row = row0 + my_row;
        const int i = global_row / a.group, head = kvh * a.group + (global_row - i * a.group);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const f32x4 v = acc[r][b] * f[r];
                *reinterpret_cast<f32x4 *>(&buf.o[wave][16 * r + r16][4 * h]) = v;
            }
            __syncthreads();
            if (busy) {
                f32x4 v = *reinterpret_cast<const f32x4 *>(&buf.o[0][my_row][4 * my]);
#pragma unroll
                for (int k = 1; k < kAttnWaves; ++k) v += *reinterpret_cast<const f32x4 *>(&buf.o[k][my_row][4 * my]);
                if (slot >= 0) {
                    *reinterpret_cast<f32x4 *>(a.part + (slot * kRows + my_row) * kDp + 16 * b + 4 * my) = v;
                } else if (global_row < rows && 16 * b < a.c.head_dim) {
                    store4(a.out + static_cast<int64_t>(s.first + i) * a.o_token + head * a.o_head + 16 * b + 4 * my,
                           total == 0.0f ? f32x4{0, 0, 0, 0} : v * inv * g, bf16, a.o_wide);
                }
            }
            __syncthreads();
        }
    }

    static __device__ __forceinline__ void store4(uint16_t *p, f32x4 v, bool bf16, bool wide) {
        const uint32_t lo = to16(v[0], bf16) | to16(v[1], bf16) << 16, hi = to16(v[2], bf16) | to16(v[3], bf16) << 16;
        if (wide) {
            *reinterpret_cast<u32x2 *>(p) = u32x2{lo, hi};
        } else {
            p[0] = static_cast<uint16_t>(lo);
            p[1] = static_cast<uint16_t>(lo >> 16);
            p[2] = static_cast<uint16_t>(hi);
            p[3] = static_cast<uint16_t>(hi >> 16);
        }
    }
};

// Sums of count(b) over the sequences before each thread's share of them, and over
// all (`scan` of kAttnThreads values).
struct Share {
    int from, to;          // this thread's sequences
    int64_t before, total;
};
template <typename Count>
__device__ __forceinline__ Share share_of(int batch, int64_t *scan, Count count) {
    Share s;
    const int each = (batch + kAttnThreads - 1) / kAttnThreads;
    s.from = static_cast<int>(threadIdx.x) * each;
    s.from = s.from < batch ? s.from : batch;
    s.to = s.from + each < batch ? s.from + each : batch;
    int64_t own = 0;
    for (int b = s.from; b < s.to; ++b) own += count(b);
    scan[threadIdx.x] = own;
    __syncthreads();
    for (int o = 1; o < kAttnThreads; o <<= 1) {
        const int64_t add = static_cast<int>(threadIdx.x) >= o ? scan[threadIdx.x - o] : 0;
        __syncthreads();
        scan[threadIdx.x] += add;
        __syncthreads();
    }
    s.before = scan[threadIdx.x] - own;
    s.total = scan[kAttnThreads - 1];
    return s;
}

// One workgroup a tile of query rows and kv head; the whole list of steps.
template <int NB, int R>
__global__ __launch_bounds__(kAttnThreads) void attn_tiles(const AttnArgs a) {
    using S = Stream<NB, R>;
    __shared__ typename S::Buffers buf;
    __shared__ int64_t scan[kAttnThreads];
    __shared__ int found[2];
    const int kvh = blockIdx.x % a.c.kv_heads;
    const int tile = blockIdx.x / a.c.kv_heads;
    const auto tiles = [&](int b) -> int64_t {
        return (static_cast<int64_t>(sequence_of(a, b).computed) * a.group + S::kRows - 1) / S::kRows;
    };
    if (threadIdx.x == 0) found[0] = -1;
    const Share mine = share_of(a.batch, scan, tiles);
    int64_t at = mine.before;
    for (int b = mine.from; b < mine.to; ++b) {
        const int64_t n = tiles(b);
        if (tile >= at && tile < at + n) {
            found[0] = b;
            found[1] = static_cast<int>(tile - at);
        }
        at += n;
    }
    __syncthreads();
    const int b = __builtin_amdgcn_readfirstlane(found[0]);
    if (b < 0) return;
    const int row0 = __builtin_amdgcn_readfirstlane(found[1]) * S::kRows;
    const Sequence s = sequence_of(a, b);
    const Steps w = steps_for(a, s, row0, S::kRows);
    S job;
    job.run(a, buf, s, w, b, kvh, row0, 0, w.count, -1);
}

// First step of workgroup g of n that share `total` steps.
__device__ __forceinline__ int64_t first_of(int64_t g, int64_t n, int64_t total) { return g * total / n; }
__device__ __forceinline__ int64_t sharing(int64_t groups, int64_t total) {
    const int64_t n = (total + kAttnWaves - 1) / kAttnWaves;
    return n < groups ? (n > 0 ? n : 1) : groups;
}

// The steps of all sequences and kv heads, one after the other, in equal shares: a
// workgroup's share may begin and end within a sequence, whose results it then
// leaves as partial ones for attn_join.
template <int NB, int R>
__global__ __launch_bounds__(kAttnThreads) void attn_shared(const AttnArgs a) {
    using S = Stream<NB, R>;
    __shared__ typename S::Buffers buf;
    __shared__ int64_t scan[kAttnThreads];
    __shared__ int64_t found[2];
    const auto count = [&](int b) -> int64_t { return steps_for(a, sequence_of(a, b), 0, S::kRows).count; };
    const Share mine = share_of(a.batch, scan, count);
    const int64_t heads = a.c.kv_heads, total = mine.total * heads, n = sharing(a.groups, total);
    if (blockIdx.x == 0) {
        int64_t at = mine.before;
        for (int b = mine.from; b < mine.to; ++b) {
            a.prefix[b] = at;
            at += count(b);
        }
        if (threadIdx.x == 0) a.prefix[a.batch] = mine.total;
    }
    if (static_cast<int64_t>(blockIdx.x) >= n || total == 0) return;
    int64_t at = first_of(blockIdx.x, n, total);
    const int64_t end = first_of(static_cast<int64_t>(blockIdx.x) + 1, n, total);
    {
        int64_t x = mine.before * heads;
        for (int b = mine.from; b < mine.to; ++b) {
            const int64_t c = count(b) * heads;
            if (at >= x && at < x + c) {
                found[0] = b;
                found[1] = at - x;
            }
            x += c;
        }
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(static_cast<int>(found[0]));
    int64_t offset = found[1];
    bool first = true;
    while (at < end) {
        const Sequence s = sequence_of(a, b);
        const Steps w = steps_for(a, s, 0, S::kRows);
        if (w.count == 0) {
            ++b;
            continue;
        }
        int kvh = __builtin_amdgcn_readfirstlane(static_cast<int>(offset / w.count));
        int i0 = __builtin_amdgcn_readfirstlane(static_cast<int>(offset - static_cast<int64_t>(kvh) * w.count));
        for (; kvh < a.c.kv_heads && at < end; ++kvh, i0 = 0) {
            const int left = static_cast<int>(end - at < w.count ? end - at : w.count);
            const int i1 = i0 + left < w.count ? i0 + left : w.count;
            const bool complete = i0 == 0 && i1 == w.count;
            S job;
            job.run(a, buf, s, w, b, kvh, 0, i0, i1, complete ? -1 : 2 * static_cast<int64_t>(blockIdx.x) + (first ? 0 : 1));
            first = false;
            at += i1 - i0;
        }
        offset = 0;
        ++b;
    }
}

// One workgroup a query row: its partial results joined, or zeros where there are none.
template <int NB>
__global__ __launch_bounds__(kAttnThreads) void attn_join(const AttnArgs a, int rows) {
    constexpr int kDp = 16 * NB, kWide = kDp / 4, kSlices = kAttnThreads / kWide;
    __shared__ f32x4 sums[kSlices][kWide];
    const int row = blockIdx.x % rows, item = blockIdx.x / rows;
    const int b = item / a.c.kv_heads, kvh = item - b * a.c.kv_heads;
    const Sequence s = sequence_of(a, b);
    if (row >= s.computed * a.group) return;
    const int64_t heads = a.c.kv_heads, before = a.prefix[b], count = a.prefix[b + 1] - before;
    const int64_t total = a.prefix[a.batch] * heads, n = sharing(a.groups, total);
    const int slice = threadIdx.x / kWide, col = threadIdx.x % kWide;
    f32x4 v = {0, 0, 0, 0};
    float sum = 0.0f;
    if (count > 0) {
        const int64_t x = before * heads + kvh * count, y = x + count - 1;
        const auto owner = [&](int64_t p) {
            int64_t g = p * n / total;
            while (g + 1 < n && first_of(g + 1, n, total) <= p) ++g;
            while (g > 0 && first_of(g, n, total) > p) --g;
            return g;
        };
        const int64_t g0 = owner(x), g1 = owner(y);
        if (g0 == g1) return;                      // its workgroup had all of it
        const auto slot = [&](int64_t g) { return 2 * g + (g == g0 && first_of(g0, n, total) < x ? 1 : 0); };
        float top = -__builtin_inff();
        for (int64_t g = g0; g <= g1; ++g) top = __builtin_fmaxf(top, a.ml[(slot(g) * rows + row) * 2]);
        if (slice < kSlices) {
            for (int64_t g = g0 + slice; g <= g1; g += kSlices) {
                const int64_t at = slot(g) * rows + row;
                const float mk = a.ml[at * 2];
                const float f = mk == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mk - top);
                v += *reinterpret_cast<const f32x4 *>(a.part + at * kDp + 4 * col) * f;
            }
            sums[slice][col] = v;
        }
        for (int64_t g = g0; g <= g1; ++g) {
            const int64_t at = slot(g) * rows + row;
            const float mk = a.ml[at * 2];
            sum += a.ml[at * 2 + 1] * (mk == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mk - top));
        }
        __syncthreads();
        if (slice > 0) return;
        v = sums[0][col];
#pragma unroll
        for (int k = 1; k < kSlices; ++k) v += sums[k][col];
    } else if (slice > 0) {
        return;
    }
    if (4 * col >= a.c.head_dim) return;
    const int i = row / a.group, head = kvh * a.group + (row - i * a.group);
    const float g = a.c.v_global != nullptr ? a.c.v_global[kvh] : 1.0f;
    Stream<NB, 1>::store4(a.out + static_cast<int64_t>(s.first + i) * a.o_token + head * a.o_head + 4 * col,
                          sum == 0.0f ? f32x4{0, 0, 0, 0} : v * (1.0f / sum) * g, a.bf16 != 0, a.o_wide);
}

}  // namespace nvfp4attn

#endif  // NVFP4_ATTN_KERNELS_H
