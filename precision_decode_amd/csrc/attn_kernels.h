// Device code of attention over a paged NVFP4 cache (nvfp4_attn.h says what it
// computes).  Not part of the C ABI.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane
// holds one query row: softmax runs along its own registers, the scores that
// leave the first product are, rounded, the B operand of the second, and the
// sums are rescaled by one number a lane.  e2m1 * e4m3 has at most 6 significant
// bits within 2^-10 .. 2688 and is exact in fp16, so K and V meet the fp16 matrix
// instructions as they are.  Q keeps its bits: a bf16 row is scaled by a power of
// two that brings its largest element to [2^14, 2^15), where elements down to 2^-31
// of it stay exact (subnormal ones too) and smaller ones are rounded to 2^-24.  P
// is exp2 of the scores minus the row's running maximum, times 2^8, rounded to
// fp16: 11 significant bits for every weight down to 2^-22 of the largest.
#ifndef NVFP4_ATTN_KERNELS_H
#define NVFP4_ATTN_KERNELS_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <utility>

#include "attn_plan.h"
#include "cache_kernels.h"
#include "device_common.h"

namespace nvfp4attn {

using nvfp4dev::f16x8;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kStep = 64;                  // cache tokens of a step: four runs of 16, each within one page
constexpr int kRun = 16;
constexpr float kWeightShift = 8.0f;       // P is scaled by 2^8
constexpr float kRescaleAt = 6.0f;         // growth of the maximum (log2) that rescales the sums: P stays below 2^14
constexpr float kFarMaximum = 0x1p16f;     // a maximum (log2) from which scores are rounded before it is subtracted
constexpr int kAluCrosses = 0x2 | 0x4 | 0x400;   // a scheduling barrier for all but VALU, SALU and transcendentals
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    CacheArgs c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_token, q_head, o_token, o_head;
    const int32_t *table, *lengths, *starts;
    int64_t table_stride;
    int32_t pages, table_width, batch, group, tokens, max_query, window, sinks, bf16;
    int32_t each;          // queries of every sequence where `starts` is NULL
    uint32_t group_inverse;   // ceil(2^26 / group): row / group of rows below 32
    bool q_wide, o_wide;
    float scale;
    float *part, *ml;      // partial results: [rows][dp] sums, [rows][2] maximum and sum
    int64_t *prefix;       // [batch + 1] pieces of one kv head of the sequences before each
    int32_t groups;        // pieces into which the steps are dealt
};

struct Sequence {
    int len, first, n, computed;   // cache tokens, first query's row of Q, queries, queries that are computed
};

// Steps of 2^LOG tokens that hold `tokens` of them.
template <int LOG>
__device__ __forceinline__ int steps_of(int tokens) {
    return (tokens >> LOG) + ((tokens & ((1 << LOG) - 1)) != 0 ? 1 : 0);
}

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
        s.n = a.each;
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

// For queries first .. last of sequence s.
template <int LOG>
__device__ __forceinline__ Steps steps_between(const AttnArgs &a, const Sequence &s, int first, int last) {
    Steps w = {};
    w.p_first = s.len - s.n + first;
    w.p_last = s.len - s.n + last;
    if (first > last || w.p_last < 0) return w;
    const int hi = w.p_last + 1;
    int lo = 0;
    if (a.window > 0) {
        lo = (w.p_first > 0 ? w.p_first : 0) - a.window + 1;
        lo = lo > 0 ? lo : 0;
    }
    w.from = lo >> LOG;
    const int sinks = steps_of<LOG>(a.sinks < hi ? a.sinks : hi);
    w.sinks = sinks < w.from ? sinks : w.from;
    w.count = w.sinks + steps_of<LOG>(hi) - w.from;
    return w;
}
// For all of its queries.
template <int LOG>
__device__ __forceinline__ Steps steps_for(const AttnArgs &a, const Sequence &s) {
    return steps_between<LOG>(a, s, 0, s.computed - 1);
}
// For query rows row0 .. row0 + rows - 1 (query times heads of a kv head).
template <int LOG>
__device__ __forceinline__ Steps steps_for(const AttnArgs &a, const Sequence &s, int row0, int rows) {
    const int last_row = s.computed * a.group - 1, end = row0 + rows - 1 < last_row ? row0 + rows - 1 : last_row;
    return row0 > last_row ? Steps{} : steps_between<LOG>(a, s, row0 / a.group, end / a.group);
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

// A power of two that brings magnitude `top` (its pattern; infinities and NaN sort
// above the numbers) to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void row_power(uint32_t top, float *up, float *down) {
    int e = static_cast<int>(top >> 23) - 127;         // -127 (zero, subnormal) .. 128
    e = e < -100 ? -100 : e > 127 ? 127 : e;
    *up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
    *down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

// The largest magnitude pattern among 16-bit values, two a word.
template <int N>
__device__ __forceinline__ uint32_t top16(const u32x4 (&w)[N]) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[j][i] & 0x7FFF7FFFu));
    return top.x > top.y ? top.x : top.y;
}
// 8 bf16 values times a power of two, as fp16.
__device__ __forceinline__ f16x8 scale_bf16(u32x4 w, float up) {
    f16x8 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = static_cast<_Float16>(__uint_as_float(w[i] << 16) * up);
        x[2 * i + 1] = static_cast<_Float16>(__uint_as_float(w[i] & 0xFFFF0000u) * up);
    }
    return x;
}

__device__ __forceinline__ f16x8 nan8() {
    return __builtin_bit_cast(f16x8, u32x4{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u});
}

// Whether a query at position p (-1: none) sees token j.
__device__ __forceinline__ bool visible(const AttnArgs &a, int p, int j) {
    return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}

// A weight is exp2(score c - maximum + 8), which takes one fused operation while the
// maximum's own rounding is small beside 1.  A maximum of 2^24 and more is off by its
// rounding from the product that it was rounded from, which fp16 weights do not hold:
// there the scores are rounded as the maximum was, before it is subtracted, and the
// difference of near ones is exact.
__device__ __forceinline__ bool far_maximum(float m) { return __builtin_fabsf(m) >= kFarMaximum; }

__device__ __forceinline__ void store4(uint16_t *p, f32x4 v, bool bf16, bool wide) {
    const uint32_t lo = pair16(v[0], v[1], bf16), hi = pair16(v[2], v[3], bf16);
    if (wide) {
        *reinterpret_cast<u32x2 *>(p) = u32x2{lo, hi};
    } else {
        p[0] = static_cast<uint16_t>(lo);
        p[1] = static_cast<uint16_t>(lo >> 16);
        p[2] = static_cast<uint16_t>(hi);
        p[3] = static_cast<uint16_t>(hi >> 16);
    }
}

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

// The lane's number and its 16-lane row.  Not known to be the same from use to use,
// so that the many addresses of a step are computed in it and not kept in
// registers through the loop, which has none to spare.
struct Lane {
    uint32_t id, r16, h;
};
__device__ __forceinline__ Lane this_lane() {
    uint32_t x = threadIdx.x;
    __asm__ volatile("" : "+v"(x));
    x &= kWave - 1;
    return {x, x & 15, x >> 4};
}

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- the stream kernel
//
// A workgroup holds 16 R query rows of one sequence and kv head; its four waves
// take the steps of the cache in turn, each with running maxima, sums and outputs
// of its own that are joined at the end, so that waves never wait for each other
// within the loop.  A whole step is on its way while the one before is worked on:
// K's codes in registers, read in runs of whole 128-byte lines; V's codes and all
// scales straight into the other of a wave's two stages in LDS.  A lane of A operand
// r = lane % 16 holds token 16 (r / 4) + 4 t + r % 4 in score tile t: it then ends
// with the scores of the 16 tokens of run lane / 16, in the order in which the
// transposed LDS read hands out V's.
typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void global_void_t;

__device__ __forceinline__ uint32_t lds_address(const uint8_t *p) {
    return static_cast<uint32_t>(reinterpret_cast<size_t>((__attribute__((address_space(3))) const uint8_t *)(p)));
}
// Every load to registers and to LDS has arrived.
__device__ __forceinline__ void wait_loads() {
    nvfp4dev::phase_fence();
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));   // vmcnt 0, the other counters at their maximum
    nvfp4dev::phase_fence();
}

// Reads of what direct-to-LDS loads brought, which the kernel has waited for.  The
// compiler would put a wait for all loads in flight, the next step's too, before
// reads that it knows of.  Each waits for its own data; outputs are early-clobber, as
// a read may return while later ones still use their addresses.
template <int N>
__device__ __forceinline__ void lds_read16(uint32_t at, uint32_t apart, u32x4 (&x)[N]) {
    static_assert(N >= 1 && N <= 4, "one to four blocks");
    if constexpr (N == 1) {
        asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(x[0]) : "v"(at) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]) : "v"(at), "v"(at + apart) : "memory");
    } else if constexpr (N == 3) {
        asm volatile("ds_read_b128 %0, %3\n\tds_read_b128 %1, %4\n\tds_read_b128 %2, %5\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]) : "v"(at), "v"(at + apart), "v"(at + 2 * apart) : "memory");
    } else {
        asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
                     : "v"(at), "v"(at + apart), "v"(at + 2 * apart), "v"(at + 3 * apart) : "memory");
    }
}
// Transposed reads of blocks B .. B + 3: pieces at p0 and p1, two blocks of 8 bytes each.
__device__ __forceinline__ void lds_read_turned(uint32_t p0, uint32_t p1, i32x2 (&x)[4]) {
    asm volatile("ds_read_b64_tr_b4 %0, %4\n\tds_read_b64_tr_b4 %1, %4 offset:8\n\t"
                 "ds_read_b64_tr_b4 %2, %5\n\tds_read_b64_tr_b4 %3, %5 offset:8\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]) : "v"(p0), "v"(p1) : "memory");
}

// A workgroup's piece: part `part` of the `pieces` of sequence b (-1: none) and kv head.
struct Piece {
    int b, kvh, part, pieces;
    Sequence s;
};

template <int NB, int R>
struct Stream {
    static constexpr int kDp = 16 * NB;
    static constexpr int kRows = 16 * R;
    static constexpr int kK = kDp / 32;            // 32-element slices of a row: words a lane holds of a token
    static constexpr int kChunks = kDp / 32;       // 16-byte pieces of a token's codes
    static constexpr int kLaneBlocks = NB / 4;     // scale blocks of a lane's slice of K
    static constexpr int kCodes = kStep * kDp / 2; // bytes of V's codes in a stage
    static constexpr int kScales = 64 * NB;        // bytes of K's scales, then as many of V's: [block][64 tokens]
    static constexpr int kStage = kCodes + 2 * kScales;

    // 16 rows times up to 8 blocks of outputs are joined at a time
    static constexpr int kJoinBlocks = NB < 8 ? NB : NB % 8 == 0 ? 8 : 6;
    static constexpr int kJoinRow = 16 * kJoinBlocks + 4;

    union Buffers {
        __attribute__((aligned(16))) uint8_t v[kAttnWaves][2][kStage];
        struct {
            __attribute__((aligned(16))) float o[kAttnWaves][16][kJoinRow];
            float m[kAttnWaves][kRows], l[kAttnWaves][kRows];
        };
        Piece piece;
    };

    uint32_t kw[4][kK];                            // K's codes on their way
    int wave;
    f16x8 q[R][kK];
    float c[R];                                    // scores to log2 units
    int pos[R];
    f32x4 acc[R][NB];
    float m[R], l[R];

    // The page of step s that lane r16's run r16 / 4 lies in, -1 without one.
    __device__ __forceinline__ int entry(const AttnArgs &a, const int32_t *row, int len, int s) const {
        const int r16 = this_lane().r16;
        const int token = s * kStep + kRun * (r16 >> 2);
        int i = token >> a.c.page_log2;
        i = i < a.table_width ? i : a.table_width - 1;
        const int p = row[i];
        return token < len && p >= 0 && p < a.pages ? p : -1;
    }

    // Tokens of all heads before (page, kvh), page 0 for what is not there.
    static __device__ __forceinline__ uint64_t tokens_before(const AttnArgs &a, int page, int kvh) {
        return static_cast<uint64_t>(static_cast<uint32_t>(page < 0 ? 0 : page)) *
                   (static_cast<uint32_t>(a.c.kv_heads) << a.c.page_log2) +
               (static_cast<uint32_t>(kvh) << a.c.page_log2);
    }
    // Lane entry of run i, of all lanes.
    static __device__ __forceinline__ int page_of(int e, int i) { return __builtin_amdgcn_readlane(e, 4 * i); }
    static __device__ __forceinline__ int page_of_run(int e, uint32_t run) {
        return run == 0 ? page_of(e, 0) : run == 1 ? page_of(e, 1) : run == 2 ? page_of(e, 2) : page_of(e, 3);
    }

    // Sends for step s: K's codes to kw, the rest to `stage`.  Pages of 64 tokens and
    // more hold the whole step: addresses are then one base and offsets of the lane.
    __device__ __forceinline__ void load(const AttnArgs &a, int kvh, int s, int e, uint8_t *stage) {
        if (a.c.page_log2 >= 6) {
            load<true>(a, kvh, s, e, stage);
        } else {
            load<false>(a, kvh, s, e, stage);
        }
    }
    template <bool ONE_PAGE>
    __device__ __forceinline__ void load(const AttnArgs &a, int kvh, int s, int e, uint8_t *stage) {
        const auto [lane, r16, h] = this_lane();
        const int ps = 1 << a.c.page_log2, tok0 = s * kStep;
        const uint64_t base = tokens_before(a, page_of(e, 0), kvh);     // of ONE_PAGE
        const uint32_t first = tok0 & (ps - 1);
        // V's codes: pieces of 16 bytes, each lane's in the place that piece_at gives it
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const uint32_t at = i * kWave + lane, token = at / kChunks, piece = (at % kChunks) ^ turn(token);
            const uint8_t *p;
            if constexpr (ONE_PAGE) {
                p = a.c.v_codes + (base + first) * (kDp / 2) + (token * (kDp / 2) + 16 * piece);
            } else if constexpr (kWave / kChunks == kRun) {   // the lanes share a run
                p = a.c.v_codes + (tokens_before(a, page_of(e, i), kvh) + ((tok0 + kRun * i) & (ps - 1))) * (kDp / 2) +
                    ((token & (kRun - 1)) * (kDp / 2) + 16 * piece);
            } else {
                p = a.c.v_codes + (tokens_before(a, page_of_run(e, token >> 4), kvh) + ((tok0 + token) & (ps - 1))) * (kDp / 2) +
                    16 * piece;
            }
            __builtin_amdgcn_global_load_lds((global_void_t *)p, (lds_void_t *)(stage + i * 1024), 16, 0, 0);
        }
        // scales: pieces of 16 tokens of a block, K's then V's
#pragma unroll
        for (int i = 0; i < (8 * NB + kWave - 1) / kWave; ++i) {
            uint32_t at = i * kWave + lane;
            if (8 * NB % kWave == 0 || at < 8 * NB) {
                const bool is_v = at >= 4 * NB;
                at = is_v ? at - 4 * NB : at;
                const uint32_t block = at / 4, run = at % 4;
                const uint8_t *p = is_v ? a.c.v_scales : a.c.k_scales;
                if constexpr (ONE_PAGE) {
                    p += base * NB + first + ((block << a.c.page_log2) + kRun * run);
                } else {
                    p += tokens_before(a, page_of_run(e, run), kvh) * NB + (block << a.c.page_log2) +
                         ((tok0 + kRun * run) & (ps - 1));
                }
                __builtin_amdgcn_global_load_lds((global_void_t *)p, (lds_void_t *)(stage + kCodes + i * 1024), 16, 0, 0);
            }
        }
        // K's codes: this lane's four tokens
        const uint8_t *p;
        if constexpr (ONE_PAGE) {
            p = a.c.k_codes + (base + first) * (kDp / 2) + ((kRun * (r16 >> 2) + (r16 & 3)) * (kDp / 2) + h * (kDp / 8));
        } else {
            const uint32_t off = ((tok0 + kRun * (r16 >> 2)) & (ps - 1)) + (r16 & 3);
            p = a.c.k_codes + (tokens_before(a, e, kvh) + off) * (kDp / 2) + h * (kDp / 8);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if constexpr (kK % 4 == 0) {
#pragma unroll
                for (int j = 0; j < kK; j += 4) {
                    const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + t * (2 * kDp) + 4 * j));
                    kw[t][j] = w[0]; kw[t][j + 1] = w[1]; kw[t][j + 2] = w[2]; kw[t][j + 3] = w[3];
                }
            } else {
#pragma unroll
                for (int j = 0; j < kK; j += 2) {
                    const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p + t * (2 * kDp) + 4 * j));
                    kw[t][j] = w[0]; kw[t][j + 1] = w[1];
                }
            }
        }
    }

    // Pieces of a token change places by this, so that 16 tokens' reads of one block fall
    // on all banks.
    static __device__ __forceinline__ uint32_t turn(uint32_t token) {
        return kChunks == 2 ? (token >> 3) & 1 : kChunks == 4 ? (token >> 2) & 3 : kChunks == 6 ? (token >> 3) & 1 : (token >> 1) & 7;
    }
    static __device__ __forceinline__ uint32_t piece_at(uint32_t token, uint32_t piece) {
        return token * (kDp / 2) + 16 * (piece ^ turn(token));
    }

    template <int B>
    __device__ __forceinline__ void block(i32x2 w, const f16x2 (&vs)[8], const f16x8 (&p)[R][2]) {
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
    // Blocks 4 G .. 4 G + 3 of the outputs.
    template <int G>
    __device__ __forceinline__ void four_blocks(uint32_t stage, uint32_t token, const f16x2 (&vs)[8], const f16x8 (&p)[R][2]) {
        i32x2 w[4];
        lds_read_turned(stage + piece_at(token, 2 * G), stage + piece_at(token, 2 * G + 1), w);
        block<4 * G>(w[0], vs, p);
        block<4 * G + 1>(w[1], vs, p);
        block<4 * G + 2>(w[2], vs, p);
        block<4 * G + 3>(w[3], vs, p);
    }
    template <int... G>
    __device__ __forceinline__ void blocks(std::integer_sequence<int, G...>, uint32_t stage, const f16x2 (&vs)[8],
                                           const f16x8 (&p)[R][2]) {
        const Lane n = this_lane();
        (four_blocks<G>(stage, kRun * n.h + n.r16, vs, p), ...);
    }

    // Rows that see a token whose block of V is NaN: NaN there.  `bad` holds the
    // tokens (bits) of this lane's run and block, none of a run whose page is not there.
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

    // Minus infinity for what row tile r does not see; `there`: which runs' pages are.
    __device__ __forceinline__ void hide(const AttnArgs &a, int r, int tok0, uint64_t there, f32x4 (&sc)[4]) const {
        const uint32_t h = this_lane().h;
        const bool page = (there >> (4 * h)) & 1u;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!page || !visible(a, pos[r], tok0 + kRun * static_cast<int>(h) + 4 * t + i)) sc[t][i] = -__builtin_inff();
    }

    // Softmax of row tile r: its running maximum and sum, the step's weights as B
    // operands.
    __device__ __forceinline__ void weigh(int r, f32x4 (&sc)[4], f16x8 (&p)[2]) {
        float top = sc[0][0];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, sc[t][i]);
        top = rows_max(top);
        top = top == -__builtin_inff() ? top : top * c[r];
        const bool grown = top - m[r] > kRescaleAt;    // also of a first score; not of NaN, nor of none
        if (__any(grown)) {
            const float to = grown ? top : m[r];
            const float f = grown ? __builtin_amdgcn_exp2f(m[r] - to) : 1.0f;
            m[r] = to;
            l[r] *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[r][b] *= f;
        }
        const float base = m[r] == -__builtin_inff() ? 0.0f : m[r];
        float factor = c[r], shift = kWeightShift - base;
        if (__any(far_maximum(base))) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[t][i] = far_maximum(base) ? sc[t][i] * c[r] - base : sc[t][i];
            factor = far_maximum(base) ? 1.0f : factor;
            shift = far_maximum(base) ? kWeightShift : shift;
        }
        float sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i], factor, shift));
                sum[i] += e;
                p[t / 2][4 * (t % 2) + i] = static_cast<_Float16>(e);
            }
        l[r] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    // Step s, whose pages e holds and whose codes and scales are there: K's in k, the
    // rest in `stage`.
    __device__ __forceinline__ void step(const AttnArgs &a, const Steps &w, int s, int e, const uint32_t (&k)[4][kK],
                                         uint32_t stage) {
        const auto [lane, r16, h] = this_lane();
        const int tok0 = s * kStep;
        const uint64_t there = __ballot(e >= 0);       // lanes 4 i: run i
        const bool pages = there == ~uint64_t(0);
        const bool whole = pages && tok0 + kStep - 1 <= w.p_first &&
                           (a.window == 0 || tok0 > w.p_last - a.window || tok0 + kStep - 1 < a.sinks);

        // scores: the lane's tokens' scales are byte r % 4 of each word of their run's
        u32x4 ks[kLaneBlocks];
        lds_read16<kLaneBlocks>(stage + kCodes + h * (kLaneBlocks * 64) + (r16 >> 2) * 16, 64, ks);
        f16x2 kf[kLaneBlocks][2];
        const uint32_t pick = (r16 & 3) * 0x0101u | 0x0400u;
#pragma unroll
        for (int j = 0; j < kLaneBlocks; ++j) {
            kf[j][0] = nvfp4dev::e4m3x2_f16(__builtin_amdgcn_perm(ks[j][1], ks[j][0], pick));
            kf[j][1] = nvfp4dev::e4m3x2_f16(__builtin_amdgcn_perm(ks[j][3], ks[j][2], pick));
        }
        f32x4 sc[R][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int r = 0; r < R; ++r) sc[r][t] = f32x4{0, 0, 0, 0};
            nvfp4dev::phase_fence();                   // else the scheduler decodes all tiles first and spills
#pragma unroll
            for (int j = 0; j < kK; ++j) {
                const _Float16 sv = kf[j / 2][t / 2][t % 2];
                const f16x2 ss = {sv, sv};
                const f16x8 x = decode8(k[t][j], ss, ss, ss, ss);
#pragma unroll
                for (int r = 0; r < R; ++r) sc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, q[r][j], sc[r][t], 0, 0, 0);
            }
        }

        // V's scales: lane r16 of run h takes block r16, 16 tokens; which of them are NaN
        u32x4 vsw[1];
        lds_read16<1>(stage + kCodes + kScales + (r16 < NB ? r16 : NB - 1) * 64 + h * 16, 0, vsw);
        uint32_t bad = 0;
        if (!whole) {
            __asm__ volatile("" : "+v"(bad));           // keeps this a branch: most steps skip it
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t nan = ((vsw[0][i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                // one bit a byte, to bits 4 i .. 4 i + 3
                bad |= ((nan >> 7) * 0x10204080u >> 28) << (4 * i);
                vsw[0][i] &= ~((nan >> 7) * 0xFFu);
            }
            // page 0 stands in for a page that is not there: what it holds is of another's
            if (!((there >> (4 * h)) & 1u)) bad = 0;
        }
        f16x2 vs[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vs[2 * t] = nvfp4dev::e4m3x2_f16(vsw[0][t]);
            vs[2 * t + 1] = e4m3_high_f16(vsw[0][t]);
        }

        f16x8 p[R][2];
        if (!whole) {
#pragma unroll
            for (int r = 0; r < R; ++r) hide(a, r, tok0, there, sc[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) weigh(r, sc[r], p[r]);

        blocks(std::make_integer_sequence<int, NB / 4>{}, stage, vs, p);
        if (!whole && __any(bad != 0)) poison(std::make_integer_sequence<int, NB>{}, a, tok0, bad);
    }

    // The query rows of sequence s, and their positions.
    __device__ __forceinline__ void fetch_queries(const AttnArgs &a, const Sequence &s, int kvh, u32x4 (&raw)[R][kK]) {
        const auto [lane, r16, h] = this_lane();
        const int rows = s.computed * a.group;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 16 * r + static_cast<int>(r16);
            const int i = static_cast<int>((static_cast<uint32_t>(row) * a.group_inverse) >> 26);
            const int head = kvh * a.group + (row - i * a.group);
            pos[r] = -1;
#pragma unroll
            for (int j = 0; j < kK; ++j) raw[r][j] = u32x4{0, 0, 0, 0};
            if (row < rows) {
                const int at = s.len - s.n + i;
                pos[r] = at < 0 ? -1 : at;
                const uint16_t *p = a.q + static_cast<int64_t>(s.first + i) * a.q_token + head * a.q_head;
#pragma unroll
                for (int j = 0; j < kK; ++j) {
                    const int e0 = static_cast<int>(h) * (kDp / 4) + 8 * j;
                    if (e0 < a.c.head_dim) raw[r][j] = load8(p + e0, a.q_wide);
                }
            }
        }
    }

    // As B operands.
    __device__ __forceinline__ void take_queries(const AttnArgs &a, int kvh, const u32x4 (&raw)[R][kK]) {
        const float g = a.scale * (a.c.k_global != nullptr ? a.c.k_global[kvh] : 1.0f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float down = 1.0f;
            if (a.bf16 != 0) {
                // a power of two that brings the row's largest element to [2^14, 2^15)
                uint32_t top = top16(raw[r]), t = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, kWave));
                top = t > top ? t : top;
                t = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave));
                float up;
                row_power((t > top ? t : top) << 16, &up, &down);
                up = g < 0.0f ? -up : up;
#pragma unroll
                for (int j = 0; j < kK; ++j) q[r][j] = scale_bf16(raw[r][j], up);
            } else {
                const uint32_t sign = g < 0.0f ? 0x80008000u : 0u;
#pragma unroll
                for (int j = 0; j < kK; ++j) q[r][j] = __builtin_bit_cast(f16x8, raw[r][j] ^ sign);
            }
            c[r] = __builtin_fabsf(g) * kLog2e * down;
            c[r] = c[r] == 0.0f ? 0x1p-126f : c[r];      // hidden scores stay minus infinity, others about 0
            if (!(__builtin_fabsf(g) < __builtin_inff())) {   // no factor of scores: those of tokens that are seen are NaN
                c[r] = 1.0f;
#pragma unroll
                for (int j = 0; j < kK; ++j) q[r][j] = nan8();
            }
        }
    }

    // Steps i0 .. i1 of the sequence's list, joined over the waves and written: to `out`,
    // or where `slot` >= 0 as a partial result.
    __device__ __forceinline__ void run(const AttnArgs &a, Buffers &buf, const Sequence &s, const Steps &w, int b, int kvh,
                                        int i0, int i1, int64_t slot) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int32_t *row = a.table + static_cast<int64_t>(b) * a.table_stride;
        int i = i0 + wave;
        const int at0 = i < i1 ? w.at(i) : -1;
        const int e0 = at0 >= 0 ? entry(a, row, s.len, at0) : -1;
        u32x4 raw[R][kK];
        fetch_queries(a, s, kvh, raw);
        if (at0 >= 0) load(a, kvh, at0, e0, buf.v[wave][0]);
        take_queries(a, kvh, raw);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int k = 0; k < NB; ++k) acc[r][k] = f32x4{0, 0, 0, 0};
        }
        if (at0 >= 0) {
            int at = at0, e = e0;
            int next = i + kAttnWaves < i1 ? w.at(i + kAttnWaves) : -1;
            int e_next = next >= 0 ? entry(a, row, s.len, next) : -1;
            for (uint32_t turn = 0;; turn ^= 1) {
                wait_loads();
                uint32_t k[4][kK];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < kK; ++j) k[t][j] = kw[t][j];
                if (next >= 0) load(a, kvh, next, e_next, buf.v[wave][turn ^ 1]);
                const int after = i + 2 * kAttnWaves < i1 ? w.at(i + 2 * kAttnWaves) : -1;
                const int e_after = after >= 0 ? entry(a, row, s.len, after) : -1;
                step(a, w, at, e, k, lds_address(buf.v[wave][turn]));
                if (next < 0) break;
                i += kAttnWaves;
                at = next;
                e = e_next;
                next = after;
                e_next = e_after;
            }
        }
        join(a, buf, s, kvh, slot);
    }

    __device__ __forceinline__ void join(const AttnArgs &a, Buffers &buf, const Sequence &s, int kvh, int64_t slot) {
        const auto [lane, r16, h] = this_lane();
        const int rows = s.computed * a.group;         // at most kRows, as the plan has it
        __syncthreads();                               // the waves are done with their stages
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = rows_sum(l[r]);
            if (h == 0) {
                buf.m[wave][16 * r + r16] = m[r];
                buf.l[wave][16 * r + r16] = sum;
            }
        }
        __syncthreads();
        const float g = a.c.v_global != nullptr ? a.c.v_global[kvh] : 1.0f;
        const bool bf16 = a.bf16 != 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (16 * r >= rows) break;
            float top = buf.m[0][16 * r + r16];
#pragma unroll
            for (int k = 1; k < kAttnWaves; ++k) top = __builtin_fmaxf(top, buf.m[k][16 * r + r16]);
            const float f = m[r] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[r] - top);
#pragma unroll
            for (int b0 = 0; b0 < NB; b0 += kJoinBlocks) {
                if (static_cast<int>(16 * r + r16) < rows) {
#pragma unroll
                    for (int b = 0; b < kJoinBlocks; ++b)
                        *reinterpret_cast<f32x4 *>(&buf.o[wave][r16][16 * b + 4 * h]) = acc[r][b0 + b] * f;
                }
                __syncthreads();
                const int n = rows - 16 * r < 16 ? rows - 16 * r : 16;
                for (int j = threadIdx.x; j < n * 4 * kJoinBlocks; j += kAttnThreads) {
                    const int row = 16 * r + j / (4 * kJoinBlocks), col = 4 * (j % (4 * kJoinBlocks));
                    f32x4 v = *reinterpret_cast<const f32x4 *>(&buf.o[0][row - 16 * r][col]);
#pragma unroll
                    for (int k = 1; k < kAttnWaves; ++k) v += *reinterpret_cast<const f32x4 *>(&buf.o[k][row - 16 * r][col]);
                    float best = buf.m[0][row], total = 0.0f;
#pragma unroll
                    for (int k = 1; k < kAttnWaves; ++k) best = __builtin_fmaxf(best, buf.m[k][row]);
#pragma unroll
                    for (int k = 0; k < kAttnWaves; ++k) {
                        const float mk = buf.m[k][row];
                        total += buf.l[k][row] * (mk == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mk - best));
                    }
                    if (slot >= 0) {
                        *reinterpret_cast<f32x4 *>(a.part + (slot * kRows + row) * kDp + 16 * b0 + col) = v;
                        if (b0 == 0 && col == 0) {
                            a.ml[(slot * kRows + row) * 2] = best;
                            a.ml[(slot * kRows + row) * 2 + 1] = total;
                        }
                    } else if (16 * b0 + col < a.c.head_dim) {
                        const int i = static_cast<int>((static_cast<uint32_t>(row) * a.group_inverse) >> 26);
                        const int head = kvh * a.group + (row - i * a.group);
                        store4(a.out + static_cast<int64_t>(s.first + i) * a.o_token + head * a.o_head + 16 * b0 + col,
                               total == 0.0f ? f32x4{0, 0, 0, 0} : v * (1.0f / total) * g, bf16, a.o_wide);
                    }
                }
                __syncthreads();
            }
        }
        // the last round's barrier also frees m and l; without a round nothing reads them
        if (rows <= 0) __syncthreads();
    }
};

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v)),
                   hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Sums over the lanes, and over the lanes up to and with each.
__device__ __forceinline__ uint32_t wave_upto(uint32_t v) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t x = static_cast<uint32_t>(__shfl_up(static_cast<int>(v), o, kWave));
        v += lane >= o ? x : 0u;
    }
    return v;
}
__device__ __forceinline__ int64_t wave_total(int v) {   // 64 values below 2^25
    uint32_t x = static_cast<uint32_t>(v);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) x += static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), o, kWave));
    return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(x)));
}

// count(b) of up to 64 sequences from b0 on, one a lane, and their sum over the lanes
// up to and with each (below 64 * 2^25).
struct Counts {
    uint32_t own, upto;
    __device__ __forceinline__ uint32_t all() const {
        return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), kWave - 1));
    }
};
template <typename Count>
__device__ __forceinline__ Counts counts_from(int b0, int batch, Count count) {
    const int lane = threadIdx.x & (kWave - 1);
    Counts c;
    c.own = b0 + lane < batch ? static_cast<uint32_t>(count(b0 + lane)) : 0u;
    c.upto = wave_upto(c.own);
    return c;
}
// The sequence that holds `at` where each counts count(b), and where its counts begin;
// batch if none does.  Every wave finds it by itself.
template <typename Count>
__device__ __forceinline__ int sequence_with(int64_t at, int batch, Count count, int64_t *before) {
    int64_t base = 0;
    for (int b0 = 0; b0 < batch; b0 += kWave) {
        const Counts c = counts_from(b0, batch, count);
        const uint64_t past = __ballot(base + static_cast<int64_t>(c.upto) > at);
        if (past != 0) {
            const int n = __builtin_ctzll(past);
            *before = uniform64(base + static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(c.upto - c.own), n)));
            return b0 + n;
        }
        base += c.all();
    }
    return batch;
}

// One workgroup a sequence and kv head, all of its steps: caches of up to 512 tokens, where
// a second launch to join pieces would cost as much as the steps (100 tokens: 5.5 us).
template <int NB, int R>
__global__ __launch_bounds__(kAttnThreads, nvfp4attnplan::groups_per_unit(16 * NB, 16 * R)) void attn_whole(const AttnArgs a) {
    using S = Stream<NB, R>;
    __shared__ typename S::Buffers buf;
    const int b = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x - b * a.c.kv_heads;
    const Sequence s = sequence_of(a, b);
    const Steps w = steps_for<6>(a, s);
    S job;
    job.run(a, buf, s, w, b, kvh, 0, w.count, -1);
}

// Steps of a piece: the steps of all sequences and kv heads over the pieces wanted, a
// step for each wave at least.
__device__ __forceinline__ int piece_steps(int64_t total, int pieces) {
    const int64_t each = total >> 31 == 0 ? static_cast<uint32_t>(total + pieces - 1) / static_cast<uint32_t>(pieces)
                                          : (total + pieces - 1) / pieces;
    // a sequence has less than 2^26 steps
    return each < kAttnWaves ? kAttnWaves : each < (1 << 26) ? static_cast<int>(each) : 1 << 26;
}

// By one wave.  The first workgroup's also leaves the pieces before each sequence for
// attn_join.
__device__ __forceinline__ Piece find_piece(const AttnArgs &a) {
    const int lane = threadIdx.x & (kWave - 1);
    // the first 64 sequences stay in registers, one a lane
    Sequence own = {};
    int steps = 0;
    if (lane < a.batch) {
        own = sequence_of(a, lane);
        steps = steps_for<6>(a, own).count;
    }
    const auto count = [&](int b) { return steps_for<6>(a, sequence_of(a, b)).count; };
    int64_t total = wave_total(steps);
    for (int b = kWave + lane; b - lane < a.batch; b += kWave) total += wave_total(b < a.batch ? count(b) : 0);
    const int each = piece_steps(total * a.c.kv_heads, a.groups);

    Piece p = {-1, 0, 0, 0, {}};
    int64_t before = 0;                                // pieces of one kv head of the sequences before
    for (int b0 = 0; b0 < a.batch; b0 += kWave) {
        const int n = b0 == 0 ? steps : b0 + lane < a.batch ? count(b0 + lane) : 0;
        const uint32_t mine = static_cast<uint32_t>(n + each - 1) / static_cast<uint32_t>(each);   // n < 2^25
        const uint32_t upto = wave_upto(mine);
        const int64_t end = (before + upto) * a.c.kv_heads;
        if (blockIdx.x == 0 && b0 + lane < a.batch) a.prefix[b0 + lane] = before + upto - mine;
        const uint64_t past = __ballot(end > static_cast<int64_t>(blockIdx.x));
        if (past != 0 && p.b < 0) {
            const int k = __builtin_ctzll(past);
            p.b = b0 + k;
            p.pieces = __builtin_amdgcn_readlane(static_cast<int>(mine), k);
            const int64_t start = (before + static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto - mine), k))) * a.c.kv_heads;
            const uint32_t at = static_cast<uint32_t>(static_cast<int64_t>(blockIdx.x) - start);
            p.kvh = static_cast<int>(at / static_cast<uint32_t>(p.pieces));
            p.part = static_cast<int>(at) - p.kvh * p.pieces;
            if (blockIdx.x != 0) break;                // the first workgroup goes on with the prefix
        }
        before += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), kWave - 1));
    }
    if (blockIdx.x == 0 && lane == 0) a.prefix[a.batch] = before;
    if (p.b >= kWave) {
        p.s = sequence_of(a, p.b);
    } else if (p.b >= 0) {
        p.s.len = __builtin_amdgcn_readlane(own.len, p.b);
        p.s.first = __builtin_amdgcn_readlane(own.first, p.b);
        p.s.n = __builtin_amdgcn_readlane(own.n, p.b);
        p.s.computed = __builtin_amdgcn_readlane(own.computed, p.b);
    }
    return p;
}

// Every sequence and kv head in pieces of nearly equal length, one a workgroup, about as
// many as the chip holds at once: twice as many cost a start and an end more each
// (131072 tokens: 47 us against 42; speculative tokens 49 against 36).  A sequence in
// one piece is finished by it, those in several leave partial results for attn_join.
// The pieces follow from the lengths on the device.
//
// A step of 64 tokens and 128 elements takes some 600 vector instructions a wave, most of
// them the decode of two 4-bit codes at a time and the products with their scales, and 32
// matrix ones.  64 histories of up to 4096 tokens, 32 heads on 8 of 128 (192 MB): 51 us,
// 3.8 TB/s, and 5 for attn_join; together 55, 44 with the arithmetic of the steps left out
// and 45 with their loads left out but the first (one query on 131072 tokens: 41, 33 and
// 37).  Either alone takes most of the time, and they overlap only in part: vector
// instructions are issued for 0.53 of the time, and a wave waits for 0.44 of its own.
template <int NB, int R>
__global__ __launch_bounds__(kAttnThreads, nvfp4attnplan::groups_per_unit(16 * NB, 16 * R)) void attn_pieces(const AttnArgs a) {
    using S = Stream<NB, R>;
    __shared__ typename S::Buffers buf;
    if (threadIdx.x < kWave) {                         // one wave finds it for all
        const Piece p = find_piece(a);
        if (threadIdx.x == 0) buf.piece = p;
    }
    __syncthreads();
    const Piece piece = buf.piece;
    __syncthreads();                                   // before the stages take its place
    const int b = __builtin_amdgcn_readfirstlane(piece.b);
    if (b < 0) return;
    const Sequence s = {__builtin_amdgcn_readfirstlane(piece.s.len), __builtin_amdgcn_readfirstlane(piece.s.first),
                        __builtin_amdgcn_readfirstlane(piece.s.n), __builtin_amdgcn_readfirstlane(piece.s.computed)};
    const int kvh = __builtin_amdgcn_readfirstlane(piece.kvh), part = __builtin_amdgcn_readfirstlane(piece.part),
              pieces = __builtin_amdgcn_readfirstlane(piece.pieces);
    const Steps w = steps_for<6>(a, s);
    // pieces of a sequence differ by a step at most
    const int base = w.count / pieces, longer = w.count - base * pieces;
    const int i0 = part * base + (part < longer ? part : longer), i1 = i0 + base + (part < longer ? 1 : 0);
    S job;
    job.run(a, buf, s, w, b, kvh, i0, i1, pieces == 1 ? -1 : static_cast<int64_t>(blockIdx.x));
}

// Weighted sum of `n` partial results (sums from `part` on, `stride` floats apart, and
// maximum and sum at `ml`, `ml_stride` apart) of one row: WAVES waves take the results in
// turn, a lane NB / 4 outputs.  The loads of up to 8 results a wave, and of the maxima,
// are on their way together (past the last result they read it again, with no weight).
template <int NB, int WAVES>
struct Joiner {
    static constexpr int kDp = 16 * NB, kEach = NB / 4;
    typedef float Vec __attribute__((ext_vector_type(kEach)));
    struct Buffers {
        Vec sums[WAVES][kWave];
        float total[WAVES];
    };

    template <int AHEAD>
    static __device__ __forceinline__ void sum(const float *part, int64_t stride, const float *ml, int64_t ml_stride, int n,
                                               int wave, Vec &v, float &total) {
        const int lane = threadIdx.x & (kWave - 1);
        Vec ahead[AHEAD];
        f32x2 ahead_ml[AHEAD];
        const auto fetch = [&](int base) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int k = base + wave + i * WAVES, at = k < n ? k : n - 1;
                const float *p = part + at * stride + kEach * lane;
                if constexpr (kEach == 3) {
#pragma unroll
                    for (int j = 0; j < 3; ++j) ahead[i][j] = p[j];
                } else {
                    ahead[i] = *reinterpret_cast<const Vec *>(p);
                }
                ahead_ml[i] = *reinterpret_cast<const f32x2 *>(ml + at * ml_stride);
            }
        };
        fetch(0);
        float top = -__builtin_inff();
        for (int k = lane; k < n; k += kWave) top = __builtin_fmaxf(top, ml[k * ml_stride]);
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, kWave));
        for (int base = 0;;) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float m = ahead_ml[i][0];
                const bool none = base + wave + i * WAVES >= n;
                const float f = none || m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - top);
                v += none ? Vec{} : ahead[i] * f;
                total += none ? 0.0f : ahead_ml[i][1] * f;
            }
            base += AHEAD * WAVES;
            if (base >= n) break;
            fetch(base);
        }
    }

    // The row's outputs of this lane; true in the first of the waves, `wave` 0, only.
    // One wave exchanges nothing: `buf` may be NULL.
    static __device__ __forceinline__ bool run(Buffers *buf, const float *part, int64_t stride, const float *ml,
                                               int64_t ml_stride, int n, int wave, Vec *out, float *total) {
        const int lane = threadIdx.x & (kWave - 1);
        Vec v = {};
        float sum = 0.0f;
        if (n > 2 * WAVES) {
            Joiner::template sum<8>(part, stride, ml, ml_stride, n, wave, v, sum);
        } else if (n > WAVES) {
            Joiner::template sum<2>(part, stride, ml, ml_stride, n, wave, v, sum);
        } else if (n > 0) {
            Joiner::template sum<1>(part, stride, ml, ml_stride, n, wave, v, sum);
        }
        if constexpr (WAVES > 1) {
            if (wave > 0) {
                buf->sums[wave][lane] = v;
                if (lane == 0) buf->total[wave] = sum;
            }
            __syncthreads();
            if (wave > 0) return false;
#pragma unroll
            for (int k = 1; k < WAVES; ++k) {
                v += buf->sums[k][lane];
                sum += buf->total[k];
            }
        }
        *out = v;
        *total = sum;
        return true;
    }

    static __device__ __forceinline__ void store(const AttnArgs &a, const Sequence &s, int kvh, int row, Vec v, float total) {
        const int lane = threadIdx.x & (kWave - 1), e = kEach * lane;
        const int i = row / a.group, head = kvh * a.group + (row - i * a.group);
        const float g = a.c.v_global != nullptr ? a.c.v_global[kvh] : 1.0f;
        uint16_t *out = a.out + static_cast<int64_t>(s.first + i) * a.o_token + head * a.o_head + e;
        v = total == 0.0f ? Vec{} : v * (1.0f / total) * g;
        // rows that may be written 16 bytes at a time may be written 4
        if (kEach == 2 && a.o_wide) {
            if (e < a.c.head_dim)
                *reinterpret_cast<uint32_t *>(out) = pair16(v[0], v[kEach - 1], a.bf16 != 0);
            return;
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (e + j < a.c.head_dim) out[j] = static_cast<uint16_t>(to16(v[j], a.bf16 != 0));
    }
};

// A chain of latencies: lengths, the pieces' statistics, their sums (5 - 6.5 us).
// One workgroup a query row (`used` of the `rows` that a partial result holds): the
// results of its pieces joined, or zeros where there are none.
template <int NB>
__global__ __launch_bounds__(kAttnThreads) void attn_join(const AttnArgs a, int rows, int used) {
    using J = Joiner<NB, kAttnWaves>;
    __shared__ typename J::Buffers buf;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int item = blockIdx.x / used, row = blockIdx.x - item * used;
    const int b = item / a.c.kv_heads, kvh = item - b * a.c.kv_heads;
    const int64_t before = a.prefix[b];
    const int pieces = static_cast<int>(a.prefix[b + 1] - before);
    if (pieces == 1) return;                           // finished by its workgroup
    const Sequence s = sequence_of(a, b);
    if (row >= s.computed * a.group) return;
    const int64_t first = before * a.c.kv_heads + static_cast<int64_t>(kvh) * pieces;
    typename J::Vec v;
    float total;
    if (J::run(&buf, a.part + (first * rows + row) * J::kDp, static_cast<int64_t>(rows) * J::kDp,
               a.ml + (first * rows + row) * 2, 2 * rows, pieces, wave, &v, &total))
        J::store(a, s, kvh, row, v, total);
}

// A barrier that orders the workgroup's LDS accesses and waits for them alone:
// __syncthreads also waits for the codes on their way from memory.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---------------------------------------------------------------- the tile kernel
//
// Many query rows: a workgroup holds 32 of them a wave and walks the cache in steps
// of T tokens, which its waves decode once into LDS, as fp16, for all of them: K as
// [token][element], V turned, as [element][token].  Products run on the 32 x 32
// matrix instructions.  Codes are loaded two steps ahead into registers and decoded
// one step ahead into the other of two buffers, so that one barrier a step is
// enough; one half of the waves decodes before its products and the other after them,
// so that the two waves of a SIMD need the VALU and the matrix cores at different
// times (a prompt of 4096 tokens, 32 heads on 8 of 128: 208 us in step, 190 so).  8 waves
// of 256 rows decode a step half as often as 4 of 128 (221 us), which are taken where 256
// would leave compute units idle.
template <int NB, int WAVES>
struct Tile {
    static constexpr int kDp = 16 * NB;
    static constexpr int kLog = NB <= 8 ? 6 : 5;   // more tokens' scores do not fit the registers
    static constexpr int kT = 1 << kLog;
    static constexpr int kRuns = kT / kRun;
    static constexpr int kRows = 32 * WAVES;
    static constexpr int kUnits = 2 * kRuns;       // runs of K, then of V, that are decoded by a wave each
    static constexpr int kOwn = (kUnits + WAVES - 1) / WAVES;
    static constexpr int kPieces = (kDp / 2 + kWave - 1) / kWave;   // 16-byte pieces of a run's codes a lane has
    static constexpr int kSlices = kDp / 16;       // k steps of the first product
    static constexpr int kOuts = kDp / 32;         // output tiles of 32 elements
    static constexpr int kRead = NB / 4;           // transposed reads of a lane: blocks of 16 over four lane groups

    struct Buffers {
        __attribute__((aligned(16))) _Float16 k[2][kT * kDp];
        __attribute__((aligned(16))) _Float16 v[2][kT * kDp];
        __attribute__((aligned(16))) uint8_t raw[kRuns][kRun * kDp / 2];
        uint32_t bad[2][kRuns];            // whether a run of V holds NaN, and which tokens of which block
        uint16_t nan[2][kRuns][NB];
    };

    // a unit's codes and scales on their way
    u32x4 code[kOwn][kPieces];
    u32x4 scale[kOwn][kPieces > kRead ? kPieces : kRead];   // of K one word of two bytes each

    int wave;
    f16x8 q[kSlices];
    float c;
    int pos;
    f32x16 sc[kT / 32];                            // a step's scores, then its weights
    f16x8 p[kT / 16];
    f32x16 acc[kOuts];
    float m, l;

    static __device__ __forceinline__ uint32_t k_at(uint32_t token, uint32_t chunk) {   // chunks of 8 elements
        const uint32_t f = NB == 8 || NB == 16 ? token & 15 : (token >> 1) & 7;
        return token * kDp + 8 * (chunk ^ f);
    }
    static __device__ __forceinline__ uint32_t v_at(uint32_t element, uint32_t chunk) {   // chunks of 8 tokens
        const uint32_t f = kT == 64 ? (element >> 1) & 7 : (element >> 2) & 3;
        return element * kT + 8 * (chunk ^ f);
    }
    static __device__ __forceinline__ uint32_t raw_at(uint32_t token, uint32_t piece) {
        constexpr int kEach = kDp / 32;
        const uint32_t f = kEach == 2 ? (token >> 3) & 1 : kEach == 4 ? (token >> 2) & 3
                           : kEach == 6 ? (token >> 3) & 1 : (token >> 1) & 7;
        return token * (kDp / 2) + 16 * (piece ^ f);
    }

    // Bytes of an element's offset that a row's turn by up to TURN chunks of 16 changes.
    template <int TURN>
    static __device__ __forceinline__ uint32_t turned_low(uint32_t elements) {
        return 2 * elements & (16 * TURN);
    }

    // The page of step s that run lane % kRuns lies in, -1 without one.
    __device__ __forceinline__ int entry(const AttnArgs &a, const int32_t *row, int len, int s) const {
        const int token = s * kT + kRun * static_cast<int>(this_lane().id % kRuns);
        int i = token >> a.c.page_log2;
        i = i < a.table_width ? i : a.table_width - 1;
        const int p = row[i];
        return token < len && p >= 0 && p < a.pages ? p : -1;
    }

    __device__ __forceinline__ void load(const AttnArgs &a, int kvh, int s, int e) {
        const Lane n = this_lane();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int unit = wave + o * WAVES;
            if (unit >= kUnits) break;
            const bool is_v = unit >= kRuns;
            const int run = is_v ? unit - kRuns : unit;
            int page = __builtin_amdgcn_readlane(e, run);
            page = page < 0 ? 0 : page;
            const uint64_t head = static_cast<uint64_t>(static_cast<uint32_t>(page)) * static_cast<uint32_t>(a.c.kv_heads) +
                                  static_cast<uint32_t>(kvh);
            const uint64_t tokens = head << a.c.page_log2;
            const uint32_t off = (s * kT + kRun * run) & ((1 << a.c.page_log2) - 1);
            const uint8_t *codes = (is_v ? a.c.v_codes : a.c.k_codes) + (tokens + off) * (kDp / 2);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t at = i * kWave + n.id;
                if ((i + 1) * kWave <= kDp / 2 || at < kDp / 2)
                    code[o][i] = *reinterpret_cast<const u32x4 *>(codes + 16 * at);
            }
            if (is_v) {
                const uint8_t *scales = a.c.v_scales + tokens * NB + off;
#pragma unroll
                for (int i = 0; i < kRead; ++i)
                    scale[o][i] = *reinterpret_cast<const u32x4 *>(scales + ((4 * i + n.h) << a.c.page_log2));
            } else {
                const uint8_t *scales = a.c.k_scales + tokens * NB + off;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint32_t at = i * kWave + n.id, token = at / (kDp / 32), piece = at % (kDp / 32);
                    if ((i + 1) * kWave <= kDp / 2 || at < kDp / 2) {
                        scale[o][i][0] = scales[((2 * piece) << a.c.page_log2) + token];
                        scale[o][i][1] = scales[((2 * piece + 1) << a.c.page_log2) + token];
                    }
                }
            }
        }
    }

    // Decodes the loaded units into buffer `to`.
    __device__ __forceinline__ void decode(Buffers &buf, int to) {
        typedef __attribute__((address_space(3))) i32x2 lds2;
        const Lane n = this_lane();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int unit = wave + o * WAVES;
            if (unit >= kUnits) break;
            if (unit < kRuns) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint32_t at = i * kWave + n.id, token = at / (kDp / 32), piece = at % (kDp / 32);
                    if ((i + 1) * kWave <= kDp / 2 || at < kDp / 2) {
                        const _Float16 s0 = nvfp4dev::e4m3x2_f16(scale[o][i][0])[0], s1 = nvfp4dev::e4m3x2_f16(scale[o][i][1])[0];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const f16x2 ss = j < 2 ? f16x2{s0, s0} : f16x2{s1, s1};
                            *reinterpret_cast<f16x8 *>(&buf.k[to][k_at(kRun * unit + token, 4 * piece + j)]) =
                                decode8(code[o][i][j], ss, ss, ss, ss);
                        }
                    }
                }
            } else {
                const int run = unit - kRuns;
                uint8_t *raw = buf.raw[run];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint32_t at = i * kWave + n.id;
                    if ((i + 1) * kWave <= kDp / 2 || at < kDp / 2)
                        *reinterpret_cast<u32x4 *>(raw + raw_at(at / (kDp / 32), at % (kDp / 32))) = code[o][i];
                }
                wave_fence();
                // tokens in the order in which the scores leave the first product: 0-3, 8-11, 4-7, 12-15
                const uint32_t token = (n.r16 & 3) | (n.r16 & 4) << 1 | (n.r16 & 8) >> 1;
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < kRead; ++i) {
                    const uint32_t block = 4 * i + n.h;
                    const i32x2 w = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds2 *)(raw + raw_at(token, block / 2) + 8 * (block % 2)));
                    // a NaN block counts as 0 here; who sees it is told by its flags
                    u32x4 x = scale[o][i];
                    uint32_t bad = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t nan = ((x[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        any |= nan;
                        bad |= nan >> (7 - k);         // bits k, 8 + k, 16 + k, 24 + k: tokens 4 k ..
                        x[k] &= ~(nan | (nan - (nan >> 7)));
                    }
                    if (n.r16 == 0) {
                        uint32_t bits = 0;
                        if (bad != 0) {
                            for (int k = 0; k < 4; ++k)
                                for (int j = 0; j < 4; ++j) bits |= (bad >> (8 * j + k) & 1u) << (4 * k + j);
                        }
                        buf.nan[to][run][block] = static_cast<uint16_t>(bits);
                    }
                    const f16x8 lo = decode8(static_cast<uint32_t>(w[0]), nvfp4dev::e4m3x2_f16(x[0]), e4m3_high_f16(x[0]),
                                             nvfp4dev::e4m3x2_f16(x[2]), e4m3_high_f16(x[2]));
                    const f16x8 hi = decode8(static_cast<uint32_t>(w[1]), nvfp4dev::e4m3x2_f16(x[1]), e4m3_high_f16(x[1]),
                                             nvfp4dev::e4m3x2_f16(x[3]), e4m3_high_f16(x[3]));
                    const uint32_t element = 16 * block + n.r16;
                    *reinterpret_cast<f16x8 *>(&buf.v[to][v_at(element, 2 * run)]) = lo;
                    *reinterpret_cast<f16x8 *>(&buf.v[to][v_at(element, 2 * run + 1)]) = hi;
                }
                const bool some = __any(any != 0);
                if (n.id == 0) buf.bad[to][run] = some ? 1u : 0u;
            }
        }
    }

    __device__ __forceinline__ void load_query(const AttnArgs &a, const Sequence &s, int kvh, int row) {
        const Lane n = this_lane();
        const uint32_t h = n.id >> 5;
        const float g = a.scale * (a.c.k_global != nullptr ? a.c.k_global[kvh] : 1.0f);
        const int i = row / a.group, head = kvh * a.group + (row - i * a.group);
        pos = -1;
        u32x4 raw[kSlices];
#pragma unroll
        for (int j = 0; j < kSlices; ++j) raw[j] = u32x4{0, 0, 0, 0};
        if (row < s.computed * a.group) {
            const int at = s.len - s.n + i;
            pos = at < 0 ? -1 : at;
            const uint16_t *p = a.q + static_cast<int64_t>(s.first + i) * a.q_token + head * a.q_head;
#pragma unroll
            for (int j = 0; j < kSlices; ++j)
                if (16 * j < a.c.head_dim) raw[j] = load8(p + 16 * j + 8 * h, a.q_wide);
        }
        float down = 1.0f;
        if (a.bf16 != 0) {
            const uint32_t top = top16(raw), other = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave));
            float up;
            row_power((other > top ? other : top) << 16, &up, &down);
            up = g < 0.0f ? -up : up;
#pragma unroll
            for (int j = 0; j < kSlices; ++j) q[j] = scale_bf16(raw[j], up);
        } else {
            const uint32_t sign = g < 0.0f ? 0x80008000u : 0u;
#pragma unroll
            for (int j = 0; j < kSlices; ++j) q[j] = __builtin_bit_cast(f16x8, raw[j] ^ sign);
        }
        c = __builtin_fabsf(g) * kLog2e * down;
        c = c == 0.0f ? 0x1p-126f : c;                 // as in the stream kernel
        if (!(__builtin_fabsf(g) < __builtin_inff())) {
            c = 1.0f;
#pragma unroll
            for (int j = 0; j < kSlices; ++j) q[j] = nan8();
        }
    }

    // Operands are read kAhead products before they are needed.  A read's address is the
    // lane's row, its place turned by the chunk's low bits, and a constant.  Heads of more
    // than 192 have registers for three (4096 tokens, 16 heads on 4 of 256: 329 us with 27
    // of them spilled, 378 with four, 342 with two; five ragged prompts of up to 701 tokens,
    // 12 heads on 3: 112, 120 and 117).
    static constexpr int kAhead = NB <= 8 ? 8 : NB <= 12 ? 4 : 3;
    static constexpr int kTurnK = NB == 8 || NB == 16 ? 15 : 7, kTurnV = kT == 64 ? 7 : 3;

    // Scores of K in buffer `from`.
    __device__ __forceinline__ void scores(const Buffers &buf, int from) {
        const Lane n = this_lane();
        const uint32_t at = k_at(n.id & 31, n.id >> 5), low = turned_low<kTurnK>(at);
        const uint8_t *row = reinterpret_cast<const uint8_t *>(&buf.k[from][at]);
        constexpr int kU = kT / 32;
        const auto read = [&](int i) {             // product i: tokens 32 (i mod kU) .., elements 16 (i / kU) ..
            const int u = i % kU, chunk = 2 * (i / kU);
            return *reinterpret_cast<const f16x8 *>(row + ((low ^ (16 * (chunk & kTurnK))) - low) +
                                                    (16 * (chunk & ~kTurnK) + 64 * u * kDp));
        };
        constexpr int kProducts = kT / 32 * kSlices;
        f16x8 ahead[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ahead[i] = read(i);
#pragma unroll
        for (int u = 0; u < kT / 32; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[u][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kProducts; ++i) {
            __builtin_amdgcn_sched_barrier(kAluCrosses);
            sc[i % kU] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ahead[i % kAhead], q[i / kU], sc[i % kU], 0, 0, 0);
            if (i + kAhead < kProducts) ahead[i % kAhead] = read(i + kAhead);
        }
    }

    // Softmax of the scores of step s: the running maximum and sum, the weights.
    // `there`: bit r where run r's page is.
    __device__ __forceinline__ void weigh(const AttnArgs &a, int s, uint64_t there, int p_first, int p_last) {
        const int tok0 = s * kT;
        const uint64_t all = (uint64_t(1) << kRuns) - 1;
        const bool whole = (there & all) == all && tok0 + kT - 1 <= p_first &&
                           (a.window == 0 || tok0 > p_last - a.window || tok0 + kT - 1 < a.sinks);
        if (!whole) {
            const int h = static_cast<int>(this_lane().id >> 5);
#pragma unroll
            for (int u = 0; u < kT / 32; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int token = 32 * u + 8 * (i / 4) + 4 * h + i % 4;
                    if (!((there >> (token / kRun)) & 1u) || !visible(a, pos, tok0 + token)) sc[u][i] = -__builtin_inff();
                }
        }
        float top = sc[0][0];
#pragma unroll
        for (int u = 0; u < kT / 32; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, sc[u][i]);
        top = xor32(top, true);
        top = top == -__builtin_inff() ? top : top * c;
        const bool grown = top - m > kRescaleAt;       // also of a first score; not of NaN, nor of none
        if (__any(grown)) {
            const float to = grown ? top : m;
            const float f = grown ? __builtin_amdgcn_exp2f(m - to) : 1.0f;
            m = to;
            l *= f;
#pragma unroll
            for (int o = 0; o < kOuts; ++o)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[o][i] *= f;
        }
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float factor = c, shift = kWeightShift - base;
        if (__any(far_maximum(base))) {
#pragma unroll
            for (int u = 0; u < kT / 32; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) sc[u][i] = far_maximum(base) ? sc[u][i] * c - base : sc[u][i];
            factor = far_maximum(base) ? 1.0f : factor;
            shift = far_maximum(base) ? kWeightShift : shift;
        }
        float sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kT / 32; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][i], factor, shift));
                sum[i % 4] += e;
                p[2 * u + i / 8][i % 8] = static_cast<_Float16>(e);
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    // The weights of step s times V in buffer `from`.
    __device__ __forceinline__ void sums(const AttnArgs &a, const Buffers &buf, int from, int s, uint64_t there) {
        const Lane n = this_lane();
        const uint32_t at = v_at(n.id & 31, n.id >> 5), low = turned_low<kTurnV>(at);
        const uint8_t *row = reinterpret_cast<const uint8_t *>(&buf.v[from][at]);
        const auto read = [&](int i) {
            const int o = i % kOuts, chunk = 2 * (i / kOuts);
            return *reinterpret_cast<const f16x8 *>(row + ((low ^ (16 * (chunk & kTurnV))) - low) +
                                                    (16 * (chunk & ~kTurnV) + 64 * o * kT));
        };
        constexpr int kSums = kT / 16 * kOuts;
        f16x8 ahead[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < kSums) ahead[i] = read(i);
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            acc[i % kOuts] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ahead[i % kAhead], p[i / kOuts], acc[i % kOuts], 0, 0, 0);
            if (i + kAhead < kSums) ahead[i % kAhead] = read(i + kAhead);
            __builtin_amdgcn_sched_barrier(kAluCrosses);
        }
        uint32_t bad = 0;
#pragma unroll
        for (int r = 0; r < kRuns; ++r) bad |= buf.bad[from][r];
        if (__builtin_amdgcn_readfirstlane(static_cast<int>(bad)) != 0) poison(a, buf, from, s * kT, there);
    }

    // Rows that see a token whose block of V is NaN: NaN there.
    __device__ __forceinline__ void poison(const AttnArgs &a, const Buffers &buf, int from, int tok0, uint64_t there) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
            for (int run = 0; run < kRuns; ++run) {
                uint32_t bits = __builtin_amdgcn_readfirstlane(static_cast<int>(buf.nan[from][run][b]));
                if (!((there >> run) & 1u)) bits = 0;
                while (bits != 0) {
                    const int j = tok0 + kRun * run + __builtin_ctz(bits);
                    bits &= bits - 1;
                    if (visible(a, pos, j)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[b / 2][8 * (b % 2) + i] = __uint_as_float(0x7FC00000u);
                    }
                }
            }
    }

    // Steps i0 .. i1 of the list for the rows from row0 on; results to `out`, or where
    // `part` is not NULL there ([kRows][dp] sums, then [kRows][2] maximum and sum).
    __device__ __forceinline__ void run(const AttnArgs &a, Buffers &buf, const Sequence &s, const Steps &w, int b, int kvh,
                                        int row0, int i0, int i1, float *part) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int32_t *table = a.table + static_cast<int64_t>(b) * a.table_stride;
        const Lane n = this_lane();
        const int first = row0 + 32 * wave, row = first + static_cast<int>(n.id & 31);
        load_query(a, s, kvh, row);
        // positions of this wave's first and last query
        const int last_row = s.computed * a.group - 1;
        const int end = first + 31 < last_row ? first + 31 : last_row;
        const int p_first = s.len - s.n + first / a.group;
        const int p_last = first <= last_row ? s.len - s.n + end / a.group : -1;
        m = -__builtin_inff();
        l = 0.0f;
#pragma unroll
        for (int o = 0; o < kOuts; ++o)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[o][i] = 0.0f;
        if (i0 < i1) {
            uint64_t there, there_next = 0;
            {
                const int e = entry(a, table, s.len, w.at(i0));
                there = __ballot(e >= 0);
                load(a, kvh, w.at(i0), e);
                decode(buf, 0);
            }
            if (i0 + 1 < i1) {
                const int e = entry(a, table, s.len, w.at(i0 + 1));
                there_next = __ballot(e >= 0);
                load(a, kvh, w.at(i0 + 1), e);
            }
            int e_after = i0 + 2 < i1 ? entry(a, table, s.len, w.at(i0 + 2)) : -1;
            lds_barrier();
            for (int i = i0; i < i1; ++i) {
                const int from = (i - i0) & 1;
                const auto ahead = [&]() {
                    if (i + 1 < i1) decode(buf, from ^ 1);
                    if (i + 2 < i1) load(a, kvh, w.at(i + 2), e_after);
                };
                const bool early = wave >= WAVES / 2;
                if (early) ahead();
                if (w.at(i) * kT <= p_last) {
                    scores(buf, from);
                    weigh(a, w.at(i), there, p_first, p_last);
                    sums(a, buf, from, w.at(i), there);
                }
                if (!early) ahead();
                there = there_next;
                there_next = __ballot(e_after >= 0);
                if (i + 3 < i1) e_after = entry(a, table, s.len, w.at(i + 3));
                lds_barrier();
            }
        }
        // this lane's row: elements 32 o + 8 j + 4 h ..
        const uint32_t h = this_lane().id >> 5;
        const float total = xor32(l, false);
        if (part != nullptr) {
            const int at = 32 * wave + static_cast<int>(n.id & 31);
            float *ml = part + kRows * kDp;
            if (h == 0) {
                ml[2 * at] = m;
                ml[2 * at + 1] = total;
            }
#pragma unroll
            for (int o = 0; o < kOuts; ++o)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<f32x4 *>(part + at * kDp + 32 * o + 8 * j + 4 * h) =
                        f32x4{acc[o][4 * j], acc[o][4 * j + 1], acc[o][4 * j + 2], acc[o][4 * j + 3]};
            return;
        }
        if (row > last_row) return;
        const float g = a.c.v_global != nullptr ? a.c.v_global[kvh] : 1.0f;
        const float inv = 1.0f / total;
        const int i = row / a.group, head = kvh * a.group + (row - i * a.group);
        uint16_t *out = a.out + static_cast<int64_t>(s.first + i) * a.o_token + head * a.o_head;
#pragma unroll
        for (int o = 0; o < kOuts; ++o)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = 32 * o + 8 * j + 4 * static_cast<int>(h);
                if (e < a.c.head_dim)
                    store4(out + e,
                           total == 0.0f ? f32x4{0, 0, 0, 0}
                                         : f32x4{acc[o][4 * j], acc[o][4 * j + 1], acc[o][4 * j + 2], acc[o][4 * j + 3]} * inv * g,
                           a.bf16 != 0, a.o_wide);
            }
    }
};

// Floats of a partial result of the tile kernel.
constexpr int64_t tile_part(int64_t rows, int64_t dp) { return rows * (dp + 2); }

// The sequence, first row and kv head of a workgroup of the tile kernel, b = batch
// past the last.  Tiles are numbered from the last, so that those that see the most
// of a prompt come first; workgroups next to each other take the kv heads.
struct TileJob {
    int b, kvh, row0;
};
__device__ __forceinline__ TileJob tile_job(const AttnArgs &a, int item, int tiles, int rows) {
    TileJob j;
    j.kvh = item % a.c.kv_heads;
    const int tile = tiles - 1 - item / a.c.kv_heads;
    const auto count = [&](int b) {
        return static_cast<int>((static_cast<int64_t>(sequence_of(a, b).computed) * a.group + rows - 1) / rows);
    };
    int64_t before = 0;
    j.b = __builtin_amdgcn_readfirstlane(sequence_with(tile, a.batch, count, &before));
    j.row0 = (tile - static_cast<int>(before)) * rows;
    return j;
}

// `tiles` bounds the tiles of all sequences; `splits` workgroups share a tile's steps.
// Many queries of a sequence: 32 rows a wave on the 32x32x16 instructions, and each step
// of the cache decoded once into LDS for all waves.  A prompt of 4096 tokens, 32 heads on
// 8 of 128: 180 - 190 us, 730 TFLOP/s; vector instructions (softmax, decode) are issued for
// 0.55 of the time and the matrix cores run for 0.33 of it, and the two hardly overlap
// within a wave, since a step's scores, weights and sums follow from each other.
template <int NB, int WAVES>
__global__ __launch_bounds__(WAVES * kWave, 2) void attn_tiles(const AttnArgs a, int tiles, int splits) {
    using T = Tile<NB, WAVES>;
    __shared__ typename T::Buffers buf;
    const int item = blockIdx.x / splits, split = blockIdx.x - item * splits;
    const TileJob j = tile_job(a, item, tiles, T::kRows);
    if (j.b >= a.batch) return;
    const Sequence s = sequence_of(a, j.b);
    const Steps w = steps_for<T::kLog>(a, s, j.row0, T::kRows);
    const int i0 = static_cast<int>(static_cast<int64_t>(w.count) * split / splits);
    const int i1 = static_cast<int>(static_cast<int64_t>(w.count) * (split + 1) / splits);
    T job;
    job.run(a, buf, s, w, j.b, j.kvh, j.row0, i0, i1,
            splits > 1 ? a.part + static_cast<int64_t>(blockIdx.x) * tile_part(T::kRows, T::kDp) : nullptr);
}

// Rows of a tile whose steps were shared, kJoinRows a workgroup, each by a wave: their
// partial results joined.
constexpr int kJoinRows = 8;
template <int NB>
__global__ __launch_bounds__(kAttnThreads) void attn_join_tiles(const AttnArgs a, int tiles, int splits, int rows) {
    using J = Joiner<NB, 1>;
    const int chunks = rows / kJoinRows, item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
    const TileJob j = tile_job(a, item, tiles, rows);
    if (j.b >= a.batch) return;
    const Sequence s = sequence_of(a, j.b);
    const int64_t each = tile_part(rows, J::kDp);
    const float *part = a.part + static_cast<int64_t>(item) * splits * each;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), end = s.computed * a.group - j.row0;
    for (int row = chunk * kJoinRows + wave; row < (chunk + 1) * kJoinRows && row < end; row += kAttnWaves) {
        typename J::Vec v;
        float total;
        J::run(nullptr, part + row * J::kDp, each, part + rows * J::kDp + 2 * row, each, splits, 0, &v, &total);
        J::store(a, s, j.kvh, j.row0 + row, v, total);
    }
}

}  // namespace nvfp4attn

#endif  // NVFP4_ATTN_KERNELS_H
