// Device code of the feed-forward operators (the linear layer and the
// mixture-of-experts layer on NVFP4 weights); nvfp4_ffn.hip, the only
// includer, describes the design and holds the host side.
#ifndef NVFP4_FFN_KERNELS_H
#define NVFP4_FFN_KERNELS_H

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstddef>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "device_common.h"
#include "ffn_plan.h"

namespace {

using namespace nvfp4dev;
using namespace nvfp4ffnplan;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What a kernel of products does with its accumulators and where its tokens
// come from.
enum Mode {
    kLinear = 0,    // tokens in order; epilogue to Y
    kMoeUp = 1,     // the tokens of an expert; f(gate) * up to h
    kMoeDown = 2,   // the slots of an expert; alpha2 * sum to the slot's partial output
    kSlotUp = 3,    // one slot; as kMoeUp
    kSlotDown = 4,  // one slot; the sums stay with the caller
};

struct FfnArgs {
    const uint8_t *X;           // 16-bit rows, ldx elements apart (kMoeDown: h)
    int64_t ldx;
    int64_t plane;              // kMoeDown: elements between the planes of h
    const uint8_t *W, *sW;
    const float *alpha;         // per matrix, or NULL
    const float *bias;          // kLinear, or NULL
    const void *residual;       // kLinear, or NULL
    int64_t ldr;
    void *Y;                    // kLinear: Y; kMoeUp: h; kMoeDown: partial outputs
    int64_t ldy;
    const int32_t *offsets;     // MoE: first slot of every expert
    const int32_t *list;        // MoE: slots sorted by expert
    const int32_t *active;      // MoE: experts that have slots, then -1
    int64_t n, m, k;            // tokens, rows of one matrix, K
    int32_t topk;
    int32_t act;
    int32_t y_type;
    int32_t y_planes;           // kMoeUp: planes of h to write
    float *part;                // kLinear with K split: [split][n][matrices][m] sums, or NULL
    int32_t splits;             // workgroups along K
    int32_t passes;             // MoE: workgroups along an expert's slots
};

// ---------------------------------------------------------------- arithmetic
// exp(x) and 1 / x by the hardware's instructions (one unit in the last place
// each; exp errs by |x| 2^-24 more, which every use below multiplies by a result
// that falls with |x|).
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(1.44269504f * x); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution function: with a = |z| / sqrt 2 its smaller side is
// erfc(a) / 2 = exp(-z^2 / 2) (exp(a^2) erfc(a)) / 2, and exp(a^2) erfc(a) is a
// polynomial of degree 9 in t = 1 / (1 + 0.4 a) without a constant term, a weighted
// least-squares fit, reweighted until the error is level: to 3.2e-8 of itself up to
// a = 4, 1e-7 up to 6 and 1.2e-5 up to 9.5, where exp(-a^2) is 1e-39.  With the fp32
// operations around it GELU is off by at most 4.1e-7 of itself for bf16 z from -4 on
// and 1.6e-6 from -8 on, most of it from the exponential.
__device__ __forceinline__ float normal_cdf(float z) {
    const float t = fast_rcp(__builtin_fmaf(0.4f * 0.70710678f, __builtin_fabsf(z), 1.0f));
    constexpr float c[9] = {0.22539076f, 0.23008046f, 0.17877823f, 0.27498057f, -0.09545095f,
                            0.32257387f, -0.10755151f, -0.05302797f, 0.02422655f};
    float p = c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = __builtin_fmaf(p, t, c[i]);
    const float tail = 0.5f * p * t * fast_exp(-0.5f * z * z);
    return z < 0.0f ? tail : 1.0f - tail;
}

// f of nvfp4_ffn.h in fp32.
__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
    case NVFP4_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case NVFP4_ACT_GELU: return z * normal_cdf(z);
    case NVFP4_ACT_GELU_TANH: {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        const float u = 0.79788456f * (z + 0.044715f * z * z * z);
        return z * fast_rcp(1.0f + fast_exp(-2.0f * u));
    }
    case NVFP4_ACT_SILU: return z * fast_rcp(1.0f + fast_exp(-z));
    default: return z;
    }
}

__device__ __forceinline__ void activate8(int act, float (&z)[8]) {
    auto all = [&](auto kind) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = activate(decltype(kind)::value, z[e]);
    };
    switch (act) {
    case NVFP4_ACT_RELU: return all(std::integral_constant<int, NVFP4_ACT_RELU>{});
    case NVFP4_ACT_GELU: return all(std::integral_constant<int, NVFP4_ACT_GELU>{});
    case NVFP4_ACT_GELU_TANH: return all(std::integral_constant<int, NVFP4_ACT_GELU_TANH>{});
    case NVFP4_ACT_SILU: return all(std::integral_constant<int, NVFP4_ACT_SILU>{});
    default: return;
    }
}

__device__ __forceinline__ float bf16_value(uint16_t b) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16);
}

__device__ __forceinline__ float load_as_float(const void *p, int64_t i, int type) {
    if (type == NVFP4_OUT_F32) return static_cast<const float *>(p)[i];
    const uint16_t b = static_cast<const uint16_t *>(p)[i];
    return type == NVFP4_OUT_BF16 ? bf16_value(b) : static_cast<float>(__builtin_bit_cast(_Float16, b));
}

__device__ __forceinline__ uint16_t round16(float v, bool bf16) {
    return bf16 ? bf16_rne(v) : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

__device__ __forceinline__ void store_rounded(void *p, int64_t i, int type, float v) {
    if (type == NVFP4_OUT_F32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = round16(v, type == NVFP4_OUT_BF16);
}

// The i-th bf16 plane of v: the planes of a value are its rounding to bf16,
// the rounding of what that leaves, and so on; two hold 16 significant bits,
// three hold an fp32 value whole.  Infinities and NaN have no rest.
__device__ __forceinline__ void split_planes(float v, int planes, uint16_t (&o)[kMaxPlanes]) {
#pragma unroll
    for (int i = 0; i < kMaxPlanes; ++i) {
        o[i] = i < planes ? bf16_rne(v) : uint16_t(0);
        const float hi = bf16_value(o[i]);
        v = (o[i] & 0x7F80u) == 0x7F80u ? 0.0f : v - hi;
    }
}

// ---------------------------------------------------------------- decode
// 8 codes (4 bytes) times their block scale as a matrix-core operand, exact.
// fp16: packed multiplies.  bf16: gfx950 has no packed bf16 multiply, so the
// products are formed in fp32, where they are exact with the low 16 bits
// zero, and their upper halves are taken.
__device__ __forceinline__ f16x8 decode8(uint32_t q, f16x2 s) {
    const f16x2 a = e2m1x2_f16<0>(q) * s, b = e2m1x2_f16<1>(q) * s, c = e2m1x2_f16<2>(q) * s,
                d = e2m1x2_f16<3>(q) * s;
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
template <int SEL>
__device__ __forceinline__ uint32_t decode2_bf16(uint32_t q, float s) {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, SEL);
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, v.y * s),
                                 __builtin_bit_cast(uint32_t, v.x * s), 0x07060302u);
}
__device__ __forceinline__ u32x4 decode8(uint32_t q, float s) {
    return u32x4{decode2_bf16<0>(q, s), decode2_bf16<1>(q, s), decode2_bf16<2>(q, s),
                 decode2_bf16<3>(q, s)};
}

// acc += w (rows) x (tokens) over 32 elements of K, 8 per lane.
template <bool BF16>
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 acc) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                       __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w),
                                                      __builtin_bit_cast(f16x8, x), acc, 0, 0, 0);
}

// ---------------------------------------------------------------- tokens
struct TokenRange {
    int32_t first, end;   // positions in the token order (kLinear) or in the slot list
};

template <int MODE>
__device__ __forceinline__ TokenRange expert_range(const FfnArgs &a, int expert) {
    if (MODE == kLinear) return {0, static_cast<int32_t>(a.n)};
    return {a.offsets[expert], a.offsets[expert + 1]};
}

// Output row (kLinear: token, else slot) and X row of position p.
template <int MODE>
__device__ __forceinline__ int32_t out_row(const FfnArgs &a, int32_t p) {
    return MODE == kMoeUp || MODE == kMoeDown ? a.list[p] : p;
}
template <int MODE>
__device__ __forceinline__ int32_t x_row(const FfnArgs &a, int32_t row) {
    return MODE == kMoeUp || MODE == kSlotUp ? row / a.topk : row;
}

// ---------------------------------------------------------------- epilogue
// Rows r .. r+3 of the matrix (those below m) of one token or slot, from the
// fp32 sums of the gate (or only) matrix and of the up matrix.  The matrices of
// the MoE layer have a multiple of 16 rows.
template <int MODE, int G>
__device__ __forceinline__ void finish4(const FfnArgs &a, int expert, int split, int64_t row, int64_t r,
                                        const f32x4 (&sum)[G]) {
    if (MODE == kMoeDown) {
        if (r < a.m)
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.Y) + row * a.ldy + r) =
                (a.alpha ? a.alpha[expert] : 1.0f) * sum[0];
        return;
    }
    if (MODE == kMoeUp || MODE == kSlotUp) {
        if (r >= a.m) return;
        const float al = a.alpha ? a.alpha[2 * expert] : 1.0f, au = a.alpha ? a.alpha[2 * expert + 1] : 1.0f;
        uint16_t p[4][kMaxPlanes];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            split_planes(activate(a.act, al * sum[0][e]) * (au * sum[G - 1][e]), a.y_planes, p[e]);
#pragma unroll
        for (int i = 0; i < kMaxPlanes; ++i)
            if (i < a.y_planes) {
                const uint64_t v = p[0][i] | uint64_t(p[1][i]) << 16 | uint64_t(p[2][i]) << 32 | uint64_t(p[3][i]) << 48;
                *reinterpret_cast<uint64_t *>(static_cast<uint16_t *>(a.Y) + i * a.plane + row * a.ldy + r) = v;
            }
        return;
    }
    if (a.part) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < a.m) a.part[((split * a.n + row) * G + g) * a.m + r + e] = sum[g][e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (r + e >= a.m) return;
        float z = (a.alpha ? a.alpha[0] : 1.0f) * sum[0][e];
        if (a.bias) z += a.bias[r + e];
        z = activate(a.act, z);
        if constexpr (G == 2) {
            float u = (a.alpha ? a.alpha[1] : 1.0f) * sum[1][e];
            if (a.bias) u += a.bias[a.m + r + e];
            z *= u;
        }
        if (a.residual) z += load_as_float(a.residual, row * a.ldr + r + e, a.y_type);
        store_rounded(a.Y, row * a.ldy + r + e, a.y_type, z);
    }
}

// ---------------------------------------------------------------- simple kernel
constexpr int kSimpleWaves = 4;

// Byte offsets of the codes and of the scale of elements e .. e+7 of a row
// (e a multiple of 8) in either layout; `row` counts over all matrices before
// it in row-major order, and the packed layout starts every matrix on a tile.
template <bool PACKED>
__device__ __forceinline__ void weight_at(int64_t matrix, int64_t row, int64_t m, int64_t k, int64_t e,
                                          int64_t *code, int64_t *scale) {
    if (PACKED) {
        const int64_t wins = (k + kWinElems - 1) / kWinElems, tiles = (m + kTile - 1) / kTile;
        const int64_t b = (matrix * tiles + row / kTile) * wins + e / kWinElems;
        const int64_t lane = row % kTile + 16 * ((e % kWinElems) / 64);
        *code = 2048 * b + 1024 * ((e % 64) / 32) + 16 * lane + (e % 32) / 2;
        *scale = 256 * b + 4 * lane + (e % 64) / 16;
    } else {
        *code = (matrix * m + row) * (k / 2) + e / 2;
        *scale = (matrix * m + row) * (k / 16) + e / 16;
    }
}

// One workgroup owns 16 rows of a matrix (G = 2: of a gate and an up matrix)
// and, in turn, every 16 tokens of its range (kLinear: 16 tokens alone).
// Its waves take interleaved steps of 32 elements of K; their sums are added
// in wave order through LDS.  Every load is made for its own 8 elements with
// no assumption on alignment beyond the elements', so this kernel takes every
// valid call.
template <bool BF16, bool PACKED, int G, int P, int MODE>
__global__ void __launch_bounds__(kSimpleWaves * kWave) ffn_simple(const FfnArgs a) {
    __shared__ f32x4 red[(kSimpleWaves - 1) * G * kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int li = lane & 15, kq = lane >> 4;
    const uint32_t tiles = static_cast<uint32_t>((a.m + kTile - 1) / kTile);
    const uint32_t group = blockIdx.x / tiles;   // place in the list of experts, or 16 tokens of the linear layer
    const int64_t row0 = int64_t(blockIdx.x - group * tiles) * kTile;
    const int expert = MODE == kLinear ? 0 : a.active[group];
    if (expert < 0) return;   // workgroup-uniform
    TokenRange range = expert_range<MODE>(a, expert);
    if (MODE == kLinear) {
        range.first = group * kTile;
        if (range.end > range.first + kTile) range.end = range.first + kTile;
    }
    const bool row_in = row0 + li < a.m;
    for (int32_t p0 = range.first; p0 < range.end; p0 += kTile) {
        const bool tok_in = p0 + li < range.end;
        const int32_t orow = tok_in ? out_row<MODE>(a, p0 + li) : 0;
        const uint8_t *x = a.X + 2 * (x_row<MODE>(a, orow) * a.ldx);
        f32x4 acc[G] = {};
        for (int64_t e0 = 32 * wave; e0 < a.k; e0 += 32 * kSimpleWaves) {
            const int64_t e = e0 + 8 * kq;
            u32x4 xv[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                xv[p] = u32x4{0, 0, 0, 0};
                if (tok_in && e < a.k) __builtin_memcpy(&xv[p], x + 2 * (p * a.plane + e), 16);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t q = 0, s = 0;
                if (row_in && e < a.k) {
                    int64_t co, so;
                    weight_at<PACKED>(G * int64_t(expert) + g, row0 + li, a.m, a.k, e, &co, &so);
                    __builtin_memcpy(&q, a.W + co, 4);
                    s = a.sW[so];
                }
                u32x4 w;
                if constexpr (BF16) {
                    w = decode8(q, e4m3x2_f32(s).x);
                } else {
                    const f16x2 sv = e4m3x2_f16(s);
                    w = __builtin_bit_cast(u32x4, decode8(q, f16x2{sv.x, sv.x}));
                }
#pragma unroll
                for (int p = 0; p < P; ++p) acc[g] = mfma<BF16>(w, xv[p], acc[g]);
            }
        }
        if (wave > 0)
#pragma unroll
            for (int g = 0; g < G; ++g) red[((wave - 1) * G + g) * kWave + lane] = acc[g];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                for (int w = 1; w < kSimpleWaves; ++w) acc[g] += red[((w - 1) * G + g) * kWave + lane];
            if (tok_in) finish4<MODE, G>(a, expert, 0, orow, row0 + 4 * kq, acc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- stream kernel
// 32 codes (16 bytes) and the two scale bytes 2 H, 2 H + 1 of s -> the four
// operands of elements 0-7, 8-15 (first scale) and 16-23, 24-31 (second).
template <bool BF16, int H>
__device__ __forceinline__ void decode32(u32x4 q, uint32_t s, u32x4 (&o)[4]) {
    if constexpr (BF16) {
        const f32x2 v = e4m3x2_f32(s >> (16 * H));
        o[0] = decode8(q.x, v.x);
        o[1] = decode8(q.y, v.x);
        o[2] = decode8(q.z, v.y);
        o[3] = decode8(q.w, v.y);
    } else {
        const f16x2 v = e4m3x2_f16(s >> (16 * H));
        const f16x2 a = {v.x, v.x}, b = {v.y, v.y};
        o[0] = __builtin_bit_cast(u32x4, decode8(q.x, a));
        o[1] = __builtin_bit_cast(u32x4, decode8(q.y, a));
        o[2] = __builtin_bit_cast(u32x4, decode8(q.z, b));
        o[3] = __builtin_bit_cast(u32x4, decode8(q.w, b));
    }
}

// Weight layouts of the fast kernels.
enum Layout {
    kRows = 0,          // row-major, k a multiple of 64, codes on 16 bytes and scales on 4
    kPackedTiles = 1,   // nvfp4_mma_pack_weight's
    kRows16 = 2,        // row-major, any k and scales, codes on 4 bytes
};

// The four scales of a lane's 64 elements, as loaded: put together only when they
// are used, since before that the loads would have to be waited for.
template <int L>
struct ScaleWord {
    uint32_t part[L == kRows16 ? 4 : 1];
    __device__ __forceinline__ uint32_t value() const {
        if constexpr (L == kRows16) return part[0] | part[1] << 8 | part[2] << 16 | part[3] << 24;
        else return part[0];
    }
};

constexpr int kWinCodeBytes = 2048, kWinScaleBytes = 256;   // of a packed window of a tile
// Descriptor range where every used offset is known to be valid: kReach as the
// descriptor's unsigned 32 bits, so that kOutOfRange is the first offset past it.
constexpr int kAnyRange = static_cast<int>(static_cast<uint32_t>(kReach));
static_assert(kReach == int64_t(kOutOfRange), "offsets from kOutOfRange on read zeros");

// The weights of one matrix as a workgroup reads them: R tiles of 16 rows from
// row0, window by window (256 elements of K).  Lane i + 16 q holds, of row i of
// each tile, the 64 elements from 64 q on, in two halves, and their four scales.
// Rows past m and elements past k read zeros without touching memory; `left` is
// the number of elements from the window on that exist.  L = kRows16: k is any
// multiple of 16 and the scales have any alignment, so the codes come in loads of
// a block each and the scales byte by byte.
template <int L, int R>
struct WeightTiles {
    __amdgpu_buffer_rsrc_t wdesc, sdesc;
    uint32_t code[R], scale[R];   // the lane's offsets at window 0 (or out of range)
    int first;                    // the lane's first element of a window

    __device__ __forceinline__ WeightTiles(const FfnArgs &a, int64_t matrix, int64_t row0, int li, int kq)
        : first(64 * kq) {
        if (L == kPackedTiles) {
            const int64_t wins = (a.k + kWinElems - 1) / kWinElems, tiles = (a.m + kTile - 1) / kTile;
            const int64_t t0 = matrix * tiles + row0 / kTile;
            wdesc = buffer_of(a.W + t0 * wins * kWinCodeBytes, kAnyRange);
            sdesc = buffer_of(a.sW + t0 * wins * kWinScaleBytes, kAnyRange);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool in = row0 + r * kTile < a.m;
                const uint32_t w = static_cast<uint32_t>(r * wins), lane = li + 16 * kq;
                code[r] = in ? w * kWinCodeBytes + 16 * lane : kOutOfRange;
                scale[r] = in ? w * kWinScaleBytes + 4 * lane : kOutOfRange;
            }
        } else {
            wdesc = buffer_of(a.W + (matrix * a.m + row0) * (a.k / 2), kAnyRange);
            sdesc = buffer_of(a.sW + (matrix * a.m + row0) * (a.k / 16), kAnyRange);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool in = row0 + r * kTile + li < a.m;
                const uint32_t row = r * kTile + li;
                code[r] = in ? row * static_cast<uint32_t>(a.k / 2) + 32 * kq : kOutOfRange;
                scale[r] = in ? row * static_cast<uint32_t>(a.k / 16) + 4 * kq : kOutOfRange;
            }
        }
    }
    __device__ __forceinline__ uint32_t past(int left, int block) const {
        return first + 16 * block < left ? 0u : kOutOfRange;
    }
    // POLICY: kNonTemporal for weights that a workgroup reads once.
    template <int POLICY>
    __device__ __forceinline__ void load_half(int r, uint32_t window, int left, int h, u32x4 &q) const {
        if constexpr (L == kRows16) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(
                    wdesc, (code[r] + 16 * h + 8 * b) | past(left, 2 * h + b), window * 128, 0);
                q[2 * b] = v[0];
                q[2 * b + 1] = v[1];
            }
        } else {
            q = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                              wdesc, (code[r] | past(left, 0)) + h * (L == kPackedTiles ? 1024 : 16),
                                              window * (L == kPackedTiles ? kWinCodeBytes : 128), POLICY));
        }
    }
    template <int POLICY>
    __device__ __forceinline__ void load_scale(int r, uint32_t window, int left, ScaleWord<L> &s) const {
        if constexpr (L == kRows16) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                s.part[b] = __builtin_amdgcn_raw_buffer_load_b8(sdesc, (scale[r] + b) | past(left, b), window * 16, 0);
        } else {
            s.part[0] = __builtin_amdgcn_raw_buffer_load_b32(sdesc, scale[r] | past(left, 0),
                                                             window * (L == kPackedTiles ? kWinScaleBytes : 16), POLICY);
        }
    }
    // For the stream kernels: non-temporal also where another block of tokens, pass or
    // slot reads the same weights again.
    __device__ __forceinline__ void load(int r, uint32_t window, int left, u32x4 (&q)[2], ScaleWord<L> &s) const {
        load_half<kNonTemporal>(r, window, left, 0, q[0]);
        load_half<kNonTemporal>(r, window, left, 1, q[1]);
        load_scale<L == kPackedTiles ? kNonTemporal : 0>(r, window, left, s);
    }
};

// Orders a wave's own LDS writes before its later reads (and the reverse)
// for the compiler; the hardware runs one wave's LDS operations in order.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The sums of R tiles of 16 rows of each of G matrices for up to 2 NX tokens: a
// wave takes every `waves`-th window of 256 elements of K of its part of K from
// window `wave` on, U in flight.  This is the shape for few tokens, where the
// weights' bytes are the bound: every weight byte is read in 1 KiB instructions
// (packed) and decoded, once for up to 2 NX tokens; more tokens (blocks of the
// linear layer, passes over an expert's slots) read and decode it again.
//
// The tokens' elements of a window (512 bytes each) are read row by row, two
// tokens per instruction, as far ahead as the weights, and go through a slot
// of LDS that belongs to the wave, from where every lane reads its eight
// 16-byte operand pieces: read straight from memory in operand order, each
// instruction would touch a different line in every lane.  The 16-byte pieces
// are swizzled by the token, so the 16 lanes that read the same piece of 16
// tokens hit distinct banks.  NX = instructions = half the tokens staged.  The
// tokens' rows need no alignment beyond their elements'.
template <bool BF16, int L, int G, int P, int MODE, int R, int U, int NX>
__device__ __forceinline__ void stream_sums(const FfnArgs &a, int expert, int64_t row0, int split, int32_t p0,
                                            int32_t end, u32x4 *slot, int wave, int waves, f32x4 (&acc)[G][R]) {
    const int lane = threadIdx.x & (kWave - 1);
    const int li = lane & 15, kq = lane >> 4;
    const uint32_t k = static_cast<uint32_t>(a.k);
    const int wins = static_cast<int>((k + kWinElems - 1) / kWinElems);
    const int win0 = static_cast<int>(int64_t(split) * wins / a.splits);
    const int nwin = static_cast<int>(int64_t(split + 1) * wins / a.splits) - win0;
    const int niter = nwin > wave ? (nwin - wave + waves - 1) / waves : 0;

    const WeightTiles<L, R> w0(a, G * int64_t(expert), row0, li, kq);
    const WeightTiles<L, R> w1(a, G * int64_t(expert) + (G - 1), row0, li, kq);

    // X: kLinear from token p0 on, else from row 0 (the host keeps rows * ldx in 31 bits)
    const uint8_t *xbase = a.X + (MODE == kLinear ? 2 * (int64_t(p0) * a.ldx) : 0);
    __amdgpu_buffer_rsrc_t xdesc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) xdesc[p] = buffer_of(xbase + 2 * p * a.plane, kAnyRange);
    uint32_t xo[NX];
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const int32_t t = p0 + 2 * j + (lane >> 5);
        xo[j] = kOutOfRange;
        if (t < end) {
            const int32_t row = MODE == kLinear ? t - p0 : x_row<MODE>(a, out_row<MODE>(a, t));
            xo[j] = 2 * static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ldx) + 16 * (lane & 31);
        }
    }
    const int tok = li & (2 * NX - 1);   // columns past the staged tokens repeat them and are dropped

    u32x4 wq[U][G][R][2], xq[U][P][NX];
    ScaleWord<L> ws[U][G][R];
    auto issue = [&](int i, int u) {
        const uint32_t win = static_cast<uint32_t>(win0 + wave + waves * i);
        const bool run = i < niter;
        const uint32_t xpast = run && win * kWinElems + 8 * (lane & 31) < k ? 0u : kOutOfRange;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < NX; ++j)
                xq[u][p][j] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(xdesc[p], (xo[j] + win * 512) | xpast, 0, 0));
        const int left = run ? static_cast<int>(k - win * kWinElems) : 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w0.load(r, win, left, wq[u][0][r], ws[u][0][r]);
            if constexpr (G == 2) w1.load(r, win, left, wq[u][1][r], ws[u][1][r]);
        }
    };
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[g][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto consume = [&](int u) {
        wave_lds_fence();
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const int t = 2 * j + (lane >> 5);
                slot[(p * 2 * NX + t) * 32 + ((lane & 31) ^ (t & 15))] = xq[u][p][j];
            }
        wave_lds_fence();
        auto half = [&](auto hc) {
            constexpr int h = decltype(hc)::value;
            u32x4 xv[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int c = 0; c < 4; ++c) xv[p][c] = slot[(p * 2 * NX + tok) * 32 + ((8 * kq + 4 * h + c) ^ tok)];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    u32x4 wo[4];
                    decode32<BF16, h>(wq[u][g][r][h], ws[u][g][r].value(), wo);
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[g][r] = mfma<BF16>(wo[c], xv[p][c], acc[g][r]);
                }
        };
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
    };

    phase_fence();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        issue(u, u);
        phase_fence();
    }
    // the last windows apart, so that no loads are issued that are not used: even
    // those out of range, which cause no traffic, take their time
    int i = 0;
    for (; i + U < niter; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            consume(u);
            issue(i + u + U, u);   // past the wave's windows: zeros
            phase_fence();
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i + u < niter) consume(u);   // wave-uniform
}

// The same sums for one token, in VALU dot products.  On the matrix cores 15 of 16
// columns would be dropped, and a weight costs the VALU, which bounds the stream,
// more there: bf16 elements take 32 operations per 16 to be decoded with their
// scale; here 8 conversions, 8 dot products of two elements and one multiply-add
// with the block's scale (7168 x 16384, bf16: 16.0 -> 14.4 us).  Lane i + 16 q ends
// with the sum of row i of every tile, the same for all q.  The token's elements
// of a window go through the wave's LDS slot, every lane quarter's 128 bytes 16
// bytes further, so that the quarters' reads hit distinct banks.
constexpr int kDotSlot = 4 * (8 + 1);   // 16-byte pieces of a window
// A block is summed before its scale is known to make its products smaller: 16
// products of a bf16 value and a code reach 96 times the largest fp32 value, so
// the codes are converted to 2^-7 times their value and the scales to 2^7 times
// theirs, both exactly and at no cost.  A product of a bf16 value and a code so
// converted is a multiple of 2^-141, and fp32 subnormals are kept by every step, so
// nothing is lost below either.  fp16 values are at most 65504.
constexpr float kDotDown = 0x1p-7f, kDotUp = 0x1p7f;
template <bool BF16>
__device__ __forceinline__ float dot_scale(uint32_t s) {
    if constexpr (BF16) {
        const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(s, kDotUp, false);
        return v.x;
    } else {
        return e4m3x2_f32(s).x;
    }
}

template <bool BF16>
__device__ __forceinline__ float dot8(uint32_t q, u32x4 x, float s) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    if constexpr (BF16) {
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, kDotDown, 0),
                                            __builtin_bit_cast(bf16x2, uint32_t(x.x)), s, false);
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, kDotDown, 1),
                                            __builtin_bit_cast(bf16x2, uint32_t(x.y)), s, false);
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, kDotDown, 2),
                                            __builtin_bit_cast(bf16x2, uint32_t(x.z)), s, false);
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, kDotDown, 3),
                                               __builtin_bit_cast(bf16x2, uint32_t(x.w)), s, false);
    } else {
        s = __builtin_amdgcn_fdot2(e2m1x2_f16<0>(q), halves(x.x), s, false);
        s = __builtin_amdgcn_fdot2(e2m1x2_f16<1>(q), halves(x.y), s, false);
        s = __builtin_amdgcn_fdot2(e2m1x2_f16<2>(q), halves(x.z), s, false);
        return __builtin_amdgcn_fdot2(e2m1x2_f16<3>(q), halves(x.w), s, false);
    }
}

template <bool BF16, int L, int G, int R, int U>
__device__ __forceinline__ void dot_sums(const FfnArgs &a, int64_t row0, int split, int32_t token, u32x4 *slot, int wave,
                                         int waves, float (&acc)[G][R]) {
    const int lane = threadIdx.x & (kWave - 1);
    const int li = lane & 15, kq = lane >> 4;
    const uint32_t k = static_cast<uint32_t>(a.k);
    const int wins = static_cast<int>((k + kWinElems - 1) / kWinElems);
    const int win0 = static_cast<int>(int64_t(split) * wins / a.splits);
    const int nwin = static_cast<int>(int64_t(split + 1) * wins / a.splits) - win0;
    const int niter = nwin > wave ? (nwin - wave + waves - 1) / waves : 0;

    const WeightTiles<L, R> w0(a, 0, row0, li, kq);
    const WeightTiles<L, R> w1(a, G - 1, row0, li, kq);
    const __amdgpu_buffer_rsrc_t xdesc = buffer_of(a.X + 2 * (token * a.ldx), kAnyRange);

    u32x4 wq[U][G][R][2], xq[U];
    ScaleWord<L> ws[U][G][R];
    auto issue = [&](int i, int u) {
        const uint32_t win = static_cast<uint32_t>(win0 + wave + waves * i);
        const int left = i < niter ? static_cast<int>(k - win * kWinElems) : 0;
        const uint32_t xo = lane < 32 && 8 * lane < left ? 16 * lane : kOutOfRange;
        xq[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xdesc, xo, win * 512, 0));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w0.load(r, win, left, wq[u][0][r], ws[u][0][r]);
            if constexpr (G == 2) w1.load(r, win, left, wq[u][1][r], ws[u][1][r]);
        }
    };
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[g][r] = 0.0f;
    auto consume = [&](int u) {
        wave_lds_fence();
        if (lane < 32) slot[lane + (lane >> 3)] = xq[u];
        wave_lds_fence();
#pragma unroll
        for (int b = 0; b < 4; ++b) {   // blocks of 16 elements
            u32x4 xv[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) xv[c] = slot[9 * kq + 2 * b + c];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float s = 0.0f;
#pragma unroll
                    for (int c = 0; c < 2; ++c) s = dot8<BF16>(wq[u][g][r][b / 2][2 * (b & 1) + c], xv[c], s);
                    acc[g][r] = __builtin_fmaf(dot_scale<BF16>(ws[u][g][r].value() >> (8 * b)), s, acc[g][r]);
                }
        }
    };

    phase_fence();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        issue(u, u);
        phase_fence();
    }
    int i = 0;
    for (; i + U < niter; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            consume(u);
            issue(i + u + U, u);
            phase_fence();
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i + u < niter) consume(u);   // wave-uniform
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) {   // the four quarters of a row
            acc[g][r] += __shfl_xor(acc[g][r], 16);
            acc[g][r] += __shfl_xor(acc[g][r], 32);
        }
}

// One workgroup owns R tiles of 16 rows of each of G matrices and up to 2 NX
// tokens (NX = 0: one, in dot products); its W waves take the windows of its part
// of K in turn, and their sums are added in wave order through LDS.
template <bool BF16, int L, int G, int P, int MODE, int R, int U, int W, int NX>
__device__ __forceinline__ void stream_pass(const FfnArgs &a, int expert, int64_t row0, int split, int32_t p0,
                                            int32_t end, u32x4 *lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int li = lane & 15, kq = lane >> 4;
    static_assert(W > 1, "the waves' sums go through LDS");
    // the sums of wave w, matrix g and tile r, four rows of a token, for this lane
    const f32x4 *red = reinterpret_cast<const f32x4 *>(lds);
    auto at = [&](int w, int g, int r) {
        return NX == 0 ? ((w * G + g) * R + r) * 4 + kq : ((w * G + g) * R + r) * kWave + lane;
    };
    if constexpr (NX == 0) {
        float sum[G][R];
        static_assert(MODE == kLinear && P == 1, "one token of the linear layer");
        dot_sums<BF16, L, G, R, U>(a, row0, split, p0, lds + wave * kDotSlot, wave, W, sum);
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane < kTile) reinterpret_cast<float *>(lds)[((wave * G + g) * R + r) * kTile + lane] = sum[g][r];
        __syncthreads();
    } else {
        f32x4 acc[G][R];
        stream_sums<BF16, L, G, P, MODE, R, U, NX>(a, expert, row0, split, p0, end, lds + wave * (P * 2 * NX * 32), wave,
                                                   W, acc);
        __syncthreads();
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int r = 0; r < R; ++r) reinterpret_cast<f32x4 *>(lds)[at(wave, g, r)] = acc[g][r];
        __syncthreads();
    }
    // wave r % W finishes row tile r
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r % W != wave) continue;
        f32x4 sum[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            sum[g] = red[at(0, g, r)];
            for (int w = 1; w < W; ++w) sum[g] += red[at(w, g, r)];
        }
        if (p0 + li < end && li < (NX == 0 ? 1 : 2 * NX))
            finish4<MODE, G>(a, expert, split, out_row<MODE>(a, p0 + li), row0 + r * kTile + 4 * kq, sum);
    }
    if (MODE != kLinear) __syncthreads();   // before the next pass writes LDS
}

// LDS of a stream workgroup in 16-byte pieces: the waves' slots, later their sums.
template <int G, int P, int R, int W, int NX>
constexpr int stream_lds() {
    return NX == 0 ? W * (kDotSlot > G * R * 4 ? kDotSlot : G * R * 4)
                   : W * kWave * (P * NX > G * R ? P * NX : G * R);
}

template <bool BF16, int L, int G, int P, int MODE, int R, int U, int W, int NXMAX>
__global__ void __launch_bounds__(W * kWave, 2) ffn_stream(const FfnArgs a) {
    __shared__ u32x4 lds[stream_lds<G, P, R, W, NXMAX>()];
    const uint32_t strips = static_cast<uint32_t>((a.m + R * kTile - 1) / (R * kTile));
    // block of tokens and split, or place in the list of experts and pass
    const uint32_t q = blockIdx.x / strips;
    const int64_t row0 = int64_t(blockIdx.x - q * strips) * (R * kTile);
    if constexpr (MODE == kLinear) {
        constexpr int32_t kTokens = NXMAX == 0 ? 1 : 2 * NXMAX;
        const int32_t block = q / a.splits, p = block * kTokens, left = static_cast<int32_t>(a.n) - p;
        stream_pass<BF16, L, G, P, MODE, R, U, W, NXMAX>(a, 0, row0, q - block * a.splits, p,
                                                         left < kTokens ? p + left : p + kTokens, lds);
    } else {
        const uint32_t place = q / a.passes, pass = q - place * a.passes;
        const int expert = a.active[place];
        if (expert < 0) return;   // workgroup-uniform
        const TokenRange range = expert_range<MODE>(a, expert);
        for (int32_t p = range.first + pass * 2 * NXMAX; p < range.end; p += a.passes * 2 * NXMAX) {
            const int32_t end = range.end - p > 2 * NXMAX ? p + 2 * NXMAX : range.end;
            const int n = end - p;   // workgroup-uniform
            if (n <= 2)
                stream_pass<BF16, L, G, P, MODE, R, U, W, 1>(a, expert, row0, 0, p, end, lds);
            else if (n <= 4)
                stream_pass<BF16, L, G, P, MODE, R, U, W, 2>(a, expert, row0, 0, p, end, lds);
            else if (NXMAX == 4 || n <= 8)
                stream_pass<BF16, L, G, P, MODE, R, U, W, 4>(a, expert, row0, 0, p, end, lds);
            else
                stream_pass<BF16, L, G, P, MODE, R, U, W, NXMAX>(a, expert, row0, 0, p, end, lds);
        }
    }
}

// ---------------------------------------------------------------- tile kernel
// 8 consecutive values of a row of Y's type, aligned to their elements only: 16
// bytes go in one access all the same.
struct Row8 {
    u32x4 v[2];
};
__device__ __forceinline__ Row8 load_row8(const void *p, int64_t i, int type) {
    Row8 o;
    if (type == NVFP4_OUT_F32) {
        __builtin_memcpy(&o, static_cast<const float *>(p) + i, 32);
    } else {
        __builtin_memcpy(&o.v[0], static_cast<const uint16_t *>(p) + i, 16);
        o.v[1] = o.v[0];
    }
    return o;
}
__device__ __forceinline__ void add_row8(const Row8 &o, int type, float (&z)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = o.v[0][e / 2];
        const uint16_t b = static_cast<uint16_t>(w >> (16 * (e & 1)));
        z[e] += type == NVFP4_OUT_F32 ? __builtin_bit_cast(float, uint32_t(o.v[e / 4][e % 4]))
                : type == NVFP4_OUT_BF16 ? bf16_value(b)
                                         : static_cast<float>(__builtin_bit_cast(_Float16, b));
    }
}
__device__ __forceinline__ uint32_t round16x2(float lo, float hi, bool bf16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    if (bf16) return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
    return bits(f16x2{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
}
__device__ __forceinline__ void store_row8(void *p, int64_t i, int type, const float (&z)[8]) {
    if (type == NVFP4_OUT_F32) {
        __builtin_memcpy(static_cast<float *>(p) + i, z, 32);
        return;
    }
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = round16x2(z[2 * e], z[2 * e + 1], type == NVFP4_OUT_BF16);
    __builtin_memcpy(static_cast<uint16_t *>(p) + i, &o, 16);
}

// Orders the workgroup's LDS accesses around the barrier and leaves global
// loads in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

constexpr int kStageElems = 128;    // K elements of one stage: half of every lane's part of a window
constexpr int kXcds = 8;            // dies, each with its own L2; workgroup i runs on die i % 8

template <typename F, int... I>
__device__ __forceinline__ void each_tile(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
typedef __attribute__((address_space(3))) char lds_void_t;
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
template <int G, int Q, int NT, int WM, int WK>
struct TileShape {
    static constexpr int waves = WM * WK;
    static constexpr int rows = kTile * Q * WM;       // of each matrix
    static constexpr int tokens = kTile * NT;
    static constexpr int stage = tokens * kStageElems / 8;             // 16-byte pieces
    static constexpr int stride = kTile * Q * G * 4 + 16;              // bytes of a token in the epilogue
    static constexpr int out_tiles = Q == 1 ? 2 : 1;                   // token tiles a wave's epilogue takes at a time
    static constexpr int wave_out = out_tiles * kTile * stride;        // bytes of them
    static constexpr int out_waves = WM * (WK < NT / out_tiles ? WK : NT / out_tiles);   // waves that have any
};

// More than 16 tokens.  A workgroup owns 16 Q WM rows of each of G matrices and
// 16 NT tokens; WK groups of WM waves take the windows of K in turn and add their
// sums through LDS at the end.  A wave holds the sums of G Q row tiles by NT token
// tiles.
//
// Weights go from memory straight into the registers of the wave that owns their
// rows, in 1 KiB instructions (packed), and are decoded there, once for all NT
// token tiles, between the matrix instructions: 16 (bf16) or 8 (fp16) VALU
// operations per operand, against NT matrix instructions of 16 cycles.  The
// tokens go through LDS, in stages of half a window (128 elements), copied there
// directly while the other of two buffers is multiplied: a token's 16 pieces of
// 16 bytes lie in positions xored with its number, so that the 16 lanes that read
// the same piece of 16 tokens hit distinct banks (lanes that read different pieces
// meet all the same: 4 conflict cycles per LDS instruction are counted).  Two buffers
// are two variables: in one, every read would wait for the copies into the other half.
//
// 4096 tokens x (4096 x 7168) in 256 x 256 tiles: bf16 192-196 us, 1.24 PFLOP/s,
// fp16 192, where a library's bf16 product reaches 1.54; with SiLU, bias and
// residual 206-209 us (up to 230 on other GPUs).  256 x 128 tiles, which decode every
// weight for half as many tokens, take 214 and 203 us, 128 x 128 tiles 274 and 266.
// In 256 x 128 tiles the loop without the loads and the decode, so with matrix
// instructions and LDS reads alone, takes 180 us, without the LDS reads 167: the
// matrix cores do not sustain their nominal rate on such operands; the tokens' copies
// add 20 us, the weights' loads 15 and the decode 12 (fp16) or 25.  Waves of 64
// rows by 128 tokens decode as little, but spill or leave one wave per SIMD.
template <bool BF16, int L, int G, int Q, int NT, int WM, int WK>
__device__ __forceinline__ void tile_product(const FfnArgs &a) {
    using S = TileShape<G, Q, NT, WM, WK>;
    constexpr int RT = G * Q;
    static_assert(S::out_waves * S::wave_out <= 2 * 16 * S::stage * WK && S::out_waves % 2 == 0, "the epilogue fits");
    static_assert(WK == 1 || (S::waves * NT * kWave <= S::stage * WK && RT <= 2), "the groups' sums fit");
    __shared__ u32x4 lds0[WK * S::stage], lds1[WK * S::stage];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int li = lane & 15, kq = lane >> 4;
    const int wm = wave % WM, kg = wave / WM;   // wave of its group, group
    const uint32_t k = static_cast<uint32_t>(a.k);

    // Workgroup -> (split, strip of rows, block of tokens): every die takes a
    // run of consecutive tiles, ordered in bands of four token blocks, so that
    // its L2 serves few different rows and tokens.
    const uint32_t strips = static_cast<uint32_t>((a.m + S::rows - 1) / S::rows);
    const uint32_t blocks = static_cast<uint32_t>((a.n + S::tokens - 1) / S::tokens);
    const uint32_t total = gridDim.x, die = blockIdx.x % kXcds;
    uint32_t id = die * (total / kXcds) + (die < total % kXcds ? die : total % kXcds) + blockIdx.x / kXcds;
    const int split = static_cast<int>(id / (strips * blocks));
    id -= split * strips * blocks;
    const uint32_t band = id / (4 * strips), width = blocks - 4 * band < 4 ? blocks - 4 * band : 4;
    id -= 4 * band * strips;
    const int64_t row0 = int64_t(id / width) * S::rows + kTile * Q * wm;
    const int64_t tok0 = int64_t(4 * band + id % width) * S::tokens;

    const int wins = static_cast<int>((k + kWinElems - 1) / kWinElems);
    const int win0 = static_cast<int>(int64_t(split) * wins / a.splits);
    const int win1 = static_cast<int>(int64_t(split + 1) * wins / a.splits);

    const WeightTiles<L, Q> w0(a, 0, row0, li, kq);
    const WeightTiles<L, Q> w1(a, G - 1, row0, li, kq);

    // staging: copy i of 4 tokens: lane l fills position l % 16 of token t = 4 i + l / 16
    // with piece (l % 16) ^ (t & 15); piece 4 q + c holds elements 64 q + 32 h + 8 c
    // of the window
    constexpr int kCopies = S::tokens / 4 / WM;
    static_assert(S::tokens % (4 * WM) == 0, "whole copies per wave");
    const __amdgpu_buffer_rsrc_t xdesc = buffer_of(a.X + 2 * (tok0 * a.ldx), kAnyRange);
    const int tlast = a.n - tok0 < S::tokens ? static_cast<int>(a.n - tok0) - 1 : S::tokens - 1;
    const int piece = li ^ ((4 * kCopies * wm + kq) & 15);
    uint32_t xo[kCopies];   // rows past the last repeat it and are not stored
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
        const int t = 4 * (kCopies * wm + j) + kq;
        xo[j] = 2 * ((t < tlast ? t : tlast) * static_cast<uint32_t>(a.ldx) +
                     64 * ((piece >> 2) ^ (j & 3)) + 8 * (piece & 3));
    }
    u32x4 wq[2][RT];
    ScaleWord<L> ws[2][RT];
    auto load = [&](auto hc, int win, int slot) {
        constexpr int h = decltype(hc)::value;
        const int left = win < win1 ? static_cast<int>(k - win * kWinElems) : 0;   // elements from this window on
        lds_void_t *to = h == 0 ? (lds_void_t *)lds0 : (lds_void_t *)lds1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const WeightTiles<L, Q> &w = r < Q ? w0 : w1;
            w.template load_half<0>(r % Q, win, left, h, wq[h][r]);
            if (h == 0) w.template load_scale<0>(r % Q, win, left, ws[slot][r]);
        }
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                xdesc, to + 16 * S::stage * kg + 1024 * (kCopies * wm + j), 16,
                xo[j] | (64 * ((piece >> 2) ^ (j & 3)) + (L == kRows16 ? 32 * h + 8 * (piece & 3) : 0) < left ? 0u
                                                                                                       : kOutOfRange),
                2 * (win * kWinElems + 32 * h), 0, 0);
    };
    f32x4 acc[RT][NT] = {};
    u32x4 wo[2][RT];   // operands of this step of 32 elements and of the next
    auto decode = [&](u32x4 q, int c, int h, uint32_t s, u32x4 &o) {
        const uint32_t b = s >> (16 * h + 8 * (c / 2));
        if constexpr (BF16) {
            o = decode8(q[c], e4m3x2_f32(b).x);
        } else {
            const f16x2 v = e4m3x2_f16(b);
            o = __builtin_bit_cast(u32x4, decode8(q[c], f16x2{v.x, v.x}));
        }
        __asm__ volatile("" : "+v"(o));
    };
    // One stage: 4 steps of 32 elements, each in groups of two token tiles.  A
    // group reads the next group's tokens and decodes part of the next step's
    // weights (of the next stage's first one at the end) between its products.
    // The empty asm statements hold each product to its group: the compiler would
    // gather them, and the registers they need, across the whole stage.
    auto compute = [&](auto hc) {
        constexpr int h = decltype(hc)::value;
        constexpr int kPairs = NT / 2;
        u32x4 xv[2][2];
        auto read = [&](int c, int t, u32x4 &to) {
            to = (h == 0 ? lds0 : lds1)[S::stage * kg + 16 * (16 * t + li) + ((4 * kq + c) ^ li)];
        };
        read(0, 0, xv[0][0]);
        read(0, 1, xv[0][1]);
        phase_fence();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int t = 0; t < kPairs; ++t) {
                const int g = (c * kPairs + t) & 1;
                if (t + 1 < kPairs || c + 1 < 4) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        read(t + 1 < kPairs ? c : c + 1, t + 1 < kPairs ? 2 * (t + 1) + i : i, xv[g ^ 1][i]);
                }
#pragma unroll
                for (int r = RT * t / kPairs; r < RT * (t + 1) / kPairs; ++r) {
                    if (c < 3) decode(wq[h][r], c + 1, h, ws[0][r].value(), wo[(c + 1) & 1][r]);
                    else decode(wq[1 - h][r], 0, 1 - h, ws[h][r].value(), wo[0][r]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        acc[r][2 * t + i] = mfma<BF16>(wo[c & 1][r], xv[g][i], acc[r][2 * t + i]);
                // issue order: the reads, then VALU operations between the products
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
                for (int i = 0; i < 2 * RT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, BF16 ? 4 : 2, 0);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < RT; ++r) __asm__ volatile("" : "+v"(acc[r][2 * t + i]));
                phase_fence();
            }
        }
    };
    constexpr auto h0 = std::integral_constant<int, 0>{};
    constexpr auto h1 = std::integral_constant<int, 1>{};
    // the groups of waves take the windows in turn; all make the same number of
    // rounds, past the last window on zeros
    load(h0, win0 + kg, 0);
    wait_vmcnt<0>();
#pragma unroll
    for (int r = 0; r < RT; ++r) decode(wq[0][r], 0, 0, ws[0][r].value(), wo[0][r]);
    lds_barrier();
    for (int win = win0 + kg; win < win1 + kg; win += WK) {
        load(h1, win, 0);
        phase_fence();
        compute(h0);
        wait_vmcnt<0>();
        lds_barrier();
        load(h0, win + WK, 1);
        phase_fence();
        compute(h1);
        wait_vmcnt<0>();
#pragma unroll
        for (int r = 0; r < RT; ++r) ws[0][r] = ws[1][r];
        lds_barrier();
    }
    if (WK > 1) {
        // each group's sums to LDS; then every group adds those of its token tiles
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                reinterpret_cast<f32x4 *>(r == 0 ? lds0 : lds1)[(wave * NT + t) * kWave + lane] = acc[r][t];
        lds_barrier();
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t / S::out_tiles % WK != kg) continue;
                const f32x4 *from = reinterpret_cast<const f32x4 *>(r == 0 ? lds0 : lds1) + (wm * NT + t) * kWave + lane;
                f32x4 sum = from[0];
#pragma unroll
                for (int i = 1; i < WK; ++i) sum += from[i * WM * NT * kWave];
                acc[r][t] = sum;
            }
        lds_barrier();
    }

    // Epilogue.  The sums go through LDS, which turns them into rows of 8
    // consecutive outputs of one token: each wave has its own part and takes
    // out_tiles token tiles at a time, with the residual of the next already on
    // its way.
    uint8_t *out = reinterpret_cast<uint8_t *>(2 * wave < S::out_waves ? lds0 : lds1) + wave % (S::out_waves / 2) * S::wave_out;
    constexpr int kGroups = 2 * Q;                       // groups of 8 rows of a matrix
    constexpr int kStep = kWave / kGroups;               // tokens per iteration
    constexpr int kIters = S::out_tiles * kTile / kStep;
    const int64_t r = row0 + 8 * (lane % kGroups);
    const int64_t first = tok0 + lane / kGroups;   // the lane's first token
    const int rows = a.m - r < 8 ? static_cast<int>(a.m - r) : 8;    // of the lane's 8, those that exist
    const bool whole = rows == 8;
    const float al = a.alpha ? a.alpha[0] : 1.0f, au = G == 2 && a.alpha ? a.alpha[1] : 1.0f;
    float b[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) b[g][e] = a.bias && e < rows ? a.bias[g * a.m + r + e] : 0.0f;
    Row8 res[2][kIters];
    auto fetch = [&](int t, Row8 (&to)[kIters]) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int64_t row = first + kTile * t + kStep * i;
            if (a.residual && whole && t < NT && row < a.n) to[i] = load_row8(a.residual, row * a.ldr + r, a.y_type);
        }
    };
    if (!a.part) fetch(S::out_tiles * kg, res[0]);
#pragma unroll 1
    for (int t = S::out_tiles * kg; t < NT; t += S::out_tiles * WK) {
        wave_lds_fence();
        // the sums are picked by constant indices: any other would put them in memory
        each_tile([&](auto tc) {
            constexpr int T = decltype(tc)::value;
            if (t != T - T % S::out_tiles) return;
#pragma unroll
            for (int q = 0; q < RT; ++q)
                *reinterpret_cast<f32x4 *>(out + (T % S::out_tiles * kTile + li) * S::stride +
                                           4 * (kTile * q + 4 * kq)) = acc[q][T];
        }, std::make_integer_sequence<int, NT>{});
        wave_lds_fence();
        if (!a.part) fetch(t + S::out_tiles * WK, res[1]);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int64_t row = first + kTile * t + kStep * i;
            if (row >= a.n || rows <= 0) continue;
            float z[8], u[8];
            const uint8_t *from = out + (lane / kGroups + kStep * i) * S::stride + 32 * (lane % kGroups);
            __builtin_memcpy(z, from, 32);
            if (G == 2) __builtin_memcpy(u, from + 4 * kTile * Q, 32);
            if (a.part) {
                float *to = a.part + ((split * a.n + row) * G) * a.m + r;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float(&v)[8] = g == 0 ? z : u;
                    if (whole) {
                        store_row8(to, g * a.m, NVFP4_OUT_F32, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < rows) to[g * a.m + e] = v[e];
                    }
                }
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = z[e] * al + b[0][e];
            activate8(a.act, z);
            if constexpr (G == 2)
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] *= u[e] * au + b[1][e];
            if (whole) {
                if (a.residual) add_row8(res[0][i], a.y_type, z);
                store_row8(a.Y, row * a.ldy + r, a.y_type, z);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < rows) {
                    if (a.residual) z[e] += load_as_float(a.residual, row * a.ldr + r + e, a.y_type);
                    store_rounded(a.Y, row * a.ldy + r + e, a.y_type, z[e]);
                }
        }
#pragma unroll
        for (int i = 0; i < kIters; ++i) res[0][i] = res[1][i];
    }
}

template <bool BF16, int L, int G, int Q, int NT, int WM, int WK>
__global__ void __launch_bounds__(WM *WK *kWave, 2) ffn_tile(const FfnArgs a) {
    tile_product<BF16, L, G, Q, NT, WM, WK>(a);
}

// ---------------------------------------------------------------- split sums
constexpr int kFinishThreads = 256;

// The epilogue of a linear layer whose K was split across workgroups: the
// splits' sums in split order.  One thread per four rows of one token.
template <int G>
__global__ void __launch_bounds__(kFinishThreads) linear_finish(FfnArgs a) {
    const int64_t quads = (a.m + 3) / 4;
    const int64_t i = int64_t(blockIdx.x) * kFinishThreads + threadIdx.x;
    if (i >= a.n * quads) return;
    const int64_t row = i / quads, r = 4 * (i - row * quads);
    const float *part = a.part + row * G * a.m + r;
    a.part = nullptr;
    f32x4 sum[G] = {};
    if (a.m % 4 == 0) {
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s)
#pragma unroll
            for (int g = 0; g < G; ++g) sum[g] += *reinterpret_cast<const f32x4 *>(part + (s * a.n * G + g) * a.m);
    } else {
        for (int s = 0; s < a.splits; ++s)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < a.m) sum[g][e] += part[(s * a.n * G + g) * a.m + e];
    }
    finish4<kLinear, G>(a, 0, 0, row, r, sum);
}

// ---------------------------------------------------------------- alignment of X
// Copies 16-bit rows with any stride and alignment to rows of k elements (a
// multiple of 16) on 16-byte boundaries: 8 elements a thread at a time.
__global__ void __launch_bounds__(kAlignThreads) align_rows(const uint16_t *x, int64_t ldx, uint16_t *y,
                                                            int64_t rows, int64_t k) {
    const int64_t pieces = k / 8;
    for (int64_t i = int64_t(blockIdx.x) * kAlignThreads + threadIdx.x; i < rows * pieces;
         i += int64_t(gridDim.x) * kAlignThreads) {
        const int64_t row = i / pieces, e = 8 * (i - row * pieces);
        uint16_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[row * ldx + e + j];
        __builtin_memcpy(y + row * k + e, v, 16);
    }
}

// ---------------------------------------------------------------- routing
struct RouteArgs {
    const uint8_t *X;
    int64_t ldx;
    const uint8_t *router;
    const float *route_bias;
    double *logits;             // [splits][tokens][experts]: sums over parts of hidden
    int32_t *offsets, *choice, *list, *active;
    float *weights;
    int64_t tokens, experts, hidden;
    int32_t splits, groups;     // splits 0: no logits, see own_logits; groups: entries of active
    int32_t topk, scoring, renormalize;
    float routed_scale;
};

// op over the 64 lanes, the same value in every lane: DPP exchanges inside
// 16-lane rows, then swaps of rows and of 32-lane halves, as wave_sum.
template <typename OP>
__device__ __forceinline__ double wave_reduce64(double v, OP op) {
    const auto joined = [](uint32_t lo, uint32_t hi) {
        return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
    };
    const auto dpp = [&](auto ctrl) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        constexpr int c = decltype(ctrl)::value;
        v = op(v, joined(__builtin_amdgcn_mov_dpp(static_cast<int>(u), c, 0xF, 0xF, false),
                         __builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), c, 0xF, 0xF, false)));
    };
    dpp(std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
    dpp(std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
    dpp(std::integral_constant<int, 0x141>{});   // row_half_mirror
    dpp(std::integral_constant<int, 0x140>{});   // row_mirror
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t lo = static_cast<uint32_t>(u), hi = static_cast<uint32_t>(u >> 32);
    const auto l16 = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto h16 = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    v = op(joined(l16[0], h16[0]), joined(l16[1], h16[1]));
    u = __builtin_bit_cast(uint64_t, v);
    lo = static_cast<uint32_t>(u);
    hi = static_cast<uint32_t>(u >> 32);
    const auto l32 = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto h32 = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    return op(joined(l32[0], h32[0]), joined(l32[1], h32[1]));
}
__device__ __forceinline__ double wave_sum64(double v) {
    return wave_reduce64(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double wave_max64(double v) {
    return wave_reduce64(v, [](double a, double b) { return fmax(a, b); });
}

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kRouteWaves = 4;
constexpr int kRouteDepth = 4;   // steps of 32 elements a wave loads at a time

// Partial logits of 16 experts and 16 tokens over one of `splits` parts of
// hidden.  Products of 16-bit values are exact in fp64 and the fp64 sums err by
// about 2^-50, so the choice of experts is the one of the exact scores unless
// these agree to some 14 digits.  The fp64 matrix instruction takes 4 elements of
// K, one per lane quarter; a lane loads 8 consecutive ones at a time, so
// instruction j of a step of 32 multiplies elements 8 q + j of all quarters q.
// 64 experts x 7168: 1 or 16 tokens 4.7 us, 64 tokens of 4096 5.4 us (summed by
// the VALU, an expert per workgroup, they took 5, 58 and 53 us).
template <bool BF16>
__global__ void __launch_bounds__(kRouteWaves * kWave) route_logits(const RouteArgs a) {
    __shared__ double red[kRouteWaves - 1][4][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int li = lane & 15, kq = lane >> 4;
    const int64_t split = blockIdx.x % a.splits, e0 = int64_t(blockIdx.x / a.splits) * kTile;
    const int64_t t0 = int64_t(blockIdx.y) * kTile;
    const int64_t steps = (a.hidden + 31) / 32;
    const int64_t first = split * steps / a.splits + wave, last = (split + 1) * steps / a.splits;
    // rows past the last repeat it; their sums are not stored
    const int64_t er = e0 + li < a.experts ? e0 + li : a.experts - 1;
    const int64_t tr = t0 + li < a.tokens ? t0 + li : a.tokens - 1;
    const uint8_t *w = a.router + 2 * er * a.hidden, *x = a.X + 2 * tr * a.ldx;
    f64x4 acc = {};
    for (int64_t s0 = first; s0 < last; s0 += kRouteWaves * kRouteDepth) {
        u32x4 wv[kRouteDepth], xv[kRouteDepth];
#pragma unroll
        for (int d = 0; d < kRouteDepth; ++d) {
            const int64_t s = s0 + kRouteWaves * d, e = 32 * s + 8 * kq;
            wv[d] = xv[d] = u32x4{0, 0, 0, 0};
            if (s < last && e < a.hidden) {
                __builtin_memcpy(&wv[d], w + 2 * e, 16);
                __builtin_memcpy(&xv[d], x + 2 * e, 16);
            }
        }
#pragma unroll
        for (int d = 0; d < kRouteDepth; ++d)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint16_t wb = static_cast<uint16_t>(wv[d][j / 2] >> (16 * (j & 1)));
                const uint16_t xb = static_cast<uint16_t>(xv[d][j / 2] >> (16 * (j & 1)));
                const float wf = BF16 ? bf16_value(wb) : static_cast<float>(__builtin_bit_cast(_Float16, wb));
                const float xf = BF16 ? bf16_value(xb) : static_cast<float>(__builtin_bit_cast(_Float16, xb));
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(double(wf), double(xf), acc, 0, 0, 0);
            }
    }
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave - 1][i][lane] = acc[i];
    __syncthreads();
    if (wave > 0 || t0 + li >= a.tokens) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        double v = acc[i];
        for (int u = 0; u < kRouteWaves - 1; ++u) v += red[u][i][lane];
        const int64_t e = e0 + 4 * i + kq;   // the fp64 instruction's row of register i
        if (e < a.experts) a.logits[(split * a.tokens + t0 + li) * a.experts + e] = v;
    }
}

constexpr int kLogitLoads = 16;
__device__ __forceinline__ double logit(const RouteArgs &a, int64_t t, int e) {
    const double *z = a.logits + t * a.experts + e;
    const int64_t stride = a.tokens * a.experts;
    double v = 0.0;
    for (int s0 = 0; s0 < a.splits; s0 += kLogitLoads) {   // the loads of a round together
        double part[kLogitLoads];
#pragma unroll
        for (int s = 0; s < kLogitLoads; ++s) part[s] = s0 + s < a.splits ? z[(s0 + s) * stride] : 0.0;
#pragma unroll
        for (int s = 0; s < kLogitLoads; ++s) v += part[s];
    }
    return v;
}
// The key experts are chosen by; a NaN counts as the least, below -infinity.
// Without a route_bias it is the logit z: both scorings grow with it, and where
// scores saturate (sigmoids from z of 37 on are all 1 in fp64) it still tells the
// experts apart.
__device__ __forceinline__ double choice_key(const RouteArgs &a, int e, double z, double score) {
    const double key = a.route_bias ? score + double(a.route_bias[e]) : z;
    return key == key ? fmax(key, -DBL_MAX) : -INFINITY;
}
__device__ __forceinline__ float routed_weight(const RouteArgs &a, double score, double chosen) {
    return static_cast<float>((a.renormalize ? score / chosen : score) * double(a.routed_scale));
}

// Chooses the experts of one token by one wave: an expert's rank is the number
// of experts ahead of it (a larger key, or an equal one at a lower index), so the
// ranks are a permutation whatever the keys hold, and rank j < topk is slot
// token * topk + j.  score, keys, order: the wave's own LDS.
__device__ __forceinline__ void choose_token(const RouteArgs &a, int64_t t, double *score, double *keys,
                                             int32_t *order) {
    const int lane = threadIdx.x % kWave, experts = static_cast<int>(a.experts);
    const bool softmax = a.scoring == NVFP4_SCORE_SOFTMAX;
    double top = -INFINITY, sum = 0.0;
    for (int e = lane; e < experts; e += kWave) {
        score[e] = keys[e] = logit(a, t, e);
        top = fmax(top, score[e]);
    }
    if (softmax) top = wave_max64(top);
    for (int e = lane; e < experts; e += kWave) sum += score[e] = softmax ? exp(score[e] - top) : exp(-score[e]);
    if (softmax) sum = wave_sum64(sum);
    for (int e = lane; e < experts; e += kWave) {
        score[e] = softmax ? score[e] / sum : 1.0 / (1.0 + score[e]);
        keys[e] = choice_key(a, e, keys[e], score[e]);
    }
    wave_lds_fence();
    double chosen = 0.0;
    for (int e = lane; e < experts; e += kWave) {
        const double key = keys[e];
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < experts; ++o) {
            const double other = keys[o];
            rank += other > key || (other == key && o < e);
        }
        if (rank < a.topk) {
            chosen += score[e];
            order[rank] = e;
            a.choice[t * a.topk + rank] = e;
        }
    }
    chosen = wave_sum64(chosen);
    wave_lds_fence();
    for (int j = lane; j < a.topk; j += kWave)
        a.weights[t * a.topk + j] = routed_weight(a, score[order[j]], chosen);
    wave_lds_fence();
}

// The slots sorted by expert, from the choice, by one workgroup: the offsets of
// the experts, the list of slots and the list of experts that have any.  The order
// inside an expert comes from an atomic and may differ between runs, but nothing
// depends on it: every slot is a column of its own in the products.
__device__ __forceinline__ void sort_slots(const RouteArgs &a) {
    __shared__ int32_t count[kMaxExperts], cursor[kMaxExperts];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int experts = static_cast<int>(a.experts);
    const int64_t slots = a.tokens * a.topk;
    for (int e = threadIdx.x; e < experts; e += blockDim.x) count[e] = 0;
    __syncthreads();   // and the choice, where this workgroup made it
    for (int64_t s = threadIdx.x; s < slots; s += blockDim.x) atomicAdd(&count[a.choice[s]], 1);
    __syncthreads();
    // lane l of wave 0 sums its run of experts, the runs are scanned (slots in the
    // low half, experts in the high)
    if (wave == 0) {
        const int per = (experts + kWave - 1) / kWave;
        const int e0 = lane * per;
        uint64_t own = 0;
        for (int e = e0; e < e0 + per && e < experts; ++e) own += count[e] > 0 ? (uint64_t(1) << 32) + count[e] : 0;
        uint64_t at = own;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const uint64_t v = __shfl_up(static_cast<unsigned long long>(at), o);
            if (lane >= o) at += v;
        }
        const int total = static_cast<int>(__shfl(static_cast<unsigned long long>(at), kWave - 1) >> 32);
        at -= own;
        for (int e = e0; e < e0 + per && e < experts; ++e) {
            a.offsets[e] = cursor[e] = static_cast<int32_t>(at);
            if (count[e] > 0) {
                a.active[at >> 32] = e;
                at += (uint64_t(1) << 32) + count[e];
            }
        }
        if (lane == kWave - 1) a.offsets[experts] = static_cast<int32_t>(at);
        for (int i = total + lane; i < a.groups; i += kWave) a.active[i] = -1;
    }
    __syncthreads();
    for (int64_t s = threadIdx.x; s < slots; s += blockDim.x)
        a.list[atomicAdd(&cursor[a.choice[s]], 1)] = static_cast<int32_t>(s);
}

// Few tokens: choice and sorting by one workgroup, a wave per token at a time.
// More: each its own kernel, a workgroup per kChooseWaves tokens (64 experts x 64
// tokens: 7 + 5 us, by one workgroup 28).
constexpr int kSelectWaves = 16, kChooseWaves = 4;
constexpr int kSelectLds = 32768;   // bytes of scores and keys

__global__ void __launch_bounds__(kSelectWaves * kWave) route_select(const RouteArgs a) {
    __shared__ double lds[kSelectLds / 8];
    __shared__ int32_t order[kSelectWaves][kMaxTopk];
    const int wave = threadIdx.x / kWave, experts = static_cast<int>(a.experts);
    const int fit = kSelectLds / 16 / experts, each = fit < kSelectWaves ? fit : kSelectWaves;   // at least 2
    double *score = lds + wave * 2 * experts;
    for (int64_t t = wave; t < a.tokens && wave < each; t += each)
        choose_token(a, t, score, score + experts, order[wave]);
    sort_slots(a);
}

__global__ void __launch_bounds__(kChooseWaves * kWave) route_choose(const RouteArgs a) {
    __shared__ double lds[kChooseWaves][2 * kMaxExperts];
    __shared__ int32_t order[kChooseWaves][kMaxTopk];
    const int wave = threadIdx.x / kWave;
    const int64_t t = int64_t(blockIdx.x) * kChooseWaves + wave;
    if (t < a.tokens) choose_token(a, t, lds[wave], lds[wave] + a.experts, order[wave]);
}

__global__ void __launch_bounds__(kSelectWaves * kWave) route_sort(const RouteArgs a) { sort_slots(a); }

// ---------------------------------------------------------------- combination
struct CombineArgs {
    const float *part, *weights;
    const void *residual;
    int64_t ldr;
    void *Y;
    int64_t ldy, tokens, hidden;
    int32_t topk, y_type;
};

constexpr int kCombineThreads = 256;

// Y of one token (blockIdx.y): its slots' partial outputs in the order of
// their ranks.  A thread makes four outputs (hidden is a multiple of 16).
__global__ void __launch_bounds__(kCombineThreads) moe_combine(const CombineArgs a) {
    const int64_t r = 4 * (int64_t(blockIdx.x) * kCombineThreads + threadIdx.x), t = blockIdx.y;
    if (r >= a.hidden) return;
    const float *part = a.part + t * a.topk * a.hidden + r, *w = a.weights + t * a.topk;
    f32x4 y = {};
#pragma unroll 8
    for (int j = 0; j < a.topk; ++j) y += w[j] * *reinterpret_cast<const f32x4 *>(part + j * a.hidden);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (a.residual) y[e] += load_as_float(a.residual, t * a.ldr + r + e, a.y_type);
        store_rounded(a.Y, t * a.ldy + r + e, a.y_type, y[e]);
    }
}

// ---------------------------------------------------------------- few slots
// The MoE layer where few experts share tokens (one token above all): a slot is
// taken by itself, so the slots need no sorting.  Its expert is chosen by each
// workgroup that multiplies for it, and the down product's workgroups, which own
// rows of a token's output, finish the output themselves: three launches, and no
// partial outputs in memory.  Where the router is small the workgroups of the up
// product compute the logits, too: two launches.  7168 x 2048, 8 of 64 experts, one token: 52 us
// (logits 4.7, up product with the choice 28, down product 17), where the five
// kernels take 65; the weights' 198 MB take 31 at the rate of a large read.

constexpr int kSlotUpWaves = 4;
constexpr int kSlotWaves = 8;                   // of the slots' down product

struct SlotArgs {
    FfnArgs f;
    RouteArgs r;
};

// The logits of one token by a workgroup, in fp64 as route_logits: a wave takes
// four experts at a time, a lane 8 elements of hidden.
template <bool BF16, int THREADS>
__device__ __forceinline__ void own_logits(const RouteArgs &a, int64_t t, double *score) {
    constexpr int kEach = 4;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, experts = static_cast<int>(a.experts);
    const uint8_t *x = a.X + 2 * t * a.ldx;
    for (int e0 = kEach * wave; e0 < experts; e0 += kEach * (THREADS / kWave)) {
        double s[kEach] = {};
        for (int64_t i = 8 * lane; i < a.hidden; i += 8 * kWave) {
            u32x4 xv, wv[kEach];
            __builtin_memcpy(&xv, x + 2 * i, 16);
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int64_t e = e0 + k < experts ? e0 + k : experts - 1;
                __builtin_memcpy(&wv[k], a.router + 2 * (e * a.hidden + i), 16);
            }
            const auto value = [](const u32x4 &v, int j) {
                const uint16_t b = static_cast<uint16_t>(v[j / 2] >> (16 * (j & 1)));
                return double(BF16 ? bf16_value(b) : static_cast<float>(__builtin_bit_cast(_Float16, b)));
            };
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < kEach; ++k) s[k] = __builtin_fma(value(wv[k], j), value(xv, j), s[k]);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            s[k] = wave_sum64(s[k]);
            if (lane == 0 && e0 + k < experts) score[e0 + k] = s[k];
        }
    }
}

// The expert of rank j of token t, to every thread of the workgroup.  `weigh`
// (workgroup-uniform): its weight, too, to memory.
template <bool BF16, int THREADS>
__device__ __forceinline__ int choose_slot(const RouteArgs &a, int64_t t, int j, bool weigh) {
    __shared__ double score[kMaxExperts], keys[kMaxExperts], red[2][THREADS / kWave];
    __shared__ int32_t rank[kMaxExperts], order[kMaxTopk];
    constexpr int kWaves = THREADS / kWave;
    const int experts = static_cast<int>(a.experts), thread = threadIdx.x, wave = thread / kWave;
    double top = -INFINITY;
    if (a.splits == 0) {   // uniform: a small router
        own_logits<BF16, THREADS>(a, t, score);
        __syncthreads();
    }
    for (int e = thread; e < experts; e += THREADS) {
        if (a.splits > 0) score[e] = logit(a, t, e);
        keys[e] = score[e];
        rank[e] = 0;
        top = fmax(top, score[e]);
    }
    const bool softmax = a.scoring == NVFP4_SCORE_SOFTMAX;
    double sum = 0.0;
    if (softmax) {
        top = wave_max64(top);
        if (thread % kWave == 0) red[0][wave] = top;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) top = fmax(top, red[0][w]);
    }
    for (int e = thread; e < experts; e += THREADS) sum += score[e] = softmax ? exp(score[e] - top) : exp(-score[e]);
    if (softmax) {
        sum = wave_sum64(sum);
        if (thread % kWave == 0) red[1][wave] = sum;
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < kWaves; ++w) sum += red[1][w];
    }
    for (int e = thread; e < experts; e += THREADS) {
        score[e] = softmax ? score[e] / sum : 1.0 / (1.0 + score[e]);
        keys[e] = choice_key(a, e, keys[e], score[e]);
    }
    __syncthreads();
    // the waves share the comparisons
    for (int e = thread % kWave; e < experts; e += kWave) {
        const double key = keys[e];
        int ahead = 0;
#pragma unroll 4
        for (int o = wave; o < experts; o += kWaves) {
            const double other = keys[o];
            ahead += other > key || (other == key && o < e);
        }
        atomicAdd(&rank[e], ahead);
    }
    __syncthreads();
    for (int e = thread; e < experts; e += THREADS)
        if (rank[e] < a.topk) order[rank[e]] = e;
    __syncthreads();
    const int expert = order[j];
    if (weigh && thread == 0) {
        double chosen = 0.0;
        if (a.renormalize)
            for (int i = 0; i < a.topk; ++i) chosen += score[order[i]];
        a.choice[t * a.topk + j] = expert;
        a.weights[t * a.topk + j] = routed_weight(a, score[expert], chosen);
    }
    return expert;
}

// h of one slot: workgroup = strip of rows and slot.
template <bool BF16, int L>
__global__ void __launch_bounds__(kSlotUpWaves * kWave, 2) ffn_slot_up(const SlotArgs s) {
    __shared__ u32x4 lds[stream_lds<2, 1, kSlotUpTiles, kSlotUpWaves, 1>()];
    const uint32_t strips = static_cast<uint32_t>((s.f.m + kSlotUpTiles * kTile - 1) / (kSlotUpTiles * kTile));
    const uint32_t slot = blockIdx.x / strips, strip = blockIdx.x - slot * strips;
    const uint32_t token = slot / s.r.topk;
    const int expert = __builtin_amdgcn_readfirstlane(
        choose_slot<BF16, kSlotUpWaves * kWave>(s.r, token, slot - token * s.r.topk, strip == 0));
    stream_pass<BF16, L, 2, 1, kSlotUp, kSlotUpTiles, 3, kSlotUpWaves, 1>(s.f, expert, int64_t(strip) * kSlotUpTiles * kTile,
                                                                          0, slot, slot + 1, lds);
}

// Y of 16 rows of one token: the waves share the token's slots, or several waves
// a slot's K where there are fewer slots than waves; the slots' outputs are added
// in the order of their ranks.
template <int L, int P>
__global__ void __launch_bounds__(kSlotWaves * kWave, 2) ffn_slot_down(const SlotArgs s, const CombineArgs y) {
    __shared__ u32x4 lds[kSlotWaves * P * 2 * 32];
    __shared__ float sums[kMaxTopk > kSlotWaves ? kMaxTopk : kSlotWaves][kTile];
    __shared__ float weights[kMaxTopk], alphas[kMaxTopk];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // the workgroups of a strip lie on the same die, whose L2 serves experts that
    // tokens share
    const uint32_t tokens = static_cast<uint32_t>(y.tokens), b = blockIdx.x / kXcds;
    const int64_t strip = int64_t(b / tokens) * kXcds + blockIdx.x % kXcds, t = b % tokens;
    if (strip * kTile >= s.f.m) return;   // workgroup-uniform
    const int topk = y.topk, share = topk < kSlotWaves ? kSlotWaves / topk : 1;
    if (static_cast<int>(threadIdx.x) < topk) {   // for the end, ahead of the weights
        const int64_t slot = t * topk + threadIdx.x;
        weights[threadIdx.x] = y.weights[slot];
        alphas[threadIdx.x] = s.f.alpha ? s.f.alpha[s.r.choice[slot]] : 1.0f;
    }
    const bool last = threadIdx.x < kTile;
    const int64_t r = strip * kTile + threadIdx.x;
    const float residual = last && y.residual ? load_as_float(y.residual, t * y.ldr + r, y.y_type) : 0.0f;
    for (int j = wave / share; j < topk; j += kSlotWaves / share) {
        const int32_t slot = static_cast<int32_t>(t * topk + j);
        f32x4 acc[1][1];
        stream_sums<true, L, 1, P, kSlotDown, 1, 2, 1>(s.f, s.r.choice[slot], strip * kTile, 0, slot, slot + 1,
                                                       lds + wave * (P * 2 * 32), wave % share, share, acc);
        if (lane % kTile == 0)
            *reinterpret_cast<f32x4 *>(&sums[j * share + wave % share][4 * (lane / kTile)]) = acc[0][0];
    }
    __syncthreads();
    if (!last) return;
    float out = 0.0f;
    for (int j = 0; j < topk; ++j) {
        float v = sums[j * share][threadIdx.x];
        for (int i = 1; i < share; ++i) v += sums[j * share + i][threadIdx.x];
        out += weights[j] * (alphas[j] * v);
    }
    if (y.residual) out += residual;
    store_rounded(y.Y, t * y.ldy + r, y.y_type, out);
}

}  // namespace

#endif  // NVFP4_FFN_KERNELS_H
