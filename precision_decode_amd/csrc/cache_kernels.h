// Device code of the key/value cache's writers and reader: head norms with the
// position rotation, NVFP4 quantisation of keys and values into their slots,
// and reading slots back (nvfp4_attn.h says what they compute).  Not part of
// the C ABI.
//
// All three move bytes: a row of head_dim elements is read once and written once,
// 16 bytes a lane.  Queries and keys of 4096 tokens normalised and rotated (64 rows of
// 128, 136 MB): 34 - 36 us, 3.9 TB/s, against 27 at the rate of a copy; vector
// instructions, 229 per 8 elements (the sum of squares, the rotation, the roundings,
// addresses), are issued for 0.92 of the time.  Keys and values of 8192 tokens, 8 heads of
// 128, into the cache: 20 us, 204 instructions per 8 elements (0.69 of the time), and back
// 12.9 us, 140 instructions (0.78).  Scales lie [block][token], a byte each, so that a
// token's writer stores and its reader loads single bytes of lines that other tokens'
// workgroups use too: 16.8 MB written for 9.4, 25.8 MB read for 9.4.
#ifndef NVFP4_CACHE_KERNELS_H
#define NVFP4_CACHE_KERNELS_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "attn_plan.h"
#include "device_common.h"
#include "nvfp4_attn.h"
#include "quant_arith.h"

namespace nvfp4attn {

using nvfp4dev::f16x2;
using nvfp4dev::f32x2;
using nvfp4dev::f32x4;
using nvfp4dev::kWave;
using nvfp4dev::u32x4;

using nvfp4attnplan::kRowThreads;
// Rows of one token that a group of lanes takes one after the other, all loads
// first: its cosines and sines are read once for them.
using nvfp4attnplan::kRowsInFlight;

struct Rows {
    const uint16_t *p;
    int64_t token, head;   // strides in elements
    bool wide;             // every row is 16-byte aligned
};

struct CacheArgs {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const float *k_global, *v_global;
    int64_t slots;         // pages * page_size
    int32_t page_log2, kv_heads, head_dim, dp;
};

struct RowArgs {
    Rows q, k, v;          // q.p is NULL in a plain cache write
    uint16_t *q_out, *k_out;
    int64_t qo_token, qo_head, ko_token, ko_head;
    bool qo_wide, ko_wide;
    const float *q_weight, *k_weight;
    const int64_t *positions;
    const float *cos_sin;
    int64_t table_rows, tokens;
    int32_t heads, kv_heads, head_dim, rot_dim;
    int32_t each;          // rows of a chunk, at most kRowsInFlight
    int32_t q_chunks, k_chunks, chunks;   // chunks of a token: queries', keys', all with values'
    int32_t interleaved, bf16, rule;
    float eps, inverse_dim;
    CacheArgs cache;
    const int64_t *slots;  // NULL: no cache
};

struct ReadArgs {
    CacheArgs cache;
    const int64_t *slots;
    void *k, *v;
    int64_t tokens;
    int32_t y_type;
    bool wide;
};

__device__ __forceinline__ float from16(uint32_t h, bool bf16) {
    return bf16 ? __uint_as_float(h << 16)
                : static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}
// Two floats rounded to nearest even, a in the low half.
__device__ __forceinline__ uint32_t pair16(float a, float b, bool bf16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return bf16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2))
                : nvfp4dev::bits(__builtin_convertvector(f32x2{a, b}, f16x2));
}
__device__ __forceinline__ uint32_t to16(float f, bool bf16) { return pair16(f, 0.0f, bf16) & 0xFFFFu; }

// 8 elements, two per word.
__device__ __forceinline__ u32x4 load8(const uint16_t *p, bool wide) {
    if (wide) return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | static_cast<uint32_t>(p[2 * i + 1]) << 16;
    return w;
}
__device__ __forceinline__ void store8(uint16_t *p, u32x4 w, bool wide) {
    if (wide) {
        *reinterpret_cast<u32x4 *>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[2 * i] = static_cast<uint16_t>(w[i]);
        p[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
}
__device__ __forceinline__ void widen(u32x4 w, bool bf16, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = from16(w[i] & 0xFFFFu, bf16);
        x[2 * i + 1] = from16(w[i] >> 16, bf16);
    }
}
__device__ __forceinline__ u32x4 narrow(const float (&x)[8], bool bf16) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pair16(x[2 * i], x[2 * i + 1], bf16);
    return w;
}

// E2M1 codes of 8 values that are neither NaN nor -0, element i at nibble i, on
// the gfx950 FP4 conversion (nearest even, saturating at 6).  The other rules
// move a value across the conversion's ties first: nearest-lower takes the ties
// that go up (0.75, 1.75, 3.5: mantissa bit 22 set, bits 20..0 clear) one ulp
// towards zero; half-step shifts its cut points 2.75, 3.75 and 5.25 onto the
// ties 2.5, 3.5 and 5 (kHalfStepScale).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], int rule) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = v[i];
        if (rule == NVFP4_ROUND_NEAREST_LOWER) {
            const uint32_t b = __float_as_uint(v[i]);
            t[i] = __uint_as_float(b - ((b & 0x005FFFFFu) == 0x00400000u ? 1u : 0u));
        } else if (rule == NVFP4_ROUND_HALF_STEP) {
            const float a = __builtin_fabsf(v[i]);
            t[i] = __builtin_copysignf(
                __builtin_amdgcn_fmed3f(
                    __builtin_fmaf(a, nvfp4quant::kHalfStepScale, nvfp4quant::kHalfStepShift), a, 2.0f),
                v[i]);
        }
    }
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[0], t[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.0f, 3);
    return w;
}

// This lane's 8 of a block's 16 values (`w` as they are stored, x as floats; the
// neighbour lane has the others): codes and the block's scale code, the arithmetic of
// nvfp4_quantize.h.  For ordinary values and scales the two divisions of an element are
// products that round as the divisions do (quot_f64, quot_short); `inverse` is 1 / g in
// 64 bits.
__device__ __forceinline__ uint32_t quantize8(u32x4 w, const float (&x)[8], float g, double inverse, bool bf16, int rule,
                                              uint32_t *scale) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    // the largest magnitude by its bit pattern, where NaN comes above infinity, and the
    // smallest that is not zero (less one: zero wraps to the top)
    u16x2 high = {0, 0}, low = {0xFFFF, 0xFFFF};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u16x2 m = __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu);
        high = __builtin_elementwise_max(high, m);
        low = __builtin_elementwise_min(low, static_cast<u16x2>(m - u16x2{1, 1}));
    }
    uint32_t top = high.x > high.y ? high.x : high.y;
    const uint32_t tiny = low.x < low.y ? low.x : low.y;
    const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(top), 0xB1, 0xF, 0xF, false));
    top = other > top ? other : top;
    // every nonzero bf16 magnitude at least 2^-100 (fp16 ones all are)
    const bool fast = g >= 0x1p-40f && g <= 0x1p30f && (!bf16 || tiny >= (27u << 7) - 1u);
    // rounding is monotonic: max |x / g| is max |x| / |g|
    const float largest = from16(top, bf16);
    float am = fast ? nvfp4quant::quot_f64(largest, inverse) : largest / __builtin_fabsf(g);
    am = am < 1e-8f ? 1e-8f : am;                     // NaN stays NaN
    const uint32_t s = nvfp4quant::e4m3_code_pos(nvfp4quant::quot_f64(am, 1.0 / 6.0));
    *scale = s;
    if (s == 0x7Fu) return 0u;                        // a NaN scale: every code is 0
    const float sv = nvfp4quant::e4m3_value_pos(s);
    const float den = sv < 1e-8f ? 1e-8f : sv;
    float v[8];
    if (fast && s != 0u) {                            // s = 0: den is no 4-bit number
        const float y = __builtin_amdgcn_rcpf(den);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = nvfp4quant::quot_short(nvfp4quant::quot_f64(x[i], inverse), den, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i] / g / den + 0.0f;   // -0 -> +0: its code is 0
    }
    return codes8(v, rule);
}

// 1 / sqrt(v) to about one unit in the last place, also where v is subnormal (which
// the instruction takes as zero).
__device__ __forceinline__ float inverse_root(float v) {
    const bool small = v < 0x1p-100f;
    const float y = __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v);
    return small ? y * 0x1p32f : y;
}

// Sum over the L lanes of a group, the same in each.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// One group of L lanes takes up to kRowsInFlight rows of one token: queries, then
// keys, then values.  L * 8 elements hold a row.
template <int L, bool kBf16>
__global__ __launch_bounds__(kRowThreads) void norm_rope_rows(const RowArgs a) {
    const int l = threadIdx.x % L;
    const uint32_t group = blockIdx.x * (kRowThreads / L) + threadIdx.x / L;   // below 2^28
    const uint32_t token = group / static_cast<uint32_t>(a.chunks);
    if (token >= static_cast<uint32_t>(a.tokens)) return;   // whole groups
    const int64_t t = token;
    // a chunk holds rows of one kind, queries first, then keys, then values
    const int chunk = static_cast<int>(group - token * static_cast<uint32_t>(a.chunks));
    const bool is_q = chunk < a.q_chunks, is_v = chunk >= a.q_chunks + a.k_chunks;
    const int first = (is_q ? chunk : is_v ? chunk - a.q_chunks - a.k_chunks : chunk - a.q_chunks) * a.each;
    const int rest = (is_q ? a.heads : a.kv_heads) - first, left = rest < a.each ? rest : a.each;
    const int e0 = 8 * l;                             // this lane's first element
    const bool inside = e0 < a.head_dim;
    const bool cached = a.slots != nullptr && !is_q;

    const Rows r = is_q ? a.q : is_v ? a.v : a.k;
    const uint16_t *from = r.p + t * r.token + first * r.head + e0;
    const float *global = is_v ? a.cache.v_global : a.cache.k_global;
    u32x4 raw[kRowsInFlight];
    float g[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        raw[i] = u32x4{0, 0, 0, 0};
        g[i] = 1.0f;
        if (i < left && inside) raw[i] = load8(from + i * r.head, r.wide);
        if (i < left && cached && global != nullptr) g[i] = global[first + i];
    }
    float weight[8];
    const float *w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
    if (w != nullptr && inside) {
        const f32x4 w0 = *reinterpret_cast<const f32x4 *>(w + e0), w1 = *reinterpret_cast<const f32x4 *>(w + e0 + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) weight[j] = j < 4 ? w0[j % 4] : w1[j % 4];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) weight[j] = 1.0f;
    }
    int64_t slot = -1;
    if (cached) {
        slot = a.slots[t];
        if (slot >= a.cache.slots) slot = -1;
    }
    const int64_t page = slot >> a.cache.page_log2;
    const int64_t off = slot & ((int64_t(1) << a.cache.page_log2) - 1);
    const int64_t head = page * a.cache.kv_heads + first;
    uint8_t *codes_at = (is_v ? a.cache.v_codes : a.cache.k_codes) + ((head << a.cache.page_log2) + off) * (a.cache.dp / 2) + 4 * l;
    uint8_t *scales_at = (is_v ? a.cache.v_scales : a.cache.k_scales) +
                         ((head * (a.cache.dp / 16) + l / 2) << a.cache.page_log2) + off;
    const int codes_step = (a.cache.dp / 2) << a.cache.page_log2, scales_step = (a.cache.dp / 16) << a.cache.page_log2;
    const int64_t to_head = is_q ? a.qo_head : a.ko_head;
    uint16_t *to = is_q ? a.q_out + t * a.qo_token + first * to_head + e0 : a.k_out + t * a.ko_token + first * to_head + e0;
    const bool to_wide = is_q ? a.qo_wide : a.ko_wide;
    // cosines and sines of this lane's elements
    const int half = a.rot_dim / 2;
    const bool turned = e0 < a.rot_dim;
    float cs[8], sn[8];
    bool known = true;
    if (a.rot_dim > 0 && !is_v) {
        const int64_t p = a.positions[t];
        known = p >= 0 && p < a.table_rows;
        if (turned && known) {
            const float *row = a.cos_sin + p * a.rot_dim;
            if (a.interleaved) {
                const f32x4 c = *reinterpret_cast<const f32x4 *>(row + e0 / 2);
                const f32x4 s = *reinterpret_cast<const f32x4 *>(row + half + e0 / 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cs[2 * j] = cs[2 * j + 1] = c[j];
                    sn[2 * j] = -s[j];
                    sn[2 * j + 1] = s[j];
                }
            } else {
                const int i0 = e0 < half ? e0 : e0 - half;
                const f32x4 *c = reinterpret_cast<const f32x4 *>(row + i0);
                const f32x4 *s = reinterpret_cast<const f32x4 *>(row + half + i0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    cs[j] = c[j / 4][j % 4];
                    sn[j] = e0 < half ? -s[j / 4][j % 4] : s[j / 4][j % 4];
                }
            }
        }
    }
    // the lane that holds the other elements of this lane's pairs
    const int partner = (threadIdx.x & (kWave - 1)) + (!turned || a.interleaved ? 0 : e0 < half ? half / 8 : -(half / 8));

#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        if (i >= left) return;                        // whole groups
        float x[8];
        widen(raw[i], kBf16, x);
        u32x4 out = raw[i];                           // values go on as they are
        if (!is_v) {
            if (w != nullptr) {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
                const float rr = inverse_root(group_sum<L>(sum) * a.inverse_dim + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * rr * weight[j];
            }
            if (a.rot_dim > 0) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = a.interleaved ? x[j ^ 1] : __shfl(x[j], partner, kWave);
                if (!known) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(0x7FC00000u);
                } else if (turned) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * cs[j] + y[j] * sn[j];
                }
            }
            out = narrow(x, kBf16);
        }
        if (!cached) {
            if (inside) store8(to + i * to_head, out, to_wide);
            continue;
        }
        // the cache holds the rows as rounded to x_type, so that this call and a
        // plain write of its outputs leave the same codes
        if (!inside) out = u32x4{0, 0, 0, 0};
        widen(out, kBf16, x);
        uint32_t scale;
        uint32_t codes = quantize8(out, x, g[i], nvfp4quant::recip_f64(static_cast<double>(g[i])), kBf16, a.rule, &scale);
        if (!inside) codes = scale = 0u;              // the padding up to dp
        if (slot < 0 || e0 >= a.cache.dp) continue;
        *reinterpret_cast<uint32_t *>(codes_at + static_cast<int64_t>(i) * codes_step) = codes;
        if (l % 2 == 0) scales_at[static_cast<int64_t>(i) * scales_step] = static_cast<uint8_t>(scale);
    }
}

// One lane reads 8 elements of a row (4 bytes of codes and their block's scale).
template <int L>
__global__ __launch_bounds__(kRowThreads) void read_rows(const ReadArgs a) {
    const int l = threadIdx.x % L;
    const uint32_t row = blockIdx.x * (kRowThreads / L) + threadIdx.x / L;   // below 2^28
    const CacheArgs &c = a.cache;
    const uint32_t token = row / (2u * static_cast<uint32_t>(c.kv_heads));
    const int e0 = 8 * l;
    if (token >= static_cast<uint32_t>(a.tokens) || e0 >= c.head_dim) return;
    const int64_t t = token;
    const int j = static_cast<int>(row - token * (2u * static_cast<uint32_t>(c.kv_heads)));
    const bool is_v = j >= c.kv_heads;
    const int h = is_v ? j - c.kv_heads : j;
    const int64_t slot = a.slots[t];
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0 && slot < c.slots) {
        const int64_t page = slot >> c.page_log2;
        const int64_t off = slot & ((int64_t(1) << c.page_log2) - 1);
        const int64_t head = page * c.kv_heads + h;
        const uint8_t *codes = is_v ? c.v_codes : c.k_codes, *scales = is_v ? c.v_scales : c.k_scales;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + ((head << c.page_log2) + off) * (c.dp / 2) + 4 * l);
        const float s = nvfp4dev::e4m3x2_f32(scales[((head * (c.dp / 16) + l / 2) << c.page_log2) + off]).x;
        const float *global = is_v ? c.v_global : c.k_global;
        const float g = global != nullptr ? global[h] : 1.0f;
        const f16x2 p[4] = {nvfp4dev::e2m1x2_f16<0>(w), nvfp4dev::e2m1x2_f16<1>(w), nvfp4dev::e2m1x2_f16<2>(w),
                            nvfp4dev::e2m1x2_f16<3>(w)};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(p[i / 2][i % 2]) * s * g;   // the first product is exact
    }
    const int64_t at = (t * c.kv_heads + h) * c.head_dim + e0;
    void *out = is_v ? a.v : a.k;
    if (a.y_type == NVFP4_OUT_F32) {
        float *o = static_cast<float *>(out) + at;
        if (a.wide) {
            reinterpret_cast<f32x4 *>(o)[0] = f32x4{x[0], x[1], x[2], x[3]};
            reinterpret_cast<f32x4 *>(o)[1] = f32x4{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = x[i];
        }
    } else {
        store8(static_cast<uint16_t *>(out) + at, narrow(x, a.y_type == NVFP4_OUT_BF16), a.wide);
    }
}

}  // namespace nvfp4attn

#endif  // NVFP4_CACHE_KERNELS_H
