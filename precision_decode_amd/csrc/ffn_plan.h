// Host-side plan of the feed-forward operators on NVFP4 weights (the linear
// layer with a fused epilogue and the mixture-of-experts layer): argument
// checks, kernel choice, grids and workspace layout.
//
// Plain C++17 with no HIP types, so that the same code is compiled into the
// library (nvfp4_ffn.hip) and into host-only checks built with g++ and the
// address and undefined-behaviour sanitizers.  Not part of the C ABI.
#ifndef NVFP4_FFN_PLAN_H
#define NVFP4_FFN_PLAN_H

#include <climits>
#include <cstddef>
#include <cstdint>

#include "nvfp4_ffn.h"

namespace nvfp4ffnplan {

constexpr int kTile = 16;                          // MFMA tile: 16 weight rows x 16 tokens
constexpr int kWinElems = 256;                     // K elements of one packed window
constexpr int64_t kMaxK = int64_t(1) << 22;        // k and ldx: keeps row offsets within 31 bits
constexpr int64_t kMaxLd = int64_t(1) << 31;       // ldy and ldr
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopk = 64;
constexpr int64_t kMaxTokens = 65535;              // of a MoE call (a grid's second dimension)
constexpr int64_t kMaxTiles = int64_t(1) << 24;    // workgroups of 256 threads: below 2^32 threads
constexpr int64_t kReach = int64_t(1) << 31;       // bytes that a kernel's 32-bit offsets reach from a base
constexpr size_t kWsAlign = 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool mul_fits(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }
inline size_t ws_round(size_t b) { return (b + kWsAlign - 1) & ~(kWsAlign - 1); }
inline int type_bytes(int32_t t) { return t == NVFP4_OUT_F32 ? 4 : 2; }

inline bool act_known(int32_t a) { return a >= NVFP4_ACT_NONE && a <= NVFP4_ACT_SILU; }
inline bool in_type_known(int32_t t) { return t == NVFP4_OUT_F16 || t == NVFP4_OUT_BF16; }
inline bool out_type_known(int32_t t) { return in_type_known(t) || t == NVFP4_OUT_F32; }
inline bool layout_known(int32_t w) { return w == NVFP4_W_ROW_MAJOR || w == NVFP4_W_PACKED; }

inline bool k_ok(int64_t k, int32_t w_layout) {
    return k >= 16 && k <= kMaxK && k % (w_layout == NVFP4_W_PACKED ? 64 : 16) == 0;
}

// Bytes of the codes and scales of `groups` matrices of rows x k.
inline bool weight_bytes(int64_t groups, int64_t rows, int64_t k, int32_t w_layout, int64_t *codes,
                         int64_t *scales) {
    const int64_t r = w_layout == NVFP4_W_PACKED ? ceil_div(rows, kTile) * kTile : rows;
    const int64_t kk = w_layout == NVFP4_W_PACKED ? ceil_div(k, kWinElems) * kWinElems : k;
    if (!mul_fits(groups, r) || !mul_fits(groups * r, kk)) return false;
    *codes = groups * r * (kk / 2);
    *scales = groups * r * (kk / 16);
    return true;
}

// Bytes from the first to past the last element of `rows` rows of `cols`
// elements, `ld` apart.
inline bool span_bytes(int64_t rows, int64_t cols, int64_t ld, int bytes, int64_t *out) {
    if (rows == 0) { *out = 0; return true; }
    if (!mul_fits(rows - 1, ld)) return false;
    const int64_t e = (rows - 1) * ld;
    if (e > INT64_MAX / bytes - cols) return false;
    *out = (e + cols) * bytes;
    return true;
}

// Rows of `width` bytes, `stride` bytes apart, that take `span` bytes from `at` on.
struct RowSpan {
    uintptr_t at;
    int64_t span, width, stride;
};

// Whether an element of one may be an element of the other.  Rows of the same
// stride may lie between each other: column ranges of one matrix.
inline bool rows_overlap(const RowSpan &a, const RowSpan &b) {
    if (a.span <= 0 || b.span <= 0 || a.at >= b.at + static_cast<uintptr_t>(b.span) ||
        b.at >= a.at + static_cast<uintptr_t>(a.span))
        return false;
    if (a.stride != b.stride || a.width > a.stride || b.width > b.stride) return true;
    const uintptr_t stride = static_cast<uintptr_t>(a.stride);
    const uintptr_t apart = b.at >= a.at ? (b.at - a.at) % stride : (stride - (a.at - b.at) % stride) % stride;
    return apart < static_cast<uintptr_t>(a.width) || apart + static_cast<uintptr_t>(b.width) > stride;
}

inline int check_linear_shape(int64_t n, int64_t m, int64_t k, int32_t w_layout) {
    if (n < 0 || m < 1 || !k_ok(k, w_layout) || n >= (int64_t(1) << 31) || m >= (int64_t(1) << 31))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    if (ceil_div(n, kTile) * ceil_div(m, kTile) >= kMaxTiles) return NVFP4_GEMV_ERR_BAD_SHAPE;
    int64_t c, s;
    if (!weight_bytes(2, m, k, w_layout, &c, &s)) return NVFP4_GEMV_ERR_BAD_SHAPE;
    return NVFP4_GEMV_OK;
}

inline int check_moe_shape(const nvfp4_moe_layer_t &l, int64_t tokens) {
    if (l.experts < 1 || l.experts > kMaxExperts || l.topk < 1 || l.topk > kMaxTopk ||
        l.topk > l.experts || tokens < 0 || tokens > kMaxTokens ||
        !k_ok(l.hidden, l.w_layout) || !k_ok(l.inter, l.w_layout) ||
        l.experts * ceil_div(l.hidden, kTile) >= kMaxTiles || l.experts * ceil_div(l.inter, kTile) >= kMaxTiles)
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    int64_t c, s;
    if (!weight_bytes(2 * l.experts, l.inter, l.hidden, l.w_layout, &c, &s) ||
        !weight_bytes(l.experts, l.hidden, l.inter, l.w_layout, &c, &s))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    return NVFP4_GEMV_OK;
}

// ---------------------------------------------------------------- linear
constexpr int64_t kStreamTokens = 16;   // tokens of a workgroup of the stream kernel
constexpr int64_t kStreamOnlyTokens = 8;
constexpr int64_t kComputeUnits = 256;  // CUs of an MI355X (8 XCDs x 32)
// Waves of a stream workgroup: 4 where the workgroups go round the compute units
// twice, else 8 (14336 x 4096, 896 workgroups: 1 token 9.8 and 12.2 us, 4 tokens
// 11.4 and 13.7; 37 tokens of 1001 x 2064, 189 workgroups: 15.4 and 9.3).
constexpr int kStreamWaves = 8, kStreamWavesMany = 4;

// Shapes of the tile kernel, largest first.  A workgroup owns rows() rows of each
// matrix and tokens() tokens; its wk groups of wm waves take the windows of K in
// turn.  A wave holds q row tiles of each matrix times nt token tiles.
// us[i]: what a weight of 28 windows (k = 7168) takes where every compute unit
// has i + 1 workgroups, as measured with bf16 (0: they do not fit).
struct TileKind {
    int q, nt, wm, wk;
    float us[4];
    constexpr int rows() const { return kTile * q * wm; }
    constexpr int tokens() const { return kTile * nt; }
    constexpr int waves() const { return wm * wk; }
};
constexpr TileKind kTileKinds[] = {
    {2, 16, 8, 1, {210, 0, 0, 0}}, {2, 8, 8, 1, {111, 0, 0, 0}}, {2, 8, 4, 2, {70, 0, 0, 0}},
    {2, 4, 4, 2, {41, 72, 0, 0}},  {1, 4, 4, 2, {32, 50, 0, 0}}, {1, 2, 4, 2, {20, 36, 50, 61}}};
// two matrices: half the rows of each, so that a wave holds as many sums
constexpr TileKind kGatedTileKinds[] = {
    {1, 16, 8, 1, {210, 0, 0, 0}}, {1, 8, 8, 1, {111, 0, 0, 0}}, {1, 8, 4, 2, {70, 0, 0, 0}},
    {1, 4, 4, 2, {41, 72, 0, 0}},  {1, 2, 4, 2, {28, 45, 0, 0}}};
constexpr int kNumTileKinds = 6, kNumGatedTileKinds = 5;
// The rows of a workgroup's tokens lie up to kMaxK elements apart and are read by
// offsets from the first one's: 256 tokens take the whole reach, to the last byte.
template <int N>
constexpr bool tokens_in_reach(const TileKind (&kinds)[N]) {
    for (const TileKind &t : kinds)
        if (t.tokens() * kMaxK * 2 > kReach) return false;
    return true;
}
static_assert(tokens_in_reach(kTileKinds) && tokens_in_reach(kGatedTileKinds), "token offsets within the reach");
// the stream kernel's, for up to 8 and up to 16 tokens, one and two matrices
constexpr float kStreamUs[2][2][4] = {{{6, 8, 0, 0}, {8, 12, 0, 0}}, {{9, 11.5f, 0, 0}, {11, 18, 0, 0}}};
constexpr int64_t kMaxStreamSplits = 64;
constexpr float kRoundUs = 3;            // until a workgroup has its first operands
constexpr float kFinishUs = 6;           // a second kernel that adds the sums of a split of K
constexpr float kFinishBytesPerUs = 3e6;
constexpr int64_t kMaxSplits = 8;

// Time of `count` workgroups that go over `wins` windows each.
inline float rounds_us(const float (&us)[4], int64_t count, int64_t wins) {
    int most = 4;
    while (us[most - 1] == 0) --most;
    const int64_t per = ceil_div(count, kComputeUnits);   // on the busiest compute unit
    const int64_t rest = per % most;
    return static_cast<float>(ceil_div(per, most)) * kRoundUs +
           (static_cast<float>(per / most) * us[most - 1] + (rest ? us[rest - 1] : 0.0f)) *
               static_cast<float>(wins) / 28.0f;
}

// Workgroups that copy X to aligned rows, a thread per 8 elements at a time: at
// most 16 rounds of the 8 that a compute unit holds, so that X of any size keeps
// the launch within 2^32 threads.
constexpr int kAlignThreads = 256;
constexpr int64_t kMaxAlignGroups = 128 * kComputeUnits;
inline int64_t align_groups(int64_t n, int64_t k) {
    const int64_t want = ceil_div(n * (k / 8), kAlignThreads);
    return want < kMaxAlignGroups ? want : kMaxAlignGroups;
}

struct LinearPlan {
    bool stream;        // stream kernel
    int tile;           // shape of the tile kernel, or -1; neither: the simple kernel
    int waves;          // of a stream workgroup
    int64_t strips;     // workgroups along the rows
    int64_t blocks;     // workgroups along the tokens
    int64_t splits;     // workgroups along K
    size_t part_bytes;  // split sums
    size_t x_bytes;     // aligned copy of X
    size_t ws_bytes() const { return ws_round(part_bytes) + ws_round(x_bytes); }
};

// `fast`: the weight's alignment allows the fast kernels; `x_aligned`: so do X's
// rows.  What the times above say is fastest: up to 8 tokens of the stream kernel
// with K whole or split, for more also of the stream kernel in blocks of 16
// tokens, which reads and decodes the weights once a block but has the most
// workgroups, and the shapes of the tile kernel, which read and decode the less
// per product the larger they are.  Measured, in us, for 256 x 256, 256 x 128,
// 128 x 128, 128 x 64, 64 x 64 tiles on 4096 x 7168: 256 tokens -, 96, 60, 37, 32;
// 512 tokens -, 96, 61, 41, 50; 1024 tokens -, 98, 70, 72, 93; 4096 tokens 194,
// 214, 274, -, -.  K whole and split: 64 tokens 20.7 and 17.8 (in two); 32 tokens,
// 7168 x 2048, 9.4 and 12.4.
inline LinearPlan plan_linear(int64_t n, int64_t m, int64_t k, bool gated, bool fast, bool x_aligned) {
    LinearPlan p = {};
    p.splits = 1;
    p.tile = -1;
    if (!fast || n == 0) return p;
    const int64_t wins = ceil_div(k, kWinElems);
    const auto finish_us = [&](int64_t s) {
        return s == 1 ? 0.0f : kFinishUs + static_cast<float>(s * n * m) * (gated ? 16.0f : 8.0f) / kFinishBytesPerUs;
    };
    p.stream = true;
    p.strips = ceil_div(m, kTile);
    p.blocks = ceil_div(n, kStreamTokens);
    float best = 0.0f;
    for (int64_t s = 1; s <= kMaxStreamSplits && (s == 1 || wins >= s * kStreamWaves); s *= 2) {
        const float us = rounds_us(kStreamUs[n > kStreamOnlyTokens][gated], p.strips * p.blocks * s, ceil_div(wins, s)) +
                         finish_us(s);
        if (s > 1 && us >= best) continue;
        best = us;
        p.splits = s;
    }
    p.waves = p.strips * p.blocks * p.splits >= 2 * kComputeUnits ? kStreamWavesMany : kStreamWaves;
    if (n > kStreamOnlyTokens) {
        const int kinds = gated ? kNumGatedTileKinds : kNumTileKinds;
        for (int i = 0; i < kinds; ++i) {
            const TileKind &t = gated ? kGatedTileKinds[i] : kTileKinds[i];
            const int64_t strips = ceil_div(m, t.rows()), blocks = ceil_div(n, t.tokens());
            for (int64_t s = 1; s <= kMaxSplits && s <= wins; s *= 2) {
                const float us = rounds_us(t.us, strips * blocks * s, ceil_div(wins, s)) + finish_us(s);
                if (us >= best) continue;
                best = us;
                p.stream = false;
                p.tile = i;
                p.strips = strips;
                p.blocks = blocks;
                p.splits = s;
            }
        }
    }
    if (p.splits > 1)
        p.part_bytes = static_cast<size_t>(p.splits) * n * m * (gated ? 2 : 1) * sizeof(float);
    if (!x_aligned && !p.stream) p.x_bytes = static_cast<size_t>(n) * k * 2;
    return p;
}

// ---------------------------------------------------------------- MoE
// Workspace of one MoE call, in bytes from its start.  The sizes go by the
// larger (fp32 output) number of planes of h, so they do not depend on it.
struct MoeWorkspace {
    size_t logits;    // double [route_splits][tokens][experts]
    size_t offsets;   // int32 [experts + 1]: first slot of every expert
    size_t choice;    // int32 [slots]: expert of every slot (slot = token * topk + j)
    size_t list;      // int32 [slots]: slots sorted by expert
    size_t active;    // int32 [moe_groups]: experts that have slots, then -1
    size_t weights;   // float [slots]
    size_t h;         // bf16 [planes][slots][inter]
    size_t part;      // float [slots][hidden]
    size_t total;
};

constexpr int kMaxPlanes = 3;
constexpr int64_t kMaxStreamBytes = kReach;       // of the rows that the stream kernel picks its tokens from

// Most experts that can have slots.
inline int64_t moe_groups(const nvfp4_moe_layer_t &l, int64_t tokens) {
    return tokens * l.topk < l.experts ? tokens * l.topk : l.experts;
}

// Whether the workgroups of `tiles` row tiles each would leave compute units with
// less than two: then every tile has its own.
inline bool few_workgroups(int64_t rows, int tiles, int64_t groups) {
    return ceil_div(rows, tiles * kTile) * groups < 2 * kComputeUnits;
}

// Workgroups that share an expert's slots, `each` of the call's workgroups taking
// `tokens_each` of them at a time: as many as twice the average number of slots
// needs, as long as the call stays within four workgroups per compute unit (44
// tokens on all 6 experts of 384 x 192: 48 -> 32 us).
inline int32_t slot_passes(int64_t tokens, int64_t topk, int64_t groups, int64_t tokens_each, int64_t each) {
    const int64_t twice = ceil_div(2 * tokens * topk, groups);
    const int64_t need = ceil_div(twice < tokens ? twice : tokens, tokens_each), room = 4 * kComputeUnits / each;
    return static_cast<int32_t>(need < room ? need : room < 1 ? 1 : room);
}

// Whether slots are taken one by one rather than by expert.  An expert that
// several slots share is then read for each, mostly from the caches, at 0.2 us
// per MB (7168 x 2048, 8 of 64 experts: 2 tokens 42 MB, 3 tokens 92 MB, 4 tokens
// 158 MB; 97, 141 and 177 us against 98, 124 and 150 by expert), and every
// workgroup of the up product chooses its expert itself; what it saves is two
// launches and the partial outputs, about 9 us.
constexpr double kFewSlotsBytes = 40e6;
constexpr int64_t kFewSlotsWorkgroups = 2048;
constexpr int kSlotUpTiles = 1;   // row tiles of gate and of up of a workgroup

inline bool few_slots(const nvfp4_moe_layer_t &l, int64_t tokens) {
    const int64_t slots = tokens * l.topk;
    if (slots * ceil_div(l.inter, kTile) >= kMaxTiles || tokens * (ceil_div(l.hidden, kTile) + 8) >= kMaxTiles / 2)
        return false;
    if (tokens == 1) return true;
    double idle = 1.0;   // chance that an expert has no slot, for independent choices
    for (int64_t i = 0; i < tokens && idle > 1e-6; ++i)
        idle *= 1.0 - static_cast<double>(l.topk) / static_cast<double>(l.experts);
    const double again = static_cast<double>(slots) - static_cast<double>(l.experts) * (1.0 - idle);
    return slots * ceil_div(l.inter, kSlotUpTiles * kTile) <= kFewSlotsWorkgroups &&
           again * static_cast<double>(l.hidden) * static_cast<double>(l.inter) * 27.0 / 16.0 <= kFewSlotsBytes;
}

// Whether, with few slots, every workgroup of the up product computes its token's
// logits itself: 8 or fewer 16-byte loads a thread, 1 to 2 us, instead of a
// kernel of 4 (7 tokens, 3 of 11 experts, 1040 x 336: 22.0 -> 19.7 us; 1 token, 2 of 6, 256 x 96:
// 15.4 -> 12.3).
constexpr int64_t kSmallRouter = 16384;
inline bool small_router(const nvfp4_moe_layer_t &l) { return l.experts * l.hidden <= kSmallRouter; }

// Parts of hidden that the logits are summed in: 512 elements each, while that
// makes no more workgroups than there are compute units.
inline int64_t route_splits(const nvfp4_moe_layer_t &l, int64_t tokens) {
    const int64_t tiles = ceil_div(l.experts, kTile) * ceil_div(tokens, kTile);
    const int64_t most = kComputeUnits / tiles, want = ceil_div(l.hidden, 512);
    return most < 1 ? 1 : want < most ? want : most;
}

inline MoeWorkspace moe_workspace(const nvfp4_moe_layer_t &l, int64_t tokens) {
    const size_t slots = static_cast<size_t>(tokens) * l.topk;
    MoeWorkspace w;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += ws_round(bytes);
        return here;
    };
    w.logits = take(static_cast<size_t>(route_splits(l, tokens)) * tokens * l.experts * 8);
    w.offsets = take(static_cast<size_t>(l.experts + 1) * 4);
    w.choice = take(slots * 4);
    w.list = take(slots * 4);
    w.active = take(static_cast<size_t>(moe_groups(l, tokens)) * 4);
    w.weights = take(slots * 4);
    w.h = take(kMaxPlanes * slots * l.inter * 2);
    w.part = take(slots * l.hidden * 4);
    w.total = at;
    return w;
}

}  // namespace nvfp4ffnplan

#endif  // NVFP4_FFN_PLAN_H
