// Feed-forward operators on NVFP4 weights for MI355X (gfx950): the linear
// layer with bias, activation and residual in its epilogue, and a whole
// mixture-of-experts layer for a few tokens.
//
// A weight element times its block scale, e2m1 * e4m3, has at most 6
// significant bits (2 times 4, 15 * 3 = 45) and, unless it is 0, lies in 2^-10 ..
// 2688, so it is exact as bf16 and as fp16.  The 16-bit activations therefore meet the 4-bit weights on the
// 16x16x32 matrix-core instructions of their own type without being
// quantised: the VALU decodes weight tiles into operands, the products are
// exact in fp32 and summed there.  The weight tile is the A operand and the
// tokens are the B operand, so a lane ends with four consecutive rows of one
// token, which the epilogue finishes and stores together.
//
// The MoE layer runs as route_logits, the choice of experts, the gate/up product,
// the down product and moe_combine.  Each slot (a token and one of its experts)
// is a column of the expert's products; h = f(gate) up goes through the
// workspace as bf16 planes (the value, the rest of its rounding, ...) that
// the down product multiplies one after another into the same sums.
//
// This file holds the host side (validation, launches, the C-ABI entry
// points); the device code is ffn_kernels.h and the argument checks, kernel
// choice and workspace layout are ffn_plan.h.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "device_common.h"
#include "ffn_kernels.h"
#include "ffn_plan.h"
#include "nvfp4_ffn.h"

namespace {

bool misaligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

struct Span {
    const void *p;
    int64_t n;
};

bool overlaps(Span a, Span b) {
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.n) && y < x + static_cast<uintptr_t>(a.n);
}

RowSpan rows_at(const void *p, int64_t cols, int64_t ld, int bytes, int64_t span) {
    return {reinterpret_cast<uintptr_t>(p), p ? span : 0, cols * bytes, ld * bytes};
}

int run(const void *fn, dim3 grid, int threads, void **args, hipStream_t stream) {
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, stream) == hipSuccess ? NVFP4_GEMV_OK
                                                                                  : NVFP4_GEMV_ERR_LAUNCH;
}

template <typename A>
int run(void (*fn)(A), dim3 grid, int threads, A a, hipStream_t stream) {
    void *args[] = {&a};
    return run(reinterpret_cast<const void *>(fn), grid, threads, args, stream);
}

template <bool BF16, bool PACKED, int G, int P, int MODE>
int launch_simple(const FfnArgs &a, dim3 grid, hipStream_t stream) {
    return run(ffn_simple<BF16, PACKED, G, P, MODE>, grid, kSimpleWaves * kWave, a, stream);
}

// ---------------------------------------------------------------- linear
struct LinearCall {
    const void *X;
    int32_t x_type;
    int64_t ldx;
    const uint8_t *W, *sfW;
    int32_t w_layout;
    const float *alpha, *bias;
    const void *residual;
    int64_t ldr;
    void *Y;
    int32_t y_type;
    int64_t ldy, n, m, k;
    int32_t activation;
    bool gated() const { return (activation & NVFP4_ACT_GATED) != 0; }
};

// The weight, its layout and its scales: pointers' alignment.
int check_weight_alignment(const void *W, const void *sf, int32_t w_layout) {
    if (w_layout == NVFP4_W_PACKED && (misaligned(W, 16) || misaligned(sf, 4)))
        return NVFP4_GEMV_ERR_ALIGNMENT;
    return NVFP4_GEMV_OK;
}

int check_linear(const LinearCall &c) {
    if (!c.X || !c.W || !c.sfW || !c.Y) return NVFP4_GEMV_ERR_NULL_POINTER;
    if (!in_type_known(c.x_type) || !out_type_known(c.y_type) || !layout_known(c.w_layout) ||
        !act_known(c.activation & ~NVFP4_ACT_GATED))
        return NVFP4_GEMV_ERR_BAD_ARGUMENT;
    int s = check_linear_shape(c.n, c.m, c.k, c.w_layout);
    if (s != NVFP4_GEMV_OK) return s;
    if (c.ldx < c.k || c.ldx > kMaxK || c.ldy < c.m || c.ldy > kMaxLd ||
        (c.residual && (c.ldr < c.m || c.ldr > kMaxLd)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const int yb = type_bytes(c.y_type);
    if (misaligned(c.X, 2) || misaligned(c.Y, yb) || misaligned(c.residual, yb) ||
        misaligned(c.alpha, 4) || misaligned(c.bias, 4))
        return NVFP4_GEMV_ERR_ALIGNMENT;
    s = check_weight_alignment(c.W, c.sfW, c.w_layout);
    if (s != NVFP4_GEMV_OK) return s;
    const int64_t mats = c.gated() ? 2 : 1;
    int64_t wb, sb, xs, ys, rs = 0;
    if (!weight_bytes(mats, c.m, c.k, c.w_layout, &wb, &sb) || !span_bytes(c.n, c.k, c.ldx, 2, &xs) ||
        !span_bytes(c.n, c.m, c.ldy, yb, &ys) ||
        (c.residual && !span_bytes(c.n, c.m, c.ldr, yb, &rs)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const Span y{c.Y, ys};
    const RowSpan yr = rows_at(c.Y, c.m, c.ldy, yb, ys);
    const bool in_place = c.residual == c.Y && c.ldr == c.ldy;
    if (rows_overlap(yr, rows_at(c.X, c.k, c.ldx, 2, xs)) || overlaps(y, {c.W, wb}) || overlaps(y, {c.sfW, sb}) ||
        overlaps(y, {c.alpha, mats * 4}) || overlaps(y, {c.bias, mats * c.m * 4}) ||
        (!in_place && rows_overlap(yr, rows_at(c.residual, c.m, c.ldr, yb, rs))))
        return NVFP4_GEMV_ERR_ALIAS;
    return NVFP4_GEMV_OK;
}

template <bool BF16, int L, int G, int NX>
int launch_linear_stream(const FfnArgs &a, const LinearPlan &p, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(p.strips * p.blocks * p.splits));
    return p.waves == kStreamWaves
               ? run(ffn_stream<BF16, L, G, 1, kLinear, 1, 2, kStreamWaves, NX>, grid, kStreamWaves * kWave, a, stream)
               : run(ffn_stream<BF16, L, G, 1, kLinear, 1, 2, kStreamWavesMany, NX>, grid, kStreamWavesMany * kWave, a,
                     stream);
}

template <bool BF16, int L, int G, int KIND>
int launch_tile(const FfnArgs &a, const LinearPlan &p, hipStream_t stream) {
    constexpr TileKind t = G == 2 ? kGatedTileKinds[KIND % kNumGatedTileKinds] : kTileKinds[KIND];
    return run(ffn_tile<BF16, L, G, t.q, t.nt, t.wm, t.wk>,
               dim3(static_cast<uint32_t>(p.strips * p.blocks * p.splits)), t.waves() * kWave, a, stream);
}

template <bool BF16, int L, int G>
int launch_linear(const FfnArgs &a, const LinearPlan &p, hipStream_t stream) {
    if (p.stream)
        return a.n == 1   ? launch_linear_stream<BF16, L, G, 0>(a, p, stream)
               : a.n == 2 ? launch_linear_stream<BF16, L, G, 1>(a, p, stream)
               : a.n <= 4 ? launch_linear_stream<BF16, L, G, 2>(a, p, stream)
               : a.n <= 8 ? launch_linear_stream<BF16, L, G, 4>(a, p, stream)
                          : launch_linear_stream<BF16, L, G, 8>(a, p, stream);
    switch (p.tile) {
    case 0: return launch_tile<BF16, L, G, 0>(a, p, stream);
    case 1: return launch_tile<BF16, L, G, 1>(a, p, stream);
    case 2: return launch_tile<BF16, L, G, 2>(a, p, stream);
    case 3: return launch_tile<BF16, L, G, 3>(a, p, stream);
    case 4: return launch_tile<BF16, L, G, 4>(a, p, stream);
    }
    if constexpr (G == 1) return launch_tile<BF16, L, 1, 5>(a, p, stream);
    return NVFP4_GEMV_ERR_LAUNCH;   // the plan has no such shape
}

// Layout of a weight for the fast kernels, or kNoLayout for the simple one.
constexpr int kNoLayout = -1;
int layout_of(const void *W, const void *sf, int64_t k, int32_t w_layout) {
    if (w_layout == NVFP4_W_PACKED) return kPackedTiles;
    if (k % 64 == 0 && !misaligned(W, 16) && !misaligned(sf, 4)) return kRows;
    return misaligned(W, 4) ? kNoLayout : kRows16;
}

template <bool BF16, int G>
int launch_linear(const FfnArgs &a, const LinearPlan &p, int layout, hipStream_t stream) {
    switch (layout) {
    case kRows: return launch_linear<BF16, kRows, G>(a, p, stream);
    case kPackedTiles: return launch_linear<BF16, kPackedTiles, G>(a, p, stream);
    case kRows16: return launch_linear<BF16, kRows16, G>(a, p, stream);
    }
    return launch_simple<BF16, false, G, 1, kLinear>(
        a, dim3(static_cast<uint32_t>(ceil_div(a.m, kTile) * ceil_div(a.n, kTile))), stream);
}

bool aligned_rows(const void *X, int64_t ldx) { return !misaligned(X, 16) && ldx % 8 == 0; }

int copy_aligned(const void *X, int64_t ldx, void *to, int64_t rows, int64_t k, hipStream_t stream) {
    const uint16_t *x = static_cast<const uint16_t *>(X);
    uint16_t *y = static_cast<uint16_t *>(to);
    void *args[] = {&x, &ldx, &y, &rows, &k};
    return run(reinterpret_cast<const void *>(align_rows),
               dim3(static_cast<uint32_t>(align_groups(rows, k))), kAlignThreads, args, stream);
}

LinearPlan plan_of(const LinearCall &c) {
    return plan_linear(c.n, c.m, c.k, c.gated(), layout_of(c.W, c.sfW, c.k, c.w_layout) != kNoLayout,
                       aligned_rows(c.X, c.ldx));
}

int linear(const LinearCall &c, const LinearPlan &p, uint8_t *ws, hipStream_t stream) {
    if (c.n == 0) return NVFP4_GEMV_OK;
    FfnArgs a = {};
    a.X = static_cast<const uint8_t *>(c.X);
    a.ldx = c.ldx;
    if (p.x_bytes > 0) {
        uint8_t *x = ws + ws_round(p.part_bytes);
        const int s = copy_aligned(c.X, c.ldx, x, c.n, c.k, stream);
        if (s != NVFP4_GEMV_OK) return s;
        a.X = x;
        a.ldx = c.k;
    }
    a.W = c.W;
    a.sW = c.sfW;
    a.alpha = c.alpha;
    a.bias = c.bias;
    a.residual = c.residual;
    a.ldr = c.ldr;
    a.Y = c.Y;
    a.ldy = c.ldy;
    a.n = c.n;
    a.m = c.m;
    a.k = c.k;
    a.topk = 1;
    a.act = c.activation & ~NVFP4_ACT_GATED;
    a.y_type = c.y_type;
    a.splits = static_cast<int32_t>(p.splits);
    a.part = p.part_bytes > 0 ? reinterpret_cast<float *>(ws) : nullptr;
    const int layout = layout_of(c.W, c.sfW, c.k, c.w_layout);
    const int s = c.x_type == NVFP4_OUT_BF16
                      ? c.gated() ? launch_linear<true, 2>(a, p, layout, stream) : launch_linear<true, 1>(a, p, layout, stream)
                  : c.gated() ? launch_linear<false, 2>(a, p, layout, stream) : launch_linear<false, 1>(a, p, layout, stream);
    if (s != NVFP4_GEMV_OK || !a.part) return s;
    const dim3 grid(static_cast<uint32_t>(ceil_div(c.n * ceil_div(c.m, 4), kFinishThreads)));
    return c.gated() ? run(linear_finish<2>, grid, kFinishThreads, a, stream)
                     : run(linear_finish<1>, grid, kFinishThreads, a, stream);
}

// ---------------------------------------------------------------- MoE
struct MoeCall {
    const nvfp4_moe_layer_t *layer;
    const void *X;
    int64_t ldx;
    const void *residual;
    int64_t ldr;
    void *Y;
    int32_t y_type;
    int64_t ldy, tokens;
};

int check_moe(const MoeCall &c) {
    if (!c.layer || !c.X || !c.Y) return NVFP4_GEMV_ERR_NULL_POINTER;
    const nvfp4_moe_layer_t &l = *c.layer;
    if (!l.router || !l.W13 || !l.sf13 || !l.W2 || !l.sf2) return NVFP4_GEMV_ERR_NULL_POINTER;
    if (!in_type_known(l.x_type) || !out_type_known(c.y_type) || !layout_known(l.w_layout) ||
        !act_known(l.activation) || l.scoring < NVFP4_SCORE_SOFTMAX || l.scoring > NVFP4_SCORE_SIGMOID ||
        l.renormalize < 0 || l.renormalize > 1 || l.reserved != 0)
        return NVFP4_GEMV_ERR_BAD_ARGUMENT;
    int s = check_moe_shape(l, c.tokens);
    if (s != NVFP4_GEMV_OK) return s;
    if (c.ldx < l.hidden || c.ldx > kMaxK || c.ldy < l.hidden || c.ldy > kMaxLd ||
        (c.residual && (c.ldr < l.hidden || c.ldr > kMaxLd)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const int yb = type_bytes(c.y_type);
    if (misaligned(c.X, 2) || misaligned(l.router, 2) || misaligned(c.Y, yb) ||
        misaligned(c.residual, yb) || misaligned(l.route_bias, 4) || misaligned(l.alpha13, 4) ||
        misaligned(l.alpha2, 4))
        return NVFP4_GEMV_ERR_ALIGNMENT;
    s = check_weight_alignment(l.W13, l.sf13, l.w_layout);
    if (s == NVFP4_GEMV_OK) s = check_weight_alignment(l.W2, l.sf2, l.w_layout);
    if (s != NVFP4_GEMV_OK) return s;
    int64_t w13, s13, w2, s2, xs, ys, rs = 0;
    if (!weight_bytes(2 * l.experts, l.inter, l.hidden, l.w_layout, &w13, &s13) ||
        !weight_bytes(l.experts, l.hidden, l.inter, l.w_layout, &w2, &s2) ||
        !span_bytes(c.tokens, l.hidden, c.ldx, 2, &xs) || !span_bytes(c.tokens, l.hidden, c.ldy, yb, &ys) ||
        (c.residual && !span_bytes(c.tokens, l.hidden, c.ldr, yb, &rs)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const Span y{c.Y, ys};
    const RowSpan yr = rows_at(c.Y, l.hidden, c.ldy, yb, ys);
    const bool in_place = c.residual == c.Y && c.ldr == c.ldy;
    if (rows_overlap(yr, rows_at(c.X, l.hidden, c.ldx, 2, xs)) || overlaps(y, {l.router, l.experts * l.hidden * 2}) ||
        overlaps(y, {l.route_bias, l.experts * 4}) || overlaps(y, {l.W13, w13}) ||
        overlaps(y, {l.sf13, s13}) || overlaps(y, {l.W2, w2}) || overlaps(y, {l.sf2, s2}) ||
        overlaps(y, {l.alpha13, l.experts * 8}) || overlaps(y, {l.alpha2, l.experts * 4}) ||
        (!in_place && rows_overlap(yr, rows_at(c.residual, l.hidden, c.ldr, yb, rs))))
        return NVFP4_GEMV_ERR_ALIAS;
    return NVFP4_GEMV_OK;
}

constexpr int kUpTiles = 2, kUpWaves = 4, kDownTiles = 4, kDownWaves = 2, kDownFewWaves = 4;

// The experts' products, in workgroups of R row tiles and W waves.  Many row
// tiles per workgroup read and stage the tokens less often; where they would
// leave compute units idle, a workgroup takes one.
template <bool BF16, int L, int R, int W>
int stream_up(FfnArgs a, int64_t groups, hipStream_t stream) {
    constexpr int NX = 8;
    const int64_t each = ceil_div(a.m, R * kTile) * groups;
    a.passes = slot_passes(a.n, a.topk, groups, 2 * NX, each);
    return run(ffn_stream<BF16, L, 2, 1, kMoeUp, R, 2, W, NX>, dim3(static_cast<uint32_t>(each * a.passes)), W * kWave, a,
               stream);
}
template <bool BF16, int L>
int stream_up(const FfnArgs &a, int64_t groups, hipStream_t stream) {
    return few_workgroups(a.m, kUpTiles, groups) ? stream_up<BF16, L, 1, kUpWaves>(a, groups, stream)
                                                 : stream_up<BF16, L, kUpTiles, kUpWaves>(a, groups, stream);
}

template <int L, int P, int R, int W>
int stream_down(FfnArgs a, int64_t groups, hipStream_t stream) {
    constexpr int NX = 4;
    const int64_t each = ceil_div(a.m, R * kTile) * groups;
    a.passes = slot_passes(a.n, a.topk, groups, 2 * NX, each);
    return run(ffn_stream<true, L, 1, P, kMoeDown, R, 2, W, NX>, dim3(static_cast<uint32_t>(each * a.passes)), W * kWave, a,
               stream);
}
template <int L, int P>
int stream_down(const FfnArgs &a, int64_t groups, hipStream_t stream) {
    return few_workgroups(a.m, kDownTiles, groups) ? stream_down<L, P, 1, kDownFewWaves>(a, groups, stream)
                                                   : stream_down<L, P, kDownTiles, kDownWaves>(a, groups, stream);
}

template <bool BF16>
int launch_up(const FfnArgs &a, int layout, bool packed, int64_t groups, hipStream_t stream) {
    switch (layout) {
    case kRows: return stream_up<BF16, kRows>(a, groups, stream);
    case kPackedTiles: return stream_up<BF16, kPackedTiles>(a, groups, stream);
    case kRows16: return stream_up<BF16, kRows16>(a, groups, stream);
    }
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.m, kTile) * groups));
    return packed ? launch_simple<BF16, true, 2, 1, kMoeUp>(a, grid, stream)
                  : launch_simple<BF16, false, 2, 1, kMoeUp>(a, grid, stream);
}

template <int P>
int launch_down(const FfnArgs &a, int layout, bool packed, int64_t groups, hipStream_t stream) {
    switch (layout) {
    case kRows: return stream_down<kRows, P>(a, groups, stream);
    case kPackedTiles: return stream_down<kPackedTiles, P>(a, groups, stream);
    case kRows16: return stream_down<kRows16, P>(a, groups, stream);
    }
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.m, kTile) * groups));
    return packed ? launch_simple<true, true, 1, P, kMoeDown>(a, grid, stream)
                  : launch_simple<true, false, 1, P, kMoeDown>(a, grid, stream);
}

template <int L>
int launch_slot_up(const SlotArgs &s, bool bf16, int64_t slots, hipStream_t stream) {
    return run(bf16 ? ffn_slot_up<true, L> : ffn_slot_up<false, L>,
               dim3(static_cast<uint32_t>(ceil_div(s.f.m, kSlotUpTiles * kTile) * slots)), kSlotUpWaves * kWave, s, stream);
}

template <int L>
int launch_slot_down(const SlotArgs &s, const CombineArgs &y, int planes, hipStream_t stream) {
    void *args[] = {const_cast<SlotArgs *>(&s), const_cast<CombineArgs *>(&y)};
    const void *fn = planes == 2 ? reinterpret_cast<const void *>(ffn_slot_down<L, 2>)
                                 : reinterpret_cast<const void *>(ffn_slot_down<L, 3>);
    const int64_t strips = ceil_div(ceil_div(s.f.m, kTile), kXcds) * kXcds;
    return run(fn, dim3(static_cast<uint32_t>(strips * y.tokens)), kSlotWaves * kWave, args, stream);
}

int moe(const MoeCall &c, uint8_t *ws, hipStream_t stream) {
    if (c.tokens == 0) return NVFP4_GEMV_OK;
    const nvfp4_moe_layer_t &l = *c.layer;
    const MoeWorkspace w = moe_workspace(l, c.tokens);
    const bool bf16 = l.x_type == NVFP4_OUT_BF16, packed = l.w_layout == NVFP4_W_PACKED;
    const int64_t slots = c.tokens * l.topk;

    RouteArgs r = {};
    r.X = static_cast<const uint8_t *>(c.X);
    r.ldx = c.ldx;
    r.router = static_cast<const uint8_t *>(l.router);
    r.route_bias = l.route_bias;
    r.logits = reinterpret_cast<double *>(ws + w.logits);
    r.offsets = reinterpret_cast<int32_t *>(ws + w.offsets);
    r.choice = reinterpret_cast<int32_t *>(ws + w.choice);
    r.list = reinterpret_cast<int32_t *>(ws + w.list);
    r.active = reinterpret_cast<int32_t *>(ws + w.active);
    r.groups = static_cast<int32_t>(moe_groups(l, c.tokens));
    r.weights = reinterpret_cast<float *>(ws + w.weights);
    r.tokens = c.tokens;
    r.experts = l.experts;
    r.hidden = l.hidden;
    r.topk = l.topk;
    r.splits = static_cast<int32_t>(route_splits(l, c.tokens));
    r.scoring = l.scoring;
    r.renormalize = l.renormalize;
    r.routed_scale = l.routed_scale;
    const int planes = c.y_type == NVFP4_OUT_F32 ? 3 : 2;
    FfnArgs up = {};
    up.splits = 1;
    up.X = r.X;
    up.ldx = c.ldx;
    int up_layout = layout_of(l.W13, l.sf13, l.hidden, l.w_layout);
    if (c.tokens * up.ldx * 2 >= kMaxStreamBytes) up_layout = kNoLayout;
    const int down_layout = slots * l.inter * 2 < kMaxStreamBytes ? layout_of(l.W2, l.sf2, l.inter, l.w_layout) : kNoLayout;
    up.plane = slots * l.inter;
    up.W = l.W13;
    up.sW = l.sf13;
    up.alpha = l.alpha13;
    up.Y = ws + w.h;
    up.ldy = l.inter;
    up.offsets = r.offsets;
    up.list = r.list;
    up.active = r.active;
    up.n = c.tokens;
    up.m = l.inter;
    up.k = l.hidden;
    up.topk = l.topk;
    up.act = l.activation;
    up.y_planes = planes;

    FfnArgs down = up;
    down.X = ws + w.h;
    down.ldx = l.inter;
    down.W = l.W2;
    down.sW = l.sf2;
    down.alpha = l.alpha2;
    down.Y = ws + w.part;
    down.ldy = l.hidden;
    down.m = l.hidden;
    down.k = l.inter;

    CombineArgs y = {};
    y.part = reinterpret_cast<const float *>(ws + w.part);
    y.weights = r.weights;
    y.residual = c.residual;
    y.ldr = c.ldr;
    y.Y = c.Y;
    y.ldy = c.ldy;
    y.tokens = c.tokens;
    y.hidden = l.hidden;
    y.topk = l.topk;
    y.y_type = c.y_type;

    const bool few = few_slots(l, c.tokens) && up_layout != kNoLayout && down_layout != kNoLayout;
    int s = NVFP4_GEMV_OK;
    if (few && small_router(l)) {
        r.splits = 0;
    } else {
        const dim3 grid(static_cast<uint32_t>(ceil_div(l.experts, kTile) * r.splits),
                        static_cast<uint32_t>(ceil_div(c.tokens, kTile)));
        s = run(bf16 ? route_logits<true> : route_logits<false>, grid, kRouteWaves * kWave, r, stream);
        if (s != NVFP4_GEMV_OK) return s;
    }
    if (few) {
        const SlotArgs u = {up, r}, d = {down, r};
        s = up_layout == kRows          ? launch_slot_up<kRows>(u, bf16, slots, stream)
            : up_layout == kPackedTiles ? launch_slot_up<kPackedTiles>(u, bf16, slots, stream)
                                        : launch_slot_up<kRows16>(u, bf16, slots, stream);
        if (s != NVFP4_GEMV_OK) return s;
        return down_layout == kRows          ? launch_slot_down<kRows>(d, y, planes, stream)
               : down_layout == kPackedTiles ? launch_slot_down<kPackedTiles>(d, y, planes, stream)
                                             : launch_slot_down<kRows16>(d, y, planes, stream);
    }

    if (c.tokens <= kSelectWaves) {
        s = run(route_select, dim3(1), kSelectWaves * kWave, r, stream);
    } else {
        s = run(route_choose, dim3(static_cast<uint32_t>(ceil_div(c.tokens, kChooseWaves))), kChooseWaves * kWave, r, stream);
        if (s == NVFP4_GEMV_OK) s = run(route_sort, dim3(1), kSelectWaves * kWave, r, stream);
    }
    if (s == NVFP4_GEMV_OK)
        s = bf16 ? launch_up<true>(up, up_layout, packed, r.groups, stream)
                 : launch_up<false>(up, up_layout, packed, r.groups, stream);
    if (s == NVFP4_GEMV_OK)
        s = planes == 2 ? launch_down<2>(down, down_layout, packed, r.groups, stream)
                        : launch_down<3>(down, down_layout, packed, r.groups, stream);
    if (s != NVFP4_GEMV_OK) return s;
    return run(moe_combine,
               dim3(static_cast<uint32_t>(ceil_div(l.hidden, 4 * kCombineThreads)), static_cast<uint32_t>(c.tokens)),
               kCombineThreads, y, stream);
}

// The library-owned workspace of the stream: nullptr and a status if it
// cannot be had.
int owned_workspace(size_t need, void *stream, void **ws) {
    *ws = nullptr;
    if (need == 0) return NVFP4_GEMV_OK;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) {
        (void)hipGetLastError();
        return NVFP4_GEMV_ERR_DEVICE;
    }
    *ws = nvfp4_stream_workspace(dev, stream, need);
    return *ws ? NVFP4_GEMV_OK : NVFP4_GEMV_ERR_WORKSPACE;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return NVFP4_GEMV_OK;
    if (!ws || bytes < need) return NVFP4_GEMV_ERR_WORKSPACE;
    return misaligned(ws, kWsAlign) ? NVFP4_GEMV_ERR_ALIGNMENT : NVFP4_GEMV_OK;
}

}  // namespace

extern "C" {

size_t nvfp4_linear_workspace_size(int64_t n, int64_t m, int64_t k, int32_t activation) {
    if (check_linear_shape(n, m, k, NVFP4_W_ROW_MAJOR) != NVFP4_GEMV_OK) return 0;
    return plan_linear(n, m, k, (activation & NVFP4_ACT_GATED) != 0, true, false).ws_bytes();
}

int nvfp4_linear_launch_ws(const void *X, int32_t x_type, int64_t ldx, const uint8_t *W,
                           const uint8_t *sfW, int32_t w_layout, const float *alpha, const float *bias,
                           const void *residual, int64_t ldr, void *Y, int32_t y_type, int64_t ldy,
                           int64_t n, int64_t m, int64_t k, int32_t activation, void *workspace,
                           size_t workspace_bytes, void *stream) {
    const LinearCall c = {X, x_type, ldx, W, sfW, w_layout, alpha, bias, residual, ldr,
                          Y, y_type, ldy, n, m, k, activation};
    int s = check_linear(c);
    if (s != NVFP4_GEMV_OK) return s;
    const LinearPlan p = plan_of(c);
    s = check_workspace(workspace, workspace_bytes, p.ws_bytes());
    if (s != NVFP4_GEMV_OK) return s;
    return linear(c, p, static_cast<uint8_t *>(workspace), static_cast<hipStream_t>(stream));
}

int nvfp4_linear_launch(const void *X, int32_t x_type, int64_t ldx, const uint8_t *W,
                        const uint8_t *sfW, int32_t w_layout, const float *alpha, const float *bias,
                        const void *residual, int64_t ldr, void *Y, int32_t y_type, int64_t ldy,
                        int64_t n, int64_t m, int64_t k, int32_t activation, void *stream) {
    const LinearCall c = {X, x_type, ldx, W, sfW, w_layout, alpha, bias, residual, ldr,
                          Y, y_type, ldy, n, m, k, activation};
    int s = check_linear(c);
    if (s != NVFP4_GEMV_OK) return s;
    const LinearPlan p = plan_of(c);
    void *ws;
    s = owned_workspace(p.ws_bytes(), stream, &ws);
    if (s != NVFP4_GEMV_OK) return s;
    return linear(c, p, static_cast<uint8_t *>(ws), static_cast<hipStream_t>(stream));
}

size_t nvfp4_moe_layer_workspace_size(const nvfp4_moe_layer_t *layer, int64_t tokens) {
    if (!layer || !layout_known(layer->w_layout) || check_moe_shape(*layer, tokens) != NVFP4_GEMV_OK) return 0;
    return tokens == 0 ? 0 : moe_workspace(*layer, tokens).total;
}

int nvfp4_moe_layer_launch_ws(const nvfp4_moe_layer_t *layer, const void *X, int64_t ldx,
                              const void *residual, int64_t ldr, void *Y, int32_t y_type, int64_t ldy,
                              int64_t tokens, void *workspace, size_t workspace_bytes, void *stream) {
    const MoeCall c = {layer, X, ldx, residual, ldr, Y, y_type, ldy, tokens};
    int s = check_moe(c);
    if (s != NVFP4_GEMV_OK) return s;
    s = check_workspace(workspace, workspace_bytes, nvfp4_moe_layer_workspace_size(layer, tokens));
    if (s != NVFP4_GEMV_OK) return s;
    return moe(c, static_cast<uint8_t *>(workspace), static_cast<hipStream_t>(stream));
}

int nvfp4_moe_layer_launch(const nvfp4_moe_layer_t *layer, const void *X, int64_t ldx,
                           const void *residual, int64_t ldr, void *Y, int32_t y_type, int64_t ldy,
                           int64_t tokens, void *stream) {
    const MoeCall c = {layer, X, ldx, residual, ldr, Y, y_type, ldy, tokens};
    int s = check_moe(c);
    if (s != NVFP4_GEMV_OK) return s;
    void *ws;
    s = owned_workspace(nvfp4_moe_layer_workspace_size(layer, tokens), stream, &ws);
    if (s != NVFP4_GEMV_OK) return s;
    return moe(c, static_cast<uint8_t *>(ws), static_cast<hipStream_t>(stream));
}

}  // extern "C"
