// Host-side plan of the attention operators on an NVFP4 cache: argument checks,
// kernel choice, grids and workspace layout.
//
// Plain C++17 with no HIP types, so that the same code is compiled into the
// library (nvfp4_attn.hip) and into a host-only check built with g++ and the
// address and undefined-behaviour sanitizers.  Not part of the C ABI.
#ifndef NVFP4_ATTN_PLAN_H
#define NVFP4_ATTN_PLAN_H

#include <climits>
#include <cstddef>
#include <cstdint>

#include "nvfp4_attn.h"

namespace nvfp4attnplan {

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokens = (int64_t(1) << 24) - 1;
constexpr int64_t kMaxHeads = 16384, kMaxKvHeads = 1024, kMaxBatch = 65535;
constexpr int64_t kStepTokens = 64;                // cache tokens of one step of the attention kernels
constexpr int64_t kComputeUnits = 256;             // CUs of an MI355X (8 XCDs x 32)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t padded_dim(int64_t d) { return ceil_div(d, 64) * 64; }
inline bool mul_fits(int64_t a, int64_t b) { return a == 0 || b <= INT64_MAX / a; }

inline int log2_of(int64_t v) {
    int n = 0;
    while ((int64_t(1) << n) < v) ++n;
    return n;
}

inline int check_dims(int64_t kv_heads, int64_t head_dim) {
    return kv_heads < 1 || kv_heads > kMaxKvHeads || head_dim < 16 || head_dim > 256 || head_dim % 16 != 0
               ? NVFP4_GEMV_ERR_BAD_SHAPE
               : NVFP4_GEMV_OK;
}

inline int check_cache_shape(const nvfp4_kv_cache_t &c) {
    if (check_dims(c.kv_heads, c.head_dim) != NVFP4_GEMV_OK || c.page_size < 16 || c.page_size > 1024 ||
        (c.page_size & (c.page_size - 1)) != 0 || c.pages < 1 || c.pages > ((int64_t(1) << 31) - 1) / c.page_size)
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    return NVFP4_GEMV_OK;
}

// Rows of a call that moves them.
inline bool rows_ok(int64_t tokens, int64_t per_token) {
    return tokens >= 0 && tokens <= kMaxTokens && tokens * per_token < (int64_t(1) << 27);
}

// Bytes of each code and scale buffer of a cache whose shape has been checked
// (below 2^31 * 2^10 * 2^7).
inline int64_t code_bytes(const nvfp4_kv_cache_t &c) {
    return c.pages * c.page_size * c.kv_heads * (padded_dim(c.head_dim) / 2);
}
inline int64_t scale_bytes(const nvfp4_kv_cache_t &c) { return code_bytes(c) / 8; }

// tokens x heads rows of `dim` elements.
struct Grid {
    const void *p;
    int64_t token, head;          // strides in elements
    int64_t tokens, heads, dim;
    int bytes;                    // of an element
};

inline int64_t extent(const Grid &g) {   // elements from the first to past the last
    return g.tokens == 0 ? 0 : (g.tokens - 1) * g.token + (g.heads - 1) * g.head + g.dim;
}
inline int check_strides(const Grid &g) {
    if (g.token < 0 || g.head < 0 || g.token > kMaxStride || g.head > kMaxStride) return NVFP4_GEMV_ERR_BAD_SHAPE;
    if (g.tokens > 1 && !mul_fits(g.tokens - 1, g.token)) return NVFP4_GEMV_ERR_BAD_SHAPE;
    const int64_t e = g.tokens > 1 ? (g.tokens - 1) * g.token : 0;
    const int64_t h = (g.heads - 1) * g.head + g.dim;   // at most 2^14 * 2^40
    return e > INT64_MAX / 8 - h ? NVFP4_GEMV_ERR_BAD_SHAPE : NVFP4_GEMV_OK;
}
// Whether no two rows of the grid share an element: heads within a token's stride
// or tokens within a head's.
inline bool rows_apart(const Grid &g) {
    const bool heads_apart = g.heads == 1 || g.head >= g.dim, tokens_apart = g.tokens <= 1 || g.token >= g.dim;
    if (!heads_apart || !tokens_apart) return false;
    return g.heads == 1 || g.tokens <= 1 || g.token >= (g.heads - 1) * g.head + g.dim ||
           g.head >= (g.tokens - 1) * g.token + g.dim;
}
// Whether a row of one may share an element with a row of the other.  Grids of
// the same token stride, each token's rows within it, may lie between each
// other: the parts of one projection's output.
inline bool grids_overlap(const Grid &a, const Grid &b) {
    const int64_t as = extent(a) * a.bytes, bs = extent(b) * b.bytes;
    if (!a.p || !b.p || as <= 0 || bs <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + static_cast<uintptr_t>(bs) || y >= x + static_cast<uintptr_t>(as)) return false;
    const int64_t aw = ((a.heads - 1) * a.head + a.dim) * a.bytes, bw = ((b.heads - 1) * b.head + b.dim) * b.bytes;
    const int64_t at = a.token * a.bytes, bt = b.token * b.bytes;
    if (at != bt || aw > at || bw > bt) return true;
    const uintptr_t stride = static_cast<uintptr_t>(at);
    const uintptr_t apart = y >= x ? (y - x) % stride : (stride - (x - y) % stride) % stride;
    return apart < static_cast<uintptr_t>(aw) || apart + static_cast<uintptr_t>(bw) > stride;
}

inline int64_t span_of(const Grid &g) { return extent(g) * g.bytes; }

// ------------------------------------------------- norms, cache writes and reads
constexpr int kRowThreads = 256;                   // of a workgroup
constexpr int kRowsInFlight = 4;
constexpr int64_t kWavesPerUnit = 16;

// Lanes of a row's group: 8 elements each, a power of two.
inline int row_lanes(int64_t dp) { return dp == 64 ? 8 : dp == 128 ? 16 : 32; }

struct RowPlan {
    int lanes;
    int32_t each;                         // rows of a chunk: those of one kind that a group of lanes takes
    int32_t q_chunks, k_chunks, chunks;   // of a token: queries', keys', all with values'
    int64_t groups;                       // workgroups
};

// The launch of norms and cache writes: `heads` and `kv_heads` rows a token, and with a
// cache as many of values.  Below 2^32 threads for every shape that rows_ok accepts, since
// a chunk holds four rows where heads are many.
inline RowPlan plan_rows(int64_t tokens, int64_t heads, int64_t kv_heads, bool cached, int64_t dp) {
    RowPlan p = {};
    const int parts = cached ? 2 : 1;
    p.lanes = row_lanes(dp);
    // One row a group of lanes until that gives each SIMD its waves, four from there on: the
    // rows of a group come one after the other, but read the cosines once.  Us with one and
    // with four, 32 + 8 heads of 128 rotated: 64 tokens 3.8 and 6.1, 512 tokens 6.2 and 7.3,
    // 1024 tokens 11.5 and 9.8, 2048 tokens 20 and 14.6; with the cache written and read back
    // 7.3 and 11.3, 11.0 and 13.8, 17.6 and 17.8, 29 and 25.  The rule changes at some 400 and
    // 340 tokens, sooner than these figures ask for (up to 2.8 us at 512 tokens).
    p.each = tokens * (heads + parts * kv_heads) * p.lanes / 64 < kComputeUnits * kWavesPerUnit ? 1 : kRowsInFlight;
    p.q_chunks = static_cast<int32_t>(ceil_div(heads, p.each));
    p.k_chunks = static_cast<int32_t>(ceil_div(kv_heads, p.each));
    p.chunks = p.q_chunks + parts * p.k_chunks;
    p.groups = ceil_div(tokens * p.chunks, kRowThreads / p.lanes);
    return p;
}

// Tokens that one launch of the reader takes, 2 kv_heads rows each: whole workgroups of
// fewer than 2^32 threads, which 2^27 - 8 rows of 32 lanes are (2^27 - 7 round up to 2^32).
inline int64_t read_tokens(int64_t kv_heads, int64_t dp) {
    return ((int64_t(1) << 32) / kRowThreads - 1) * (kRowThreads / row_lanes(dp)) / (2 * kv_heads);
}
inline int64_t read_groups(int64_t tokens, int64_t kv_heads, int64_t dp) {
    return ceil_div(tokens * 2 * kv_heads, kRowThreads / row_lanes(dp));
}

// ---------------------------------------------------------------- attention
// Query rows (tokens times heads of one kv head) that a workgroup of the stream
// kernel holds: 16, or 32 where their sums fit the registers of two waves a SIMD; more
// rows take the tile kernel (16 sequences of 32 rows of 128 on 600, 2048 and 8192 tokens:
// 19, 26 and 39 us here, 29, 77 and 61 in tiles).
inline int64_t stream_rows(int64_t dp) { return dp <= 128 ? 32 : 16; }
// Steps of the cache up to which one workgroup takes a sequence and kv head alone: the
// pieces' second launch costs some 2.5 us (32 heads on 8 of 128, one sequence of 512 tokens
// 7.4 us alone, 9.8 in pieces; 64 of them 13.4 and 19.7; one of 1024 tokens 11.2 and 9.8,
// one of 2048 20.8 and 10; 64 of 1024 tokens 20.7 and 27, which the rule does not take).
constexpr int64_t kWholeSteps = 8;

// Workgroups of four waves that a compute unit holds: what the stream kernel's
// registers are kept to (512 a lane of a SIMD, without spills).
constexpr int groups_per_unit(int64_t dp, int64_t rows) {
    return rows <= 16 ? (dp <= 64 ? 5 : dp <= 128 ? 4 : 2) : dp <= 64 ? 3 : 2;
}

// Rows of a workgroup of the tile kernel, 32 a wave: 8 waves decode a step of the cache
// half as often as 4, which fill the chip with half as many rows (prompts of 32 heads on 8
// of 128: 1024 tokens 46 us with 128 rows and 49 with 256, 2048 tokens 82 and 86, 3000
// tokens 122 and 119, 4096 tokens 217 and 180; 256 from 2048 tokens on).
constexpr int64_t kTileRows = 256, kTileRowsFew = 128;
constexpr int64_t kMaxSplits = 64, kFewTiles = 64, kManySteps = 64;

enum AttnKind { kWhole, kShared, kTiled };

struct AttnPlan {
    AttnKind kind;
    int64_t rows;         // query rows of a workgroup
    int64_t groups;       // workgroups
    int64_t pieces;       // kShared: pieces into which the cache's steps are dealt
    int64_t tiles;        // kTiled: bound on the row tiles of all sequences
    int64_t splits;       // kTiled: workgroups that share a tile's steps
    size_t part_bytes, ml_bytes, prefix_bytes;
    size_t ws_bytes() const { return part_bytes + ml_bytes + prefix_bytes; }
};

// max_query: bound on a sequence's queries, max_context on its tokens in the cache.
inline AttnPlan plan_attn(int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t batch, int64_t tokens,
                          int64_t max_query, int64_t max_context) {
    AttnPlan p = {};
    const int64_t dp = padded_dim(head_dim), group = heads / kv_heads, rows = max_query * group;
    const int64_t steps = ceil_div(max_context, kStepTokens);
    p.splits = 1;
    if (rows <= stream_rows(dp)) {
        p.rows = rows <= 16 ? 16 : 32;
        p.kind = steps <= kWholeSteps ? kWhole : kShared;
        p.groups = batch * kv_heads;
        if (p.kind == kShared) {
            // every sequence and kv head ends with a piece that may be short
            p.pieces = groups_per_unit(dp, p.rows) * kComputeUnits;
            p.groups += p.pieces;
            p.part_bytes = static_cast<size_t>(p.groups * p.rows * dp) * 4;
            p.ml_bytes = static_cast<size_t>(p.groups * p.rows * 2) * 4;
            p.prefix_bytes = static_cast<size_t>(batch + 1) * 8;
        }
        return p;
    }
    p.kind = kTiled;
    // tiles of a sequence: ceil(queries * group / rows); over all sequences at most
    const auto bound = [&](int64_t r) {
        const int64_t some = tokens * group / r + batch, each = batch * ceil_div(rows, r);
        return some < each ? some : each;
    };
    p.rows = rows > kTileRowsFew && bound(kTileRows) * kv_heads >= kComputeUnits ? kTileRows : kTileRowsFew;
    p.tiles = bound(p.rows);
    const int64_t items = p.tiles * kv_heads, fill = 2 * kComputeUnits * kTileRowsFew / p.rows;
    // A tile's steps are shared out where tiles are few; a second launch joins the parts, which
    // costs the more the more tiles there are.  Us in parts that fill the chip and in one, a
    // chunk of a prompt, 32 heads on 8 of 128: 32 items 30 and 44 on 1024 tokens, 39 and 144 on
    // 4096; 128 items 53 and 78 on 2048, 117 and 282 on 8192; 232 items 87 and 81 on 2048, 222
    // and 283 on 8192; 384 items 95 and 82 on 2048, 578 and 685 on 16384; 291 items of ragged
    // prompts (1501 tokens, window 500) 53 and 45 in two parts each.  The thresholds keep one
    // part in some cases where parts would pay: 64 to 255 items of up to 64 steps (128 items on
    // 4096 tokens 73 and 146), and from 256 items on long tables (256 on 8192: 199 and 281).
    if (steps > kWholeSteps && (items < kFewTiles || (items < kComputeUnits && steps > kManySteps))) {
        p.splits = ceil_div(fill, items);
        if (p.splits > ceil_div(steps, kWholeSteps)) p.splits = ceil_div(steps, kWholeSteps);
        if (p.splits > kMaxSplits) p.splits = kMaxSplits;
    }
    p.groups = items * p.splits;
    if (p.splits > 1) p.part_bytes = static_cast<size_t>(p.groups * p.rows * (dp + 2)) * 4;
    return p;
}

inline int check_attn_shape(const nvfp4_kv_cache_t &c, int64_t heads, int64_t batch, int64_t tokens,
                            int64_t max_query, int64_t table_width) {
    if (check_cache_shape(c) != NVFP4_GEMV_OK || heads < c.kv_heads || heads > kMaxHeads ||
        heads % c.kv_heads != 0 || tokens < 0 || tokens > kMaxTokens || tokens * heads >= (int64_t(1) << 30) ||
        batch < 1 || batch > kMaxBatch || batch * c.kv_heads > (int64_t(1) << 18) || max_query < 1 ||
        (tokens > 0 && max_query > tokens) || table_width < 1 ||
        table_width > ((int64_t(1) << 31) - 1) / c.page_size)
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    return NVFP4_GEMV_OK;
}

}  // namespace nvfp4attnplan

#endif  // NVFP4_ATTN_PLAN_H
