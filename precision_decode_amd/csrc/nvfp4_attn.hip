// Attention operators on a paged NVFP4 cache for MI355X (gfx950): head norms
// with the position rotation, cache writes and reads, attention.
//
// This file holds the host side (validation, launches, the C-ABI entry points);
// the device code is cache_kernels.h and attn_kernels.h, the argument checks,
// kernel choice and workspace layout are attn_plan.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "attn_kernels.h"
#include "attn_plan.h"
#include "cache_kernels.h"
#include "device_common.h"
#include "nvfp4_attn.h"

namespace {

using namespace nvfp4attn;
using namespace nvfp4attnplan;

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

bool type16(int32_t t) { return t == NVFP4_OUT_F16 || t == NVFP4_OUT_BF16; }
bool rule_known(int32_t r) { return r >= NVFP4_ROUND_HALF_STEP && r <= NVFP4_ROUND_NEAREST_LOWER; }

template <typename... P, typename... A>
int run(void (*fn)(P...), int64_t groups, int threads, hipStream_t stream, A... a) {
    void *args[] = {&a...};
    return hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3(static_cast<uint32_t>(groups)), dim3(threads), args,
                           0, stream) == hipSuccess
               ? NVFP4_GEMV_OK
               : NVFP4_GEMV_ERR_LAUNCH;
}

// ---------------------------------------------------------------- the cache
int check_cache(const nvfp4_kv_cache_t *c) {
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return NVFP4_GEMV_ERR_NULL_POINTER;
    return check_cache_shape(*c);
}

int check_cache_alignment(const nvfp4_kv_cache_t &c) {
    return misaligned(c.k_codes, 16) || misaligned(c.k_scales, 16) || misaligned(c.v_codes, 16) ||
                   misaligned(c.v_scales, 16) || misaligned(c.k_global, 4) || misaligned(c.v_global, 4)
               ? NVFP4_GEMV_ERR_ALIGNMENT
               : NVFP4_GEMV_OK;
}

// Whether the bytes overlap a buffer of the cache (its globals too).
bool overlaps_cache(Span s, const nvfp4_kv_cache_t &c) {
    return overlaps(s, {c.k_codes, code_bytes(c)}) || overlaps(s, {c.v_codes, code_bytes(c)}) ||
           overlaps(s, {c.k_scales, scale_bytes(c)}) || overlaps(s, {c.v_scales, scale_bytes(c)}) ||
           overlaps(s, {c.k_global, c.kv_heads * 4}) || overlaps(s, {c.v_global, c.kv_heads * 4});
}

// Buffers of a cache that is written overlap none of its others.
bool cache_overlaps_itself(const nvfp4_kv_cache_t &c) {
    const Span part[6] = {{c.k_codes, code_bytes(c)},   {c.v_codes, code_bytes(c)},  {c.k_scales, scale_bytes(c)},
                          {c.v_scales, scale_bytes(c)}, {c.k_global, c.kv_heads * 4}, {c.v_global, c.kv_heads * 4}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (overlaps(part[i], part[j])) return true;
    return false;
}

CacheArgs cache_args(const nvfp4_kv_cache_t &c) {
    CacheArgs a = {};
    a.k_codes = c.k_codes;
    a.k_scales = c.k_scales;
    a.v_codes = c.v_codes;
    a.v_scales = c.v_scales;
    a.k_global = c.k_global;
    a.v_global = c.v_global;
    a.slots = c.pages * c.page_size;
    a.page_log2 = log2_of(c.page_size);
    a.kv_heads = static_cast<int32_t>(c.kv_heads);
    a.head_dim = static_cast<int32_t>(c.head_dim);
    a.dp = static_cast<int32_t>(padded_dim(c.head_dim));
    return a;
}

bool wide_rows(const void *p, int64_t token, int64_t head) {
    return !misaligned(p, 16) && token % 8 == 0 && head % 8 == 0;
}

Rows rows_of(const void *p, int64_t token, int64_t head) {
    return {static_cast<const uint16_t *>(p), token, head, wide_rows(p, token, head)};
}

int launch_rows(RowArgs a, int64_t dp, hipStream_t stream) {
    const RowPlan p = plan_rows(a.tokens, a.heads, a.kv_heads, a.slots != nullptr, dp);
    const int lanes = p.lanes;
    const int64_t groups = p.groups;
    a.each = p.each;
    a.q_chunks = p.q_chunks;
    a.k_chunks = p.k_chunks;
    a.chunks = p.chunks;
    if (a.bf16)
        return lanes == 8    ? run(norm_rope_rows<8, true>, groups, kRowThreads, stream, a)
               : lanes == 16 ? run(norm_rope_rows<16, true>, groups, kRowThreads, stream, a)
                             : run(norm_rope_rows<32, true>, groups, kRowThreads, stream, a);
    return lanes == 8    ? run(norm_rope_rows<8, false>, groups, kRowThreads, stream, a)
           : lanes == 16 ? run(norm_rope_rows<16, false>, groups, kRowThreads, stream, a)
                         : run(norm_rope_rows<32, false>, groups, kRowThreads, stream, a);
}

// ---------------------------------------------------------------- attention
struct AttnCall {
    const nvfp4_kv_cache_t *cache;
    const void *Q;
    int64_t q_token, q_head;
    void *out;
    int64_t o_token, o_head, heads;
    int32_t x_type;
    const int32_t *table;
    int64_t table_stride, table_width;
    const int32_t *lengths, *starts;
    int64_t batch, tokens, max_query;
    float scale;
    int64_t window, sinks;
};

int check_attn(const AttnCall &c) {
    int s = check_cache(c.cache);
    if (s != NVFP4_GEMV_OK) return s;
    if (!c.Q || !c.out || !c.table || !c.lengths) return NVFP4_GEMV_ERR_NULL_POINTER;
    if (!type16(c.x_type) || !std::isfinite(c.scale)) return NVFP4_GEMV_ERR_BAD_ARGUMENT;
    s = check_attn_shape(*c.cache, c.heads, c.batch, c.tokens, c.max_query, c.table_width);
    if (s != NVFP4_GEMV_OK) return s;
    if (c.table_stride < 0 || c.table_stride > kMaxStride || c.window < 0 || c.sinks < 0 ||
        (!c.starts && (c.tokens % c.batch != 0 || c.max_query < c.tokens / c.batch)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const Grid q = {c.Q, c.q_token, c.q_head, c.tokens, c.heads, c.cache->head_dim, 2};
    const Grid o = {c.out, c.o_token, c.o_head, c.tokens, c.heads, c.cache->head_dim, 2};
    if (check_strides(q) != NVFP4_GEMV_OK || check_strides(o) != NVFP4_GEMV_OK || !rows_apart(o))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    if (misaligned(c.Q, 2) || misaligned(c.out, 2) || misaligned(c.table, 4) || misaligned(c.lengths, 4) ||
        misaligned(c.starts, 4))
        return NVFP4_GEMV_ERR_ALIGNMENT;
    s = check_cache_alignment(*c.cache);
    if (s != NVFP4_GEMV_OK) return s;
    const Span out = {c.out, span_of(o)};
    if (grids_overlap(o, q) || overlaps_cache(out, *c.cache) ||
        overlaps(out, {c.table, ((c.batch - 1) * c.table_stride + c.table_width) * 4}) ||
        overlaps(out, {c.lengths, c.batch * 4}) || overlaps(out, {c.starts, (c.batch + 1) * 4}))
        return NVFP4_GEMV_ERR_ALIAS;
    return NVFP4_GEMV_OK;
}

AttnPlan plan_of(const AttnCall &c) {
    return plan_attn(c.heads, c.cache->kv_heads, c.cache->head_dim, c.batch, c.tokens, c.max_query,
                     c.table_width * c.cache->page_size);
}

template <int NB, int R>
int launch_stream(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (p.kind == kWhole) return run(attn_whole<NB, R>, p.groups, kAttnThreads, stream, a);
    const int s = run(attn_pieces<NB, R>, p.groups, kAttnThreads, stream, a);
    if (s != NVFP4_GEMV_OK) return s;
    const int rows = 16 * R, most = a.max_query * a.group, used = most < rows ? most : rows;
    return run(attn_join<NB>, static_cast<int64_t>(a.batch) * a.c.kv_heads * used, kAttnThreads, stream, a, rows, used);
}

template <int NB>
int launch_attn(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (p.kind == kTiled) {
        const int tiles = static_cast<int>(p.tiles), splits = static_cast<int>(p.splits), rows = static_cast<int>(p.rows);
        const int s = p.rows == kTileRows ? run(attn_tiles<NB, 8>, p.groups, 8 * kWave, stream, a, tiles, splits)
                                          : run(attn_tiles<NB, 4>, p.groups, 4 * kWave, stream, a, tiles, splits);
        if (s != NVFP4_GEMV_OK || splits == 1) return s;
        return run(attn_join_tiles<NB>, p.tiles * a.c.kv_heads * (rows / kJoinRows), kAttnThreads, stream, a, tiles, splits, rows);
    }
    if (p.rows == 16) return launch_stream<NB, 1>(a, p, stream);
    if constexpr (NB <= 8) return launch_stream<NB, 2>(a, p, stream);
    return NVFP4_GEMV_ERR_LAUNCH;   // the plan has no such shape
}

int attention(const AttnCall &c, const AttnPlan &p, uint8_t *ws, hipStream_t stream) {
    if (c.tokens == 0) return NVFP4_GEMV_OK;
    const int64_t context = c.table_width * c.cache->page_size;
    AttnArgs a = {};
    a.c = cache_args(*c.cache);
    a.q = static_cast<const uint16_t *>(c.Q);
    a.out = static_cast<uint16_t *>(c.out);
    a.q_token = c.q_token;
    a.q_head = c.q_head;
    a.o_token = c.o_token;
    a.o_head = c.o_head;
    a.table = c.table;
    a.lengths = c.lengths;
    a.starts = c.starts;
    a.table_stride = c.table_stride;
    a.pages = static_cast<int32_t>(c.cache->pages);
    a.table_width = static_cast<int32_t>(c.table_width);
    a.batch = static_cast<int32_t>(c.batch);
    a.group = static_cast<int32_t>(c.heads / c.cache->kv_heads);
    a.tokens = static_cast<int32_t>(c.tokens);
    a.max_query = static_cast<int32_t>(c.max_query);
    a.each = static_cast<int32_t>(c.tokens / c.batch);
    a.group_inverse = static_cast<uint32_t>(ceil_div(int64_t(1) << 26, a.group));
    a.window = c.window < context ? static_cast<int32_t>(c.window) : 0;   // a window over everything is none
    a.sinks = static_cast<int32_t>(c.sinks < context ? c.sinks : context);
    a.bf16 = c.x_type == NVFP4_OUT_BF16;
    a.q_wide = wide_rows(c.Q, c.q_token, c.q_head);
    a.o_wide = wide_rows(c.out, c.o_token, c.o_head);
    a.scale = c.scale;
    a.groups = static_cast<int32_t>(p.pieces);
    if (p.part_bytes > 0) {
        a.part = reinterpret_cast<float *>(ws);
        a.ml = reinterpret_cast<float *>(ws + p.part_bytes);
        a.prefix = reinterpret_cast<int64_t *>(ws + p.part_bytes + p.ml_bytes);
    }
    switch (a.c.dp) {
    case 64: return launch_attn<4>(a, p, stream);
    case 128: return launch_attn<8>(a, p, stream);
    case 192: return launch_attn<12>(a, p, stream);
    }
    return launch_attn<16>(a, p, stream);
}

// The library-owned workspace of the stream: nullptr and a status if it cannot be had.
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

}  // namespace

extern "C" {

int nvfp4_kv_write_launch(const nvfp4_kv_cache_t *cache, const void *K, int64_t k_token_stride,
                          int64_t k_head_stride, const void *V, int64_t v_token_stride,
                          int64_t v_head_stride, int32_t x_type, const int64_t *slots, int64_t tokens,
                          int32_t rule, void *stream) {
    if (!slots || !K) return NVFP4_GEMV_ERR_NULL_POINTER;
    return nvfp4_qk_norm_rope_launch(nullptr, 0, 0, nullptr, nullptr, 0, 0, 0, K, k_token_stride, k_head_stride,
                                     nullptr, nullptr, 0, 0, cache ? cache->kv_heads : 1, cache ? cache->head_dim : 16,
                                     x_type, nullptr, nullptr, 0, 0, 0, 0.0f, tokens, cache, V, v_token_stride,
                                     v_head_stride, slots, rule, stream);
}

int nvfp4_qk_norm_rope_launch(const void *Q, int64_t q_token_stride, int64_t q_head_stride,
                              const float *q_weight, void *Q_out, int64_t qo_token_stride,
                              int64_t qo_head_stride, int64_t heads, const void *K,
                              int64_t k_token_stride, int64_t k_head_stride, const float *k_weight,
                              void *K_out, int64_t ko_token_stride, int64_t ko_head_stride,
                              int64_t kv_heads, int64_t head_dim, int32_t x_type,
                              const int64_t *positions, const float *cos_sin, int64_t table_rows,
                              int64_t rot_dim, int32_t interleaved, float eps, int64_t tokens,
                              const nvfp4_kv_cache_t *cache, const void *V, int64_t v_token_stride,
                              int64_t v_head_stride, const int64_t *slots, int32_t rule, void *stream) {
    const bool cached = cache != nullptr || V != nullptr || slots != nullptr;
    if ((heads > 0 && (!Q || !Q_out)) || !K || (rot_dim > 0 && (!positions || !cos_sin)) ||
        (cached ? !cache || !V || !slots : !K_out))
        return NVFP4_GEMV_ERR_NULL_POINTER;
    int s = cached ? check_cache(cache) : NVFP4_GEMV_OK;
    if (s != NVFP4_GEMV_OK) return s;
    if (!type16(x_type) || interleaved < 0 || interleaved > 1 || !rule_known(rule) || (cached && K_out) ||
        !(eps >= 0.0f) || std::isinf(eps))
        return NVFP4_GEMV_ERR_BAD_ARGUMENT;
    if (check_dims(kv_heads, head_dim) != NVFP4_GEMV_OK || heads < 0 || heads > kMaxHeads ||
        !rows_ok(tokens, heads + 2 * kv_heads) || rot_dim < 0 ||
        rot_dim > head_dim || rot_dim % 16 != 0 || (rot_dim > 0 && (table_rows < 1 || table_rows > kMaxStride)) ||
        (cached && (cache->kv_heads != kv_heads || cache->head_dim != head_dim)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    const bool has_q = heads > 0;
    const Grid q = {Q, q_token_stride, q_head_stride, has_q ? tokens : 0, has_q ? heads : 1, head_dim, 2};
    const Grid qo = {Q_out, qo_token_stride, qo_head_stride, has_q ? tokens : 0, has_q ? heads : 1, head_dim, 2};
    const Grid k = {K, k_token_stride, k_head_stride, tokens, kv_heads, head_dim, 2};
    const Grid ko = {K_out, ko_token_stride, ko_head_stride, cached ? 0 : tokens, kv_heads, head_dim, 2};
    const Grid v = {V, v_token_stride, v_head_stride, cached ? tokens : 0, kv_heads, head_dim, 2};
    if (check_strides(k) != NVFP4_GEMV_OK || (has_q && (check_strides(q) != NVFP4_GEMV_OK ||
        check_strides(qo) != NVFP4_GEMV_OK || !rows_apart(qo))) ||
        (cached ? check_strides(v) != NVFP4_GEMV_OK : check_strides(ko) != NVFP4_GEMV_OK || !rows_apart(ko)))
        return NVFP4_GEMV_ERR_BAD_SHAPE;
    if ((has_q && (misaligned(Q, 2) || misaligned(Q_out, 2))) || misaligned(K, 2) || misaligned(K_out, 2) ||
        misaligned(V, 2) || misaligned(q_weight, 16) || misaligned(k_weight, 16) || misaligned(cos_sin, 16) ||
        misaligned(positions, 8) || misaligned(slots, 8))
        return NVFP4_GEMV_ERR_ALIGNMENT;
    if (cached) {
        s = check_cache_alignment(*cache);
        if (s != NVFP4_GEMV_OK) return s;
    }
    // each output against every input but itself in place, and against the other
    const bool q_in_place = Q == Q_out && q_token_stride == qo_token_stride && q_head_stride == qo_head_stride;
    const bool k_in_place = K == K_out && k_token_stride == ko_token_stride && k_head_stride == ko_head_stride;
    if ((!q_in_place && grids_overlap(qo, q)) || (!k_in_place && grids_overlap(ko, k)) || grids_overlap(qo, k) ||
        grids_overlap(ko, q) || grids_overlap(qo, v) || grids_overlap(qo, ko))
        return NVFP4_GEMV_ERR_ALIAS;
    const Span read[] = {{q_weight, head_dim * 4}, {k_weight, head_dim * 4}, {positions, tokens * 8},
                         {cos_sin, table_rows * rot_dim * 4}, {slots, tokens * 8}};
    for (const Span &r : read)
        if (overlaps({Q_out, span_of(qo)}, r) || overlaps({K_out, span_of(ko)}, r) || (cached && overlaps_cache(r, *cache)))
            return NVFP4_GEMV_ERR_ALIAS;
    if (cached && (cache_overlaps_itself(*cache) || overlaps_cache({Q, span_of(q)}, *cache) ||
                   overlaps_cache({Q_out, span_of(qo)}, *cache) || overlaps_cache({K, span_of(k)}, *cache) ||
                   overlaps_cache({V, span_of(v)}, *cache)))
        return NVFP4_GEMV_ERR_ALIAS;
    if (tokens == 0) return NVFP4_GEMV_OK;

    RowArgs a = {};
    a.q = rows_of(Q, q_token_stride, q_head_stride);
    a.k = rows_of(K, k_token_stride, k_head_stride);
    a.v = rows_of(V, v_token_stride, v_head_stride);
    a.q_out = static_cast<uint16_t *>(Q_out);
    a.k_out = static_cast<uint16_t *>(K_out);
    a.qo_token = qo_token_stride;
    a.qo_head = qo_head_stride;
    a.ko_token = ko_token_stride;
    a.ko_head = ko_head_stride;
    a.qo_wide = wide_rows(Q_out, qo_token_stride, qo_head_stride);
    a.ko_wide = wide_rows(K_out, ko_token_stride, ko_head_stride);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.table_rows = table_rows;
    a.tokens = tokens;
    a.heads = static_cast<int32_t>(heads);
    a.kv_heads = static_cast<int32_t>(kv_heads);
    a.head_dim = static_cast<int32_t>(head_dim);
    a.rot_dim = static_cast<int32_t>(rot_dim);
    a.inverse_dim = 1.0f / static_cast<float>(head_dim);
    a.interleaved = interleaved;
    a.bf16 = x_type == NVFP4_OUT_BF16;
    a.rule = rule;
    a.eps = eps;
    if (cached) a.cache = cache_args(*cache);
    a.slots = slots;
    return launch_rows(a, padded_dim(head_dim), static_cast<hipStream_t>(stream));
}

int nvfp4_kv_read_launch(const nvfp4_kv_cache_t *cache, const int64_t *slots, int64_t tokens, void *K,
                         void *V, int32_t y_type, void *stream) {
    int s = check_cache(cache);
    if (s != NVFP4_GEMV_OK) return s;
    if (!slots || !K || !V) return NVFP4_GEMV_ERR_NULL_POINTER;
    if (!type16(y_type) && y_type != NVFP4_OUT_F32) return NVFP4_GEMV_ERR_BAD_ARGUMENT;
    if (!rows_ok(tokens, 2 * cache->kv_heads)) return NVFP4_GEMV_ERR_BAD_SHAPE;
    const int bytes = y_type == NVFP4_OUT_F32 ? 4 : 2;
    if (misaligned(K, bytes) || misaligned(V, bytes) || misaligned(slots, 8)) return NVFP4_GEMV_ERR_ALIGNMENT;
    s = check_cache_alignment(*cache);
    if (s != NVFP4_GEMV_OK) return s;
    const int64_t size = tokens * cache->kv_heads * cache->head_dim * bytes;
    const Span k = {K, size}, v = {V, size}, sl = {slots, tokens * 8};
    if (overlaps(k, v) || overlaps(k, sl) || overlaps(v, sl) || overlaps_cache(k, *cache) || overlaps_cache(v, *cache))
        return NVFP4_GEMV_ERR_ALIAS;
    if (tokens == 0) return NVFP4_GEMV_OK;
    ReadArgs a = {};
    a.cache = cache_args(*cache);
    a.y_type = y_type;
    a.wide = !misaligned(K, 16) && !misaligned(V, 16);
    const int lanes = row_lanes(a.cache.dp);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t most = read_tokens(cache->kv_heads, a.cache.dp), token = cache->kv_heads * cache->head_dim * bytes;
    for (int64_t first = 0; first < tokens && s == NVFP4_GEMV_OK; first += most) {   // one launch but next to 2^27 rows
        a.slots = slots + first;
        a.k = static_cast<uint8_t *>(K) + first * token;
        a.v = static_cast<uint8_t *>(V) + first * token;
        a.tokens = tokens - first < most ? tokens - first : most;
        const int64_t groups = read_groups(a.tokens, cache->kv_heads, a.cache.dp);
        s = lanes == 8    ? run(read_rows<8>, groups, kRowThreads, st, a)
            : lanes == 16 ? run(read_rows<16>, groups, kRowThreads, st, a)
                          : run(read_rows<32>, groups, kRowThreads, st, a);
    }
    return s;
}

size_t nvfp4_kv_attention_workspace_size(const nvfp4_kv_cache_t *cache, int64_t heads, int64_t batch,
                                         int64_t tokens, int64_t max_query, int64_t table_width) {
    if (!cache || check_attn_shape(*cache, heads, batch, tokens, max_query, table_width) != NVFP4_GEMV_OK || tokens == 0)
        return 0;
    return plan_attn(heads, cache->kv_heads, cache->head_dim, batch, tokens, max_query, table_width * cache->page_size)
        .ws_bytes();
}

int nvfp4_kv_attention_launch_ws(const nvfp4_kv_cache_t *cache, const void *Q, int64_t q_token_stride,
                                 int64_t q_head_stride, void *out, int64_t o_token_stride,
                                 int64_t o_head_stride, int64_t heads, int32_t x_type,
                                 const int32_t *block_table, int64_t table_stride, int64_t table_width,
                                 const int32_t *lengths, const int32_t *query_starts, int64_t batch,
                                 int64_t tokens, int64_t max_query, float scale, int64_t window,
                                 int64_t sinks, void *workspace, size_t workspace_bytes, void *stream) {
    const AttnCall c = {cache, Q, q_token_stride, q_head_stride, out, o_token_stride, o_head_stride, heads, x_type,
                        block_table, table_stride, table_width, lengths, query_starts, batch, tokens, max_query,
                        scale, window, sinks};
    const int s = check_attn(c);
    if (s != NVFP4_GEMV_OK) return s;
    const AttnPlan p = plan_of(c);
    if (tokens > 0 && p.ws_bytes() > 0) {
        if (!workspace || workspace_bytes < p.ws_bytes()) return NVFP4_GEMV_ERR_WORKSPACE;
        if (misaligned(workspace, 256)) return NVFP4_GEMV_ERR_ALIGNMENT;
    }
    return attention(c, p, static_cast<uint8_t *>(workspace), static_cast<hipStream_t>(stream));
}

int nvfp4_kv_attention_launch(const nvfp4_kv_cache_t *cache, const void *Q, int64_t q_token_stride,
                              int64_t q_head_stride, void *out, int64_t o_token_stride,
                              int64_t o_head_stride, int64_t heads, int32_t x_type,
                              const int32_t *block_table, int64_t table_stride, int64_t table_width,
                              const int32_t *lengths, const int32_t *query_starts, int64_t batch,
                              int64_t tokens, int64_t max_query, float scale, int64_t window,
                              int64_t sinks, void *stream) {
    const AttnCall c = {cache, Q, q_token_stride, q_head_stride, out, o_token_stride, o_head_stride, heads, x_type,
                        block_table, table_stride, table_width, lengths, query_starts, batch, tokens, max_query,
                        scale, window, sinks};
    int s = check_attn(c);
    if (s != NVFP4_GEMV_OK) return s;
    const AttnPlan p = plan_of(c);
    void *ws;
    s = owned_workspace(tokens > 0 ? p.ws_bytes() : 0, stream, &ws);
    if (s != NVFP4_GEMV_OK) return s;
    return attention(c, p, static_cast<uint8_t *>(ws), static_cast<hipStream_t>(stream));
}

}  // extern "C"
