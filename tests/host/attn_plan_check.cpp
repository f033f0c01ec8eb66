// Host-only checks of the plan of the attention operators
// (precision_decode_amd/csrc/attn_plan.h), built with g++ and the address and
// undefined-behaviour sanitizers by tests/test_attn_plan.py.  No GPU and no HIP.
// Random shapes, from tiny to the edges of the shape rules, check that every plan
// describes a launch the kernels can run: rows that a kernel of that size exists
// for, tiles for every sequence however the queries are dealt out, fewer than 2^32
// threads a launch, and a bounded workspace; and that the overlap rules of row
// grids say what a comparison of every element says.
//
// Prints "attn_plan_check ok" and exits 0 when every check holds; otherwise
// prints the failed check and exits 1.
#include <cstdint>
#include <cstdio>
#include <set>

#include "attn_plan.h"

using namespace nvfp4attnplan;

namespace {

int g_failures = 0;

#define CHECK(cond)                                                                   \
    do {                                                                              \
        if (!(cond)) {                                                                \
            std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);             \
            ++g_failures;                                                             \
        }                                                                             \
    } while (0)

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next() {   // splitmix64
    uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
int64_t pick(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(next() % uint64_t(hi - lo + 1)); }
// logarithmically spread
int64_t dim(int64_t hi) {
    const int bits = 63 - __builtin_clzll(static_cast<uint64_t>(hi));
    const int64_t top = int64_t(1) << pick(0, bits);
    return pick(1, top < hi ? 2 * top - 1 < hi ? 2 * top - 1 : hi : hi);
}

constexpr int64_t kThreads = int64_t(1) << 32;
int g_seen[3][4];

void check_shape(const nvfp4_kv_cache_t &c, int64_t heads, int64_t batch, int64_t tokens, int64_t max_query,
                 int64_t width) {
    if (check_attn_shape(c, heads, batch, tokens, max_query, width) != NVFP4_GEMV_OK || tokens == 0) return;
    const int64_t context = width * c.page_size, dp = padded_dim(c.head_dim), group = heads / c.kv_heads;
    const AttnPlan p = plan_attn(heads, c.kv_heads, c.head_dim, batch, tokens, max_query, context);
    CHECK(context < int64_t(1) << 31);
    CHECK(p.groups >= 1);
    if (p.kind != kTiled) {
        CHECK(max_query * group <= p.rows && (p.rows == 16 || (p.rows == 32 && dp <= 128)));
        CHECK(p.groups * 256 < kThreads && batch * c.kv_heads * p.rows * 256 < kThreads);
        if (p.kind == kWhole) {
            CHECK(context <= kWholeSteps * kStepTokens && p.ws_bytes() == 0 && p.groups == batch * c.kv_heads);
        } else {
            CHECK(p.pieces > 0 && p.groups == p.pieces + batch * c.kv_heads);
            CHECK(p.part_bytes == size_t(p.groups * p.rows * dp) * 4 && p.part_bytes % 256 == 0);
            CHECK((p.part_bytes + p.ml_bytes) % 8 == 0 && p.prefix_bytes >= size_t(batch + 1) * 8);
            // the steps of all sequences and heads are counted in 64 bits
            CHECK(mul_fits(batch * c.kv_heads, ceil_div(context, kStepTokens)));
        }
        ++g_seen[p.kind][p.rows / 16];
        return;
    }
    CHECK(p.rows == kTileRows || p.rows == kTileRowsFew);
    CHECK(p.groups == p.tiles * c.kv_heads * p.splits && p.groups * 2 * p.rows < kThreads);
    CHECK(p.splits >= 1 && p.splits <= kMaxSplits && p.splits <= ceil_div(context, kStepTokens));
    CHECK(p.splits == 1 ? p.ws_bytes() == 0 : p.part_bytes == size_t(p.groups * p.rows * (dp + 2)) * 4);
    if (p.splits > 1) CHECK(p.tiles * c.kv_heads * (p.rows / 8) * 256 < kThreads);
    ++g_seen[kTiled][(p.rows == kTileRows) + 2 * (p.splits > 1)];
    // queries dealt out at random, at most max_query a sequence: a tile for each
    if (batch > 64) return;
    int64_t left = tokens, tiles = 0;
    for (int64_t b = 0; b < batch; ++b) {
        int64_t n = pick(0, 3) == 0 ? pick(0, max_query) : max_query;
        if (n > left) n = left;
        left -= n;
        tiles += ceil_div(n * group, p.rows);
    }
    CHECK(tiles <= p.tiles);
}

// Elements of a grid as byte offsets.
std::set<intptr_t> bytes_of(const Grid &g) {
    std::set<intptr_t> s;
    for (int64_t t = 0; t < g.tokens; ++t)
        for (int64_t h = 0; h < g.heads; ++h)
            for (int64_t e = 0; e < g.dim; ++e) {
                const intptr_t at = reinterpret_cast<intptr_t>(g.p) + (t * g.token + h * g.head + e) * g.bytes;
                s.insert(at);
            }
    return s;
}

Grid random_grid() {
    const int64_t dim = pick(1, 4), heads = pick(1, 3), tokens = pick(0, 4);
    return {reinterpret_cast<void *>(1000 + 2 * pick(0, 60)), pick(0, 24), pick(0, 20), tokens, heads, dim, 2};
}

}  // namespace

int main() {
    const int64_t dims[] = {16, 64, 80, 128, 160, 192, 256};
    for (int i = 0; i < 200000; ++i) {
        nvfp4_kv_cache_t c = {};
        c.pages = dim((int64_t(1) << 27) - 1);
        c.page_size = int64_t(1) << pick(4, 10);
        c.kv_heads = dim(kMaxKvHeads);
        c.head_dim = dims[pick(0, 6)];
        const int64_t heads = c.kv_heads * dim(128), batch = dim(kMaxBatch);
        const int64_t tokens = pick(0, 1) ? batch * dim(64) : dim(kMaxTokens), max_query = dim(tokens);
        check_shape(c, heads, batch, tokens, pick(0, 1) ? max_query : ceil_div(tokens, batch),
                    dim((int64_t(1) << 31) / c.page_size));
    }
    CHECK(g_seen[kWhole][1] && g_seen[kWhole][2] && g_seen[kShared][1] && g_seen[kShared][2]);
    for (int i = 0; i < 4; ++i) CHECK(i == 3 || g_seen[kTiled][i]);

    int overlapping = 0, apart = 0;
    for (int i = 0; i < 100000; ++i) {
        Grid a = random_grid(), b = random_grid();
        if (pick(0, 1)) b.token = a.token;
        const std::set<intptr_t> x = bytes_of(a), y = bytes_of(b);
        bool shared = false;
        for (intptr_t v : x) shared |= y.count(v) != 0;
        // an overlap is never missed; grids of one token stride with heads in it are told apart exactly
        if (shared) CHECK(grids_overlap(a, b));
        overlapping += shared;
        apart += !grids_overlap(a, b);
        if (rows_apart(a)) CHECK(int64_t(x.size()) == a.tokens * a.heads * a.dim);
        CHECK(check_strides(a) == NVFP4_GEMV_OK);
    }
    CHECK(overlapping > 1000 && apart > 1000);
    // queries, keys and values of one projection: apart though their ranges interleave
    const Grid q = {reinterpret_cast<void *>(4096), 512, 64, 9, 4, 64, 2};
    const Grid k = {reinterpret_cast<void *>(4096 + 2 * 256), 512, 64, 9, 2, 64, 2};
    CHECK(!grids_overlap(q, k) && !grids_overlap(k, q));
    // strides at their limits do not overflow
    const Grid far = {nullptr, kMaxStride, kMaxStride, kMaxTokens, kMaxHeads, 256, 4};
    if (check_strides(far) == NVFP4_GEMV_OK) CHECK(extent(far) > 0 && span_of(far) > 0);

    if (g_failures) return 1;
    std::printf("attn_plan_check ok\n");
    return 0;
}
