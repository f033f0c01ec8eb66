// Host-only checks of the launches of norms, cache writes and cache reads
// (precision_decode_amd/csrc/attn_plan.h), built with g++ and the address and
// undefined-behaviour sanitizers by tests/test_attn_rows.py.  No GPU and no HIP.
// For every shape that the calls accept, from tiny to the borders of the rules: fewer
// than 2^32 threads a launch once rounded up to whole workgroups, a row for every
// group of lanes, and reads in parts that cover all tokens.
//
// Prints "attn_rows_check ok" and exits 0 when every check holds; otherwise
// prints the failed check and exits 1.
#include <cstdint>
#include <cstdio>

#include "attn_plan.h"

using namespace nvfp4attnplan;

namespace {

int g_failures = 0;

#define CHECK(cond)                                                                   \
    do {                                                                              \
        if (!(cond) && ++g_failures <= 20)                                            \
            std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);             \
    } while (0)

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next() {   // splitmix64
    uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
int64_t pick(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(next() % uint64_t(hi - lo + 1)); }

constexpr int64_t kThreads = int64_t(1) << 32;

void check_rows(int64_t tokens, int64_t heads, int64_t kv, int64_t dp) {
    if (!rows_ok(tokens, heads + 2 * kv) || tokens == 0) return;
    for (int cached = 0; cached < 2; ++cached) {
        const RowPlan p = plan_rows(tokens, heads, kv, cached != 0, dp);
        CHECK(8 * p.lanes >= dp && kRowThreads % p.lanes == 0 && p.each >= 1 && p.each <= kRowsInFlight);
        CHECK(p.groups * kRowThreads < kThreads && p.groups * (kRowThreads / p.lanes) >= tokens * p.chunks);
        CHECK(p.q_chunks * p.each >= heads && p.k_chunks * p.each >= kv);
        CHECK(p.chunks == p.q_chunks + (1 + cached) * p.k_chunks);
    }
}

void check_read(int64_t tokens, int64_t kv, int64_t dp) {
    if (!rows_ok(tokens, 2 * kv) || tokens == 0) return;
    const int64_t most = read_tokens(kv, dp);
    CHECK(most >= 1);
    int64_t seen = 0, launches = 0;
    for (int64_t first = 0; first < tokens; first += most, ++launches) {
        const int64_t n = tokens - first < most ? tokens - first : most, groups = read_groups(n, kv, dp);
        CHECK(groups * kRowThreads < kThreads && groups * (kRowThreads / row_lanes(dp)) >= n * 2 * kv);
        seen += n;
    }
    CHECK(seen == tokens && launches <= 2);
    if (tokens * 2 * kv <= (int64_t(1) << 27) - 8) CHECK(launches == 1);
}

}  // namespace

int main() {
    const int64_t dps[] = {64, 128, 192, 256};
    for (int i = 0; i < 300000; ++i) {
        const int64_t dp = dps[pick(0, 3)], kv = pick(1, pick(0, 1) ? 8 : kMaxKvHeads);
        const int64_t heads = pick(0, 2) ? kv * pick(0, 16) : 0, rows = heads + 2 * kv;
        const int64_t border = ((int64_t(1) << 27) - 1) / rows, top = border < kMaxTokens ? border : kMaxTokens;
        const int64_t tokens = pick(0, 3) ? pick(1, top) : top - pick(0, 3);
        check_rows(tokens, heads, kv, dp);
        check_read(tokens, kv, dp);
        const int64_t all = ((int64_t(1) << 27) - 1) / (2 * kv);
        check_read(all < kMaxTokens ? all : kMaxTokens, kv, dp);
    }
    // the rows whose workgroups of 256 threads would be 2^32 threads
    check_read(2164802, 31, 256);
    CHECK(read_tokens(31, 256) < 2164802 && read_tokens(31, 128) > 2164802);

    if (g_failures) return 1;
    std::printf("attn_rows_check ok\n");
    return 0;
}
