// Host-only checks of the plan of the linear layer and of the MoE layer
// (precision_decode_amd/csrc/ffn_plan.h), built with g++ and the address and
// undefined-behaviour sanitizers by tests/test_host_sanitized.py.  No GPU and
// no HIP.  Random shapes, from tiny to the edges of the shape rules, check that
// every plan describes a launch the kernels can run: all rows and tokens
// covered, K split into at most as many parts as it has windows, fewer than
// 2^32 threads, and no more workspace than the size query reports.
//
// Prints "ffn_plan_check ok" and exits 0 when every check holds; otherwise
// prints the failed check and exits 1.
#include <cstdint>
#include <cstdio>

#include "ffn_plan.h"

using namespace nvfp4ffnplan;

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

int g_seen[8];

void check_linear(int64_t n, int64_t m, int64_t k, bool gated) {
    if (check_linear_shape(n, m, k, NVFP4_W_ROW_MAJOR) != NVFP4_GEMV_OK) return;
    const LinearPlan most = plan_linear(n, m, k, gated, true, false);
    for (int i = 0; i < 4; ++i) {
        const LinearPlan p = plan_linear(n, m, k, gated, i & 1, i & 2);
        CHECK(p.ws_bytes() <= most.ws_bytes());
        CHECK(p.splits >= 1);
        if (!(i & 1)) {
            CHECK(!p.stream && p.tile == -1 && p.ws_bytes() == 0);
            continue;
        }
        if (n == 0) continue;
        int64_t rows, tokens, threads;
        if (p.stream) {
            rows = kTile;
            tokens = n == 1 ? 1 : kStreamTokens;
            threads = p.waves * 64;
            CHECK(p.waves == kStreamWaves || p.waves == kStreamWavesMany);
            ++g_seen[6];
        } else {
            CHECK(p.tile >= 0 && p.tile < (gated ? kNumGatedTileKinds : kNumTileKinds));
            const TileKind &t = gated ? kGatedTileKinds[p.tile] : kTileKinds[p.tile];
            rows = t.rows();
            tokens = t.tokens();
            threads = t.waves() * 64;
            ++g_seen[p.tile];
        }
        CHECK(p.strips * rows >= m && (p.strips - 1) * rows < m);
        CHECK(p.blocks * tokens >= n && (p.blocks - 1) * tokens < n);
        CHECK(p.splits <= ceil_div(k, kWinElems));
        CHECK(p.strips * p.blocks * p.splits * threads < (int64_t(1) << 32));
        CHECK(p.part_bytes == (p.splits > 1 ? size_t(p.splits) * n * m * (gated ? 8 : 4) : 0));
        CHECK(p.x_bytes == ((i & 2) || p.stream ? 0 : size_t(n) * k * 2));
    }
}

void check_moe(const nvfp4_moe_layer_t &l, int64_t tokens) {
    if (check_moe_shape(l, tokens) != NVFP4_GEMV_OK || tokens == 0) return;
    const MoeWorkspace w = moe_workspace(l, tokens);
    const size_t slots = size_t(tokens) * l.topk;
    const int64_t splits = route_splits(l, tokens), groups = moe_groups(l, tokens);
    CHECK(splits >= 1 && (splits - 1) * 32 < l.hidden);
    CHECK(groups >= 1 && groups <= l.experts && groups <= int64_t(slots));
    // the parts follow each other without overlap
    CHECK(w.logits == 0 && w.offsets >= size_t(splits) * tokens * l.experts * 8);
    CHECK(w.choice - w.offsets >= size_t(l.experts + 1) * 4);
    CHECK(w.list - w.choice >= slots * 4);
    CHECK(w.active - w.list >= slots * 4);
    CHECK(w.weights - w.active >= size_t(groups) * 4);
    CHECK(w.h - w.weights >= slots * 4);
    CHECK(w.part - w.h >= kMaxPlanes * slots * l.inter * 2);
    CHECK(w.total - w.part >= slots * l.hidden * 4);
    const int64_t each = ceil_div(l.inter, kTile) * groups;
    const int32_t passes = slot_passes(tokens, l.topk, groups, 16, each);
    CHECK(passes >= 1 && (passes == 1 || passes * each <= 4 * kComputeUnits));
    if (few_slots(l, tokens)) {
        CHECK(int64_t(slots) * ceil_div(l.inter, kSlotUpTiles * kTile) * 256 < (int64_t(1) << 32));
        CHECK(ceil_div(ceil_div(l.hidden, kTile), 8) * 8 * tokens * 512 < (int64_t(1) << 32));
        ++g_seen[7];
    }
}

}  // namespace

int main() {
    for (int i = 0; i < 200000; ++i) {
        const int64_t n = i % 50 == 0 ? 0 : dim(i % 3 ? 8192 : (int64_t(1) << 30));
        check_linear(n, dim(i % 3 ? 16384 : (int64_t(1) << 30)), 16 * dim(i % 7 ? 1024 : kMaxK / 16), next() & 1);
        nvfp4_moe_layer_t l = {};
        l.experts = dim(kMaxExperts);
        l.topk = static_cast<int32_t>(pick(1, l.experts < kMaxTopk ? l.experts : kMaxTopk));
        l.hidden = 16 * dim(i % 5 ? 512 : kMaxK / 16);
        l.inter = 16 * dim(i % 5 ? 512 : kMaxK / 16);
        check_moe(l, dim(i % 4 ? 128 : kMaxTokens));
    }
    for (int seen : g_seen) CHECK(seen > 0);   // every kernel shape, the stream kernel and few slots
    if (g_failures) return 1;
    std::printf("ffn_plan_check ok\n");
    return 0;
}
