// Host-only checks of the plan of the linear layer and of the MoE layer
// (precision_decode_amd/csrc/ffn_plan.h) at the largest sizes that its shape
// rules accept, built with g++ and the address and undefined-behaviour
// sanitizers by tests/test_ffn_limits.py.  No GPU and no HIP.
//
// Prints "ffn_limits_check ok" and exits 0 when every check holds; otherwise
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

// The tokens of a workgroup, with the longest rows as far apart as they may be,
// end within the bytes that the kernels' offsets reach.
void check_reach() {
    for (const TileKind &t : kTileKinds) CHECK(t.tokens() * kMaxK * 2 <= kReach);
    for (const TileKind &t : kGatedTileKinds) CHECK(t.tokens() * kMaxK * 2 <= kReach);
    CHECK(kStreamTokens * kMaxK * 2 <= kReach);
    CHECK(kMaxStreamBytes <= kReach);
    // a plan that takes the largest token block at the longest rows
    const LinearPlan p = plan_linear(256, 8192, kMaxK, false, true, true);
    CHECK(!p.stream && p.tile >= 0 && kTileKinds[p.tile].tokens() == 256);
}

// Rows that share no byte are not refused where their strides agree, and rows that
// share one always are.
void check_overlap() {
    for (int64_t stride = 1; stride <= 9; ++stride)
        for (int64_t other = stride; other <= stride + 1; ++other)
            for (int64_t wa = 1; wa <= stride; ++wa)
                for (int64_t wb = 1; wb <= other; ++wb)
                    for (int64_t rows = 1; rows <= 4; ++rows)
                        for (int64_t at = 0; at <= 80; ++at) {
                            const RowSpan a = {40, (rows - 1) * stride + wa, wa, stride};
                            const RowSpan b = {static_cast<uintptr_t>(at), (rows - 1) * other + wb, wb, other};
                            bool share = false;
                            for (int64_t i = 0; i < rows; ++i)
                                for (int64_t j = 0; j < rows; ++j) {
                                    const int64_t x = 40 + i * stride, y = at + j * other;
                                    share |= x < y + wb && y < x + wa;
                                }
                            const bool said = rows_overlap(a, b);
                            CHECK(said == rows_overlap(b, a));
                            CHECK(said || !share);
                            // column ranges of one matrix, b's in a row of a's or a's in a row of b's
                            const int64_t d = ((at - 40) % stride + stride) % stride;
                            const bool columns = d >= wa && d + wb <= stride;
                            if (stride == other && columns) CHECK(!said);
                            // one row each: exactly
                            if (rows == 1 && (at >= 40 + wa || at + wb <= 40)) CHECK(!said);
                        }
    CHECK(!rows_overlap({40, 0, 4, 8}, {40, 12, 4, 8}));
}

// The copy of X to aligned rows: X of any size that the GPU's memory can hold.
void check_align() {
    const int64_t sizes[][2] = {{1, 16}, {17, 272}, {4096, 7168}, {1 << 22, 16384}, {1 << 15, kMaxK}, {1 << 27, 1024}};
    for (const auto &s : sizes) {
        const int64_t groups = align_groups(s[0], s[1]);
        CHECK(groups >= 1 && groups * kAlignThreads < (int64_t(1) << 32));
        CHECK(groups <= ceil_div(s[0] * (s[1] / 8), kAlignThreads));
    }
}

}  // namespace

int main() {
    check_align();
    check_reach();
    check_overlap();
    if (g_failures) return 1;
    std::printf("ffn_limits_check ok\n");
    return 0;
}
