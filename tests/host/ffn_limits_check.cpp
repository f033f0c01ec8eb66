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

}  // namespace

int main() {
    check_reach();
    if (g_failures) return 1;
    std::printf("ffn_limits_check ok\n");
    return 0;
}
