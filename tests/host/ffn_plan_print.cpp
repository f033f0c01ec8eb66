// Reads lines "n m k gated fast x_aligned" and prints for each the plan of the
// linear layer (precision_decode_amd/csrc/ffn_plan.h): "stream WAVES SPLITS",
// "tile ROWSxTOKENS SPLITS" or "simple", and the bytes of X's aligned copy; or
// lines "moe tokens experts topk hidden inter": "few" or "sorted", and whether
// the router is small.  Built by tests/ffn_plans.py; no GPU and no HIP.
#include <cstdio>
#include <cstring>

#include "ffn_plan.h"

using namespace nvfp4ffnplan;

int main() {
    char line[256];
    while (std::fgets(line, sizeof line, stdin)) {
        long long n, m, k, i, t;
        int gated, fast, aligned;
        if (std::sscanf(line, "moe %lld %lld %lld %lld %lld", &n, &m, &t, &k, &i) == 5) {
            nvfp4_moe_layer_t l = {};
            l.experts = m;
            l.topk = static_cast<int32_t>(t);
            l.hidden = k;
            l.inter = i;
            if (check_moe_shape(l, n) != NVFP4_GEMV_OK) return 1;
            std::printf("%s %d\n", few_slots(l, n) ? "few" : "sorted", small_router(l));
            continue;
        }
        if (std::sscanf(line, "%lld %lld %lld %d %d %d", &n, &m, &k, &gated, &fast, &aligned) != 6) return 1;
        if (check_linear_shape(n, m, k, NVFP4_W_ROW_MAJOR) != NVFP4_GEMV_OK) return 1;
        const LinearPlan p = plan_linear(n, m, k, gated, fast, aligned);
        if (p.stream) {
            std::printf("stream %d %lld", p.waves, static_cast<long long>(p.splits));
        } else if (p.tile >= 0) {
            const TileKind &kind = gated ? kGatedTileKinds[p.tile] : kTileKinds[p.tile];
            std::printf("tile %dx%d %lld", kind.rows(), kind.tokens(), static_cast<long long>(p.splits));
        } else {
            std::printf("simple");
        }
        std::printf(" %llu\n", static_cast<unsigned long long>(p.x_bytes));
    }
    return 0;
}
