"""The feed-forward half of a decoder block on NVFP4 weights: the attention's
output projection, added to the residual stream, then a shared gated
feed-forward layer and a mixture-of-experts layer, each added in its epilogue.

    h = x + o Wo^T
    y = h + silu(h Wg^T) * (h Wu^T) Wd^T  +  sum over the chosen experts

Weights are random, quantised on the device and re-laid out once.  The step is
captured into a graph and replayed, as a decode loop would:

    python examples/feed_forward.py --tokens 1
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_decode_amd as pd  # noqa: E402


def quantised(groups, rows, k, generator):
    """Packed codes and scales, and the global scales, of random matrices whose products
    with unit inputs are of unit size."""
    w = torch.randn((groups, rows, k), device="cuda", generator=generator).to(torch.bfloat16)
    w *= k ** -0.5
    codes = torch.empty((groups, rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((groups, rows, k // 16), dtype=torch.uint8, device="cuda")
    global_scale = torch.empty(groups, dtype=torch.float32, device="cuda")
    pd.nvfp4_quantize_weight(w, groups, rows, k, pd.NVFP4_ROUND_NEAREST_LOWER, codes, scales, global_scale)
    return *pd.pack_weight(codes, scales), global_scale


class Block:
    def __init__(self, hidden, inter, experts, topk, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inter = hidden, inter
        self.out = quantised(1, hidden, hidden, g)
        self.gate_up = quantised(2, inter, hidden, g)
        self.down = quantised(1, hidden, inter, g)
        codes13, scales13, alpha13 = quantised(2 * experts, inter, hidden, g)
        codes2, scales2, alpha2 = quantised(experts, hidden, inter, g)
        router = (torch.randn((experts, hidden), device="cuda", generator=g) * hidden ** -0.5).to(torch.bfloat16)
        self.moe = pd.MoeLayer(router, codes13, scales13, codes2, scales2, inter=inter, topk=topk,
                               alpha13=alpha13.view(experts, 2), alpha2=alpha2, packed=True)

    def workspace(self, tokens):
        """Bytes of workspace that the step needs: reserved once for the stream of a captured graph."""
        h, i = self.hidden, self.inter
        return max(pd.nvfp4_linear_workspace_size(tokens, h, h),
                   pd.nvfp4_linear_workspace_size(tokens, i, h, pd.NVFP4_ACT_SILU | pd.NVFP4_ACT_GATED),
                   pd.nvfp4_linear_workspace_size(tokens, h, i),
                   pd.nvfp4_moe_layer_workspace_size(self.moe, tokens))

    def step(self, o, x):
        codes, scales, alpha = self.out
        h = pd.linear(o, codes, scales, self.hidden, alpha=alpha, residual=x, packed=True)
        codes, scales, alpha = self.gate_up
        g = pd.linear(h, codes, scales, self.inter, alpha=alpha, activation="silu", gated=True, packed=True)
        codes, scales, alpha = self.down
        y = pd.linear(g, codes, scales, self.hidden, alpha=alpha, residual=h, packed=True)
        return pd.moe_layer(h, self.moe, residual=y, out=y)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args(argv)
    block = Block(a.hidden, a.inter, a.experts, a.topk)
    o = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    want = block.step(o, x)

    stream = torch.cuda.Stream()
    pd.nvfp4_workspace_reserve(block.workspace(a.tokens), stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y = block.step(o, x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    same = torch.equal(y, want)
    print(f"{a.tokens} token(s), hidden {a.hidden}, {a.topk} of {a.experts} experts of {a.inter}: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a step; replay {'equals' if same else 'DIFFERS FROM'} eager")
    return same


if __name__ == "__main__":
    sys.exit(0 if main() else 1)
