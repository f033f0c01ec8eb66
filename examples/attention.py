"""The attention half of a decoder block on NVFP4 weights and an NVFP4 cache:

    q, k, v = x Wqkv^T                     one projection, its parts taken as they lie
    q, k normalised per head and rotated, k and v quantised into the cache's pages
    h = x + attention(q, cache) Wo^T       a window and a few first tokens visible

Prompts of different lengths fill the cache in one call; then the step of one token a
sequence is captured into a graph and replayed, its positions, slots and lengths
advancing on the device:

    python examples/attention.py --batch 8 --prompt 1000 --steps 100
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_decode_amd as pd  # noqa: E402


def quantised(rows, k, generator):
    """Packed codes and scales, and the global scale, of a random matrix whose products with
    unit inputs are of unit size."""
    w = (torch.randn((1, rows, k), device="cuda", generator=generator) * k ** -0.5).to(torch.bfloat16)
    codes = torch.empty((1, rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, rows, k // 16), dtype=torch.uint8, device="cuda")
    global_scale = torch.empty(1, dtype=torch.float32, device="cuda")
    pd.nvfp4_quantize_weight(w, 1, rows, k, pd.NVFP4_ROUND_NEAREST_LOWER, codes, scales, global_scale)
    return *pd.pack_weight(codes, scales), global_scale


def rotation(positions, dim, base=10000.0):
    """Cosines, then sines, of every position: float32 (positions, dim)."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2) / dim)
    return torch.cat((angle.cos(), angle.sin()), dim=1).float().cuda()


class Attention:
    def __init__(self, hidden, heads, kv_heads, head_dim, batch, context, page=64, window=0, sinks=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, head_dim
        self.page, self.window, self.sinks, self.batch = page, window, sinks, batch
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.qkv, self.out = quantised(self.rows, hidden, g), quantised(hidden, heads * head_dim, g)
        self.cos_sin = rotation(context, head_dim)
        self.norm = torch.ones(head_dim, device="cuda")
        self.width = -(-context // page)
        # the pages of a sequence lie anywhere: here dealt out in a random order
        self.table = torch.randperm(batch * self.width, device="cuda", generator=g).to(torch.int32).view(batch, -1)
        self.cache = pd.KvCache.empty(batch * self.width, kv_heads, page, head_dim)

    def workspace(self):
        """Bytes of workspace of a step of one token a sequence."""
        n = self.batch
        return max(pd.nvfp4_linear_workspace_size(n, self.rows, self.hidden),
                   pd.nvfp4_linear_workspace_size(n, self.hidden, self.heads * self.dim),
                   pd.nvfp4_kv_attention_workspace_size(self.cache, self.heads, n, n, 1, self.width))

    def slots(self, sequence, positions):
        return self.table[sequence, positions // self.page].long() * self.page + positions % self.page

    def step(self, x, positions, slots, lengths, starts=None):
        """x (tokens, hidden) plus attention; the tokens' keys and values join the cache."""
        codes, scales, alpha = self.qkv
        qkv = pd.linear(x, codes, scales, self.rows, alpha=alpha, packed=True).view(-1, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q, _ = pd.qk_norm_rope(q, k, positions, self.cos_sin, q_weight=self.norm, k_weight=self.norm, q_out=q, v=v,
                               cache=self.cache, slots=slots)
        o = pd.kv_attention(q, self.cache, self.table, lengths, query_starts=starts, window=self.window, sinks=self.sinks)
        codes, scales, alpha = self.out
        return pd.linear(o.view(-1, self.heads * self.dim), codes, scales, self.hidden, alpha=alpha, residual=x, packed=True)


class Decoder:
    """Steps of one token a sequence; positions and lengths advance on the device."""

    def __init__(self, block, lengths):
        self.block = block
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.sequence = torch.arange(block.batch, device="cuda")

    def step(self, x):
        positions = self.lengths.long()
        self.lengths += 1
        return self.block.step(x, positions, self.block.slots(self.sequence, positions), self.lengths)


def prompt_of(batch, longest):
    """Lengths of the prompts: different ones up to the longest."""
    return [max(1, longest - i * longest // (2 * batch)) for i in range(batch)]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args(argv)
    block = Attention(a.hidden, a.heads, a.kv_heads, a.head_dim, a.batch, a.prompt + a.steps + 1, window=a.window,
                      sinks=a.sinks)
    lengths = prompt_of(a.batch, a.prompt)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((sum(lengths), a.hidden), device="cuda", generator=g).to(torch.bfloat16)
    sequence = torch.repeat_interleave(torch.arange(a.batch), torch.tensor(lengths)).cuda()
    positions = torch.cat([torch.arange(n) for n in lengths]).cuda()
    ends = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    y = block.step(x, positions, block.slots(sequence, positions), ends.diff(), ends)
    x = y[ends[1:].long() - 1]

    # eager steps first, then the same ones replayed over the slots that they wrote
    eager, want = Decoder(block, lengths), []
    tokens = x
    for _ in range(a.steps):
        tokens = eager.step(tokens)
        want.append(tokens)
    stream = torch.cuda.Stream()
    pd.nvfp4_workspace_reserve(block.workspace(), stream)
    decoder, tokens = Decoder(block, lengths), x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tokens.copy_(decoder.step(tokens))
    same, spent = True, 0.0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for w in want:
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        spent += start.elapsed_time(end)
        same = same and torch.equal(tokens, w)
    print(f"{a.batch} sequences of up to {a.prompt} tokens, {a.heads} heads on {a.kv_heads} of {a.head_dim}: "
          f"{spent / max(a.steps, 1) * 1e3:.1f} us a step; replay {'equals' if same else 'DIFFERS FROM'} eager")
    return same


if __name__ == "__main__":
    sys.exit(0 if main() else 1)
