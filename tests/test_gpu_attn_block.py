"""The attention operators as they are used together: a projection's parts rotated
into the cache, attention over it and the output projection, for ragged prompts and
then token by token, against the oracle's operators; the example that captures the
step; calls on several streams at once and graphs beside each other."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import back, filled, heads_on_device, i32, on_device, queries, tables
from ffn_util import assert_close
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention.py")
    spec = importlib.util.spec_from_file_location("attention_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def numbers(t):
    return t.detach().to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (6, 3, 128)])
def test_prompts_and_tokens_against_the_oracle(example, heads, kv, dim, window, sinks):
    """Each operator's output against the oracle's on what the operator before it gave, so
    that every tolerance is that of one operator; the cache's bytes are compared exactly."""
    batch, hidden, page = 3, 256, 16
    block = example.Attention(hidden, heads, kv, dim, batch, 200, page=page, window=window, sinks=sinks, seed=3)
    rng = np.random.default_rng(5)
    lengths, counts = np.zeros(batch, np.int64), np.array([37, 1, 80])
    cache = back(block.cache)
    table = block.table.cpu().numpy()
    for _ in range(4):
        n = int(counts.sum())
        x = torch.from_numpy(rng.standard_normal((n, hidden))).to(torch.bfloat16).cuda()
        positions = np.concatenate([np.arange(a, a + c) for a, c in zip(lengths, counts)])
        sequence = np.repeat(np.arange(batch), counts)
        lengths = lengths + counts
        starts = np.concatenate(([0], np.cumsum(counts)))
        slots = table[sequence, positions // page].astype(np.int64) * page + positions % page
        dp, ds = (torch.from_numpy(v).cuda() for v in (positions, slots))
        assert torch.equal(block.slots(torch.from_numpy(sequence).cuda(), dp), ds)
        y = block.step(x, dp, ds, i32(lengths), i32(starts))

        codes, scales, alpha = block.qkv
        qkv = pd.linear(x, codes, scales, block.rows, alpha=alpha, packed=True).view(n, heads + 2 * kv, dim)
        q, k, v = (numbers(t) for t in qkv.split((heads, kv, kv), dim=1))
        w, cs = numbers(block.norm), numbers(block.cos_sin)
        parts = qkv.split((heads, kv, kv), dim=1)
        qr, kr = pd.qk_norm_rope(parts[0], parts[1], dp, block.cos_sin, q_weight=block.norm, k_weight=block.norm)
        for got, of in ((qr, q), (kr, k)):
            want, err = oa.norm_rope(of, w, positions, cs, 1e-6, False)
            assert_close(got, want, err, "bf16")
        oa.write(cache, numbers(kr), v, slots, pd.NVFP4_ROUND_NEAREST_EVEN)
        now = back(block.cache)
        for name in ("kc", "ks", "vc", "vs"):
            assert np.array_equal(now[name], cache[name]), name
        o = pd.kv_attention(qr, block.cache, block.table, i32(lengths), query_starts=i32(starts), window=window, sinks=sinks)
        want, err = oa.attention(numbers(qr), cache, table, lengths, starts, dim ** -0.5, window, sinks)
        assert_close(o, want, err, "bf16")
        codes, scales, alpha = block.out
        assert torch.equal(y, pd.linear(o.view(n, -1), codes, scales, hidden, alpha=alpha, residual=x, packed=True))
        counts = np.array([1, 1, 1])


@pytest.mark.parametrize("batch,prompt,extra", [(1, 5, []), (3, 700, []), (2, 130, ["--window", "64", "--sinks", "4"])])
def test_attention_example(example, batch, prompt, extra, capsys):
    """The step captured and replayed equals the eager one, step after step."""
    assert example.main(["--batch", str(batch), "--prompt", str(prompt), "--steps", "4", "--hidden", "512", "--heads", "8",
                         "--kv-heads", "2", "--head-dim", "64", *extra])
    assert "equals" in capsys.readouterr().out


def test_streams_at_once():
    """Each stream has a workspace of its own: calls that run side by side do not meet."""
    rng = np.random.default_rng(21)
    kvc = on_device(filled(rng, 400, 2, 16, 128), 128)
    cases = []
    for n in ([2500, 900], [40, 3000], [1700, 1700]):
        table, _ = tables(rng, n, 16, 400, 200)
        cases.append((heads_on_device(queries(rng, 2, 8, 128, "bf16"), "bf16"), i32(table), i32(n)))
    want = [pd.kv_attention(q, kvc, t, n) for q, t, n in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [pd.kv_attention(q, kvc, t, n, stream=s) for (q, t, n), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_graphs_captured_on_their_own_streams_run_side_by_side():
    rng = np.random.default_rng(22)
    kvc = on_device(filled(rng, 400, 2, 16, 64), 64)
    graphs = []
    for n in ([4000], [2000]):
        table, _ = tables(rng, n, 16, 400, 256)
        q, t, ln = heads_on_device(queries(rng, 1, 8, 64, "f16"), "f16"), i32(table), i32(n)
        want = pd.kv_attention(q, kvc, t, ln)
        s = torch.cuda.Stream()
        pd.nvfp4_workspace_reserve(pd.nvfp4_kv_attention_workspace_size(kvc, 8, 1, 1, 1, 256), s)
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pd.kv_attention(q, kvc, t, ln, out=out)
        graphs.append((g, s, out, want, (q, t, ln)))
    for _ in range(4):
        for g, s, out, _, _ in graphs:
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
        torch.cuda.synchronize()
        for _, _, out, want, _ in graphs:
            assert torch.equal(out, want)
