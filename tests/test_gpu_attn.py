"""Attention over the NVFP4 cache on the GPU against the float64 oracle, within
its derived error bounds: histories of every kind of length, head counts and
dimensions, masks that leave rows empty, pages that are not there, NaN in places
that a query does not see."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import NAN_SCALES, back, filled, heads_on_device, i32, on_device, queries, tables
from ffn_util import TYPES, assert_close
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


def check(rng, lengths, counts, heads, kv, dim, page, kind, window=0, sinks=0, scale=None, width=None, uniform=False,
          size=1.0, max_query=None, spare=2, cache=None, behind=0, strides=False):
    lengths, counts = np.asarray(lengths), np.asarray(counts)
    used = int(sum(-(-lengths // page)))
    cache = filled(rng, used + spare, kv, page, dim) if cache is None else cache
    table, free = tables(rng, lengths, page, used + spare, width)
    for p in free:                                      # pages of nobody: NaN
        cache["ks"][p], cache["vs"][p] = 0x7F, 0xFF
    for b, n in enumerate(lengths):                     # and what lies behind a sequence's end
        if n % page:
            p = table[b, n // page]
            cache["ks"][p, :, :, n % page:], cache["vs"][p, :, :, n % page:] = 0xFF, 0x7F
    starts = np.concatenate(([0], np.cumsum(counts)))
    tokens = int(starts[-1])
    q = queries(rng, tokens + behind, heads, dim, kind, size)
    s = dim ** -0.5 if scale is None else scale
    want, err = oa.attention(q, cache, table, lengths, starts, s, window, sinks)
    kvc = on_device(cache, dim)
    if strides:                                         # odd strides and addresses
        qd = heads_on_device(q, kind, token=heads * (dim + 3) + 5, head=dim + 3, offset=1)
        out = heads_on_device(np.full(q.shape, 7.0), kind, token=dim + 1, head=(tokens + behind) * (dim + 1) + 3, offset=3)
        td = torch.full((len(lengths), table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
        td[:, :table.shape[1]] = i32(table)
        td = td[:, :table.shape[1]]
    else:
        qd = heads_on_device(q, kind)
        out = torch.full((tokens + behind, heads, dim), 7.0, dtype=TYPES[kind], device="cuda")
        td = i32(table)
    got = pd.kv_attention(qd, kvc, td, i32(lengths), query_starts=None if uniform else i32(starts),
                          max_query=max_query, scale=scale, window=window, sinks=sinks, out=out)
    torch.cuda.synchronize()
    assert got is out
    assert_close(got[:tokens], want[:tokens], err[:tokens], kind, f"{lengths} {counts}")
    assert bool((got[tokens:] == 7.0).all())
    return got


# one query a sequence, short and long histories around every border
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [[1], [0], [1, 2, 15, 16, 17, 0, 63], [64, 65, 127, 128, 129], [700, 3, 513],
                                     [4097]])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 16), (4, 1, 128, 64), (5, 5, 96, 32), (24, 2, 256, 16),
                                               (7, 1, 192, 128), (3, 3, 16, 16)])
def test_one_query(kind, lengths, heads, kv, dim, page):
    rng = np.random.default_rng(sum(lengths) + heads + dim)
    check(rng, lengths, [1] * len(lengths), heads, kv, dim, page, kind, uniform=True)


# several queries: rows of 16, 32 and 64 and tiles of more, some before the first token
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (8, 1, 128), (6, 2, 80), (4, 2, 256), (9, 3, 192)])
@pytest.mark.parametrize("counts,lengths", [([3, 3], [10, 600]), ([7, 7, 7], [3, 7, 900]), ([70], [70]),
                                            ([33, 33], [1200, 33]), ([130], [200])])
def test_several_queries(heads, kv, dim, counts, lengths):
    rng = np.random.default_rng(sum(counts) + dim)
    check(rng, lengths, counts, heads, kv, dim, 16, "bf16", uniform=True, behind=0)


# ragged batches: sequences without queries, without tokens, rows behind the last
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("max_query", [None, 90])
@pytest.mark.parametrize("counts,lengths", [([1, 0, 5, 2], [40, 9, 70, 0]), ([0, 0, 1], [5, 0, 64]),
                                            ([90, 1, 17, 0, 33], [300, 1000, 17, 4, 20])])
def test_ragged(kind, max_query, counts, lengths):
    rng = np.random.default_rng(sum(counts))
    total = sum(counts) + 3
    check(rng, lengths, counts, 8, 2, 128, 32, kind, behind=3,
          max_query=None if max_query is None else min(max_query, total))


# windows and first tokens that stay
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (64, 4), (65, 64), (100, 65), (500, 1), (1000, 10),
                                          (2000, 0), (7, 300)])
@pytest.mark.parametrize("counts,lengths", [([1, 1, 1], [1, 130, 1500]), ([5, 5], [600, 5]), ([100], [700])])
def test_window(window, sinks, counts, lengths):
    rng = np.random.default_rng(window + sinks)
    check(rng, lengths, counts, 8, 2, 64, 16, "f16", window=window, sinks=sinks, uniform=True)


def test_strides_and_alignment():
    for counts, lengths in (([1, 1], [30, 2000]), ([40, 40], [90, 700])):
        check(np.random.default_rng(3), lengths, counts, 6, 2, 128, 16, "bf16", strides=True, uniform=True)
        check(np.random.default_rng(4), lengths, counts, 6, 2, 80, 16, "f16", strides=True, uniform=True)


def test_scales_and_sizes():
    for scale in (0.0, -0.3, 2.0):
        check(np.random.default_rng(5), [100, 1000], [1, 1], 8, 2, 128, 64, "bf16", scale=scale, uniform=True)
    # rows near the ends of bf16's range, which fp16 does not reach
    for size in (2.0 ** 60, 2.0 ** -60):
        check(np.random.default_rng(6), [100, 1000], [1, 1], 8, 2, 128, 64, "bf16", size=size, scale=1.0 / size / 12,
              uniform=True)
    check(np.random.default_rng(7), [100, 1000], [1, 1], 8, 2, 128, 64, "f16", size=2.0 ** -12, scale=300.0, uniform=True)


def test_rows_of_zeros_and_of_one_large_element():
    rng = np.random.default_rng(8)
    cache = filled(rng, 20, 1, 64, 128)
    table, _ = tables(rng, [1200], 64, 20)
    q = queries(rng, 1, 3, 128, "bf16")
    q[0, 0] = 0.0
    q[0, 1] = 0.0
    q[0, 1, 77] = 2.0 ** -130                 # a subnormal row
    q[0, 2, 5] = 1e4
    want, err = oa.attention(q, cache, table, [1200], [0, 1], 0.05)
    got = pd.kv_attention(heads_on_device(q, "bf16"), on_device(cache, 128), i32(table), i32([1200]), scale=0.05)
    assert_close(got, want, err, "bf16")


def test_nan_reaches_the_queries_that_see_it_and_no_others():
    rng = np.random.default_rng(9)
    for counts, lengths, window in (([6], [500], 0), ([80], [500], 0), ([6], [500], 40), ([1], [500], 0)):
        cache = filled(rng, 40, 2, 16, 128)
        table, _ = tables(rng, lengths, 16, 40)
        # NaN in V's blocks 0 and 5 of token 497 and in K of token 499, kv head 1 only
        p, o = table[0, 497 // 16], 497 % 16
        cache["vs"][p, 1, 0, o], cache["vs"][p, 1, 5, o] = NAN_SCALES
        cache["ks"][table[0, 499 // 16], 1, 3, 499 % 16] = 0x7F
        q = queries(rng, counts[0], 4, 128, "bf16")
        want, err = oa.attention(q, cache, table, lengths, [0, counts[0]], 0.1, window)
        got = pd.kv_attention(heads_on_device(q, "bf16"), on_device(cache, 128), i32(table), i32(lengths), scale=0.1,
                              window=window)
        n = counts[0]
        if n > 3:
            assert np.isnan(want[n - 3, 2, 0]) and not np.isnan(want[n - 3, 2, 16]) and not np.isnan(want[n - 4]).any()
        assert np.isnan(want[n - 1, 2]).all() and not np.isnan(want[n - 1, 0]).any()
        assert_close(got, want, err, "bf16", f"{counts} {window}")


@pytest.mark.parametrize("counts,lengths", [([1, 1], [900, 70]), ([1, 1], [100, 70]), ([70, 70], [700, 90])])
def test_pages_that_are_not_there(counts, lengths):
    rng = np.random.default_rng(10)
    cache = filled(rng, 80, 2, 16, 64)
    table, _ = tables(rng, lengths, 16, 80)
    table[0, :30:3] = -1
    table[0, 1] = 80
    table[1] = [-5, 1 << 30, 81, -(1 << 31), 80, 100][:1] * table.shape[1]      # nothing of sequence 1 is there
    starts = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, starts[-1], 4, 64, "f16")
    want, err = oa.attention(q, cache, table, lengths, starts, 0.125)
    got = pd.kv_attention(heads_on_device(q, "f16"), on_device(cache, 64), i32(table), i32(lengths))
    assert_close(got, want, err, "f16")
    assert bool((got[starts[1]:] == 0).all())


def test_lengths_and_starts_outside_their_range_stay_inside_the_buffers():
    rng = np.random.default_rng(11)
    cache = filled(rng, 12, 1, 16, 64)
    table, _ = tables(rng, [192], 16, 12)
    q = queries(rng, 4, 2, 64, "bf16")
    want, err = oa.attention(q, cache, np.repeat(table, 2, 0), [192, 0], [0, 4, 4], 0.125)
    got = pd.kv_attention(heads_on_device(q, "bf16"), on_device(cache, 64), i32(np.repeat(table, 2, 0)),
                          i32([1 << 30, -9]), query_starts=i32([-3, 1 << 29, 2]))
    assert_close(got, want, err, "bf16")


def test_long_cache_of_many_pages():
    # codes and scales beyond 2^32 bytes: 9 GiB of K, pages at both ends
    pages, kv, page, dim = 1200000, 2, 64, 128
    k = torch.zeros((pages, kv, page, dim // 2), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((pages, kv, dim // 16, page), dtype=torch.uint8, device="cuda")
    kvc = pd.KvCache(k, ks, k.clone(), ks.clone(), head_dim=dim)
    rng = np.random.default_rng(12)
    n = 64 * 12 + 5
    table = np.concatenate((np.arange(pages - 7, pages), [0, 600000, 3, 899999, 1, 7])).astype(np.int32)[None]
    small = filled(rng, 13, kv, page, dim)
    small["kg"] = small["vg"] = None
    at = torch.from_numpy(table[0].astype(np.int64)).cuda()
    for name, t in zip(("kc", "ks", "vc", "vs"), kvc.tensors):
        t[at] = torch.from_numpy(small[name]).cuda()
    for counts in (1, 40):
        q = queries(rng, counts, 4, dim, "bf16")
        want, err = oa.attention(q, small, np.arange(13)[None], [n], [0, counts], 0.02)
        got = pd.kv_attention(heads_on_device(q, "bf16"), kvc, i32(table), i32([n]), scale=0.02)
        assert_close(got, want, err, "bf16")
    del kvc, k, ks
    torch.cuda.empty_cache()


def test_many_sequences():
    rng = np.random.default_rng(13)
    lengths = rng.integers(0, 90, 700)
    check(rng, lengths, [1] * 700, 4, 1, 64, 16, "bf16", uniform=True, width=40)
    counts = rng.integers(0, 3, 700)
    check(rng, lengths, counts, 4, 1, 64, 16, "bf16", width=40)


def test_replay_with_other_lengths_and_pages():
    rng = np.random.default_rng(14)
    cache = filled(rng, 100, 2, 16, 128)
    kvc = on_device(cache, 128)
    width, batch = 40, 3
    q = torch.zeros((batch, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    table, lengths = i32(np.zeros((batch, width))), i32(np.ones(batch))
    s = torch.cuda.Stream()
    pd.nvfp4_workspace_reserve(pd.nvfp4_kv_attention_workspace_size(kvc, 8, batch, batch, 1, width), s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pd.kv_attention(q, kvc, table, lengths, out=out)
    for i in range(4):
        n = rng.integers(0, 500, batch)
        t, _ = tables(rng, n, 16, 100, width)
        x = queries(rng, batch, 8, 128, "bf16")
        table.copy_(i32(t))
        lengths.copy_(i32(n))
        q.copy_(torch.from_numpy(x))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, err = oa.attention(x, cache, t, n, np.arange(batch + 1), 128 ** -0.5)
        assert_close(out, want, err, "bf16", f"replay {i}")
        assert torch.equal(out, pd.kv_attention(q, kvc, table, lengths))


def test_results_repeat_and_do_not_depend_on_other_sequences():
    rng = np.random.default_rng(15)
    cache = filled(rng, 300, 2, 16, 128)
    kvc = on_device(cache, 128)
    table, _ = tables(rng, [1500, 900, 64], 16, 300)
    q = heads_on_device(queries(rng, 3, 8, 128, "bf16"), "bf16")
    got = [pd.kv_attention(q, kvc, i32(table), i32([1500, 900, 64])) for _ in range(3)]
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_own_workspace_and_streams():
    rng = np.random.default_rng(16)
    cache = filled(rng, 100, 2, 16, 128)
    kvc = on_device(cache, 128)
    table, _ = tables(rng, [1500], 16, 100)
    td, ln = i32(table), i32([1500])
    q = heads_on_device(queries(rng, 1, 8, 128, "bf16"), "bf16")
    want = pd.kv_attention(q, kvc, td, ln)
    need = pd.nvfp4_kv_attention_workspace_size(kvc, 8, 1, 1, 1, table.shape[1])
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    pd.nvfp4_kv_attention_launch_ws(kvc, q, 1024, 128, out, 1024, 128, 8, pd.NVFP4_OUT_BF16, td, table.shape[1],
                                    table.shape[1], ln, None, 1, 1, 1, 128 ** -0.5, 0, 0, ws, need, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    other = pd.kv_attention(q, kvc, td, ln, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    assert back(kvc)["kc"].tobytes() == cache["kc"].tobytes()      # only read
