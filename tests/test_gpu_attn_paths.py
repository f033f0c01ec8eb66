"""Attention through the kernels and plans that calls of ordinary shapes reach: tiles of
256 rows at every head dimension, tiles whose steps are shared out, pieces of sequences
after the first 64, NaN joined from pieces, batches of a prompt and single tokens; and
rows that depend on nothing of other sequences but their lengths."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import filled, heads_on_device, i32, on_device, queries, tables
from ffn_util import assert_close
from oracle import attn as oa
from test_gpu_attn import check

pytestmark = pytest.mark.gpu
DIMS = [64, 96, 128, 192, 256]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


# tiles of 256 rows: more than 128 rows a sequence, at least 256 tiles and heads
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", DIMS)
def test_tiles_of_256_rows_ragged(dim, kind, window, sinks):
    rng = np.random.default_rng(dim)
    batch = 70
    counts = rng.integers(0, 9, batch)
    counts[[0, 40]] = 8
    lengths = counts + rng.integers(0, 300, batch) * (rng.integers(0, 4, batch) > 0)
    lengths[7] = 3                                      # fewer tokens than queries
    counts[7] = 8
    # 32 rows a query, a tile a sequence and kv head
    check(rng, lengths, counts, 128, 4, dim, 16, kind, window=window, sinks=sinks, max_query=8, behind=5)


@pytest.mark.parametrize("dim", DIMS)
def test_tiles_of_256_rows_prompt(dim):
    rng = np.random.default_rng(dim + 1)
    # 100 queries of 32 rows: 13 tiles, beside 60 sequences of one query
    lengths = np.concatenate(([409], rng.integers(1, 200, 60)))
    for window, sinks in ((0, 0), (133, 70)):
        check(rng, lengths, [100] + [1] * 60, 128, 4, dim, 64, "bf16", window=window, sinks=sinks, max_query=100)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("counts,lengths,window,sinks", [([64], [600], 0, 0), ([64], [600], 170, 66), ([64], [4200], 700, 66),
                                                        ([30, 0, 9, 25], [2190, 70, 40, 900], 0, 0)])
def test_many_tiles_with_shared_steps(dim, counts, lengths, window, sinks):
    """64 to 255 tiles and heads with a table of more than 4096 tokens: steps in 8 parts."""
    rng = np.random.default_rng(sum(lengths) + dim)
    check(rng, lengths, counts, 128, 2, dim, 16, "f16", window=window, sinks=sinks, width=264, max_query=max(counts))


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (4, 1, 128), (16, 1, 128), (3, 3, 192), (8, 2, 256)])
@pytest.mark.parametrize("most", [1, 2])
def test_pieces_after_the_first_64_sequences(heads, kv, dim, most):
    rng = np.random.default_rng(dim + most)
    batch = 130
    counts = rng.integers(0, most + 1, batch)
    lengths = counts + rng.integers(0, 3, batch) * rng.integers(0, 60, batch)
    for b, n in ((3, 1300), (63, 700), (64, 2900), (65, 0), (66, 611), (100, 1024), (127, 65), (128, 1999), (129, 640)):
        lengths[b], counts[b] = n, most
    check(rng, lengths, counts, heads, kv, dim, 32, "bf16", max_query=most, width=96, behind=2)
    check(rng, lengths, counts, heads, kv, dim, 32, "f16", max_query=most, width=96, window=500, sinks=9)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 24])
def test_nan_through_the_pieces(dim, n):
    """NaN blocks of K and V in single pieces reach the rows of their kv head, in their block,
    through the join; a window hides them again."""
    rng = np.random.default_rng(dim + n)
    tokens = 1800
    for window in (0, 200):
        cache = filled(rng, 180, 2, 16, dim)
        table, _ = tables(rng, [tokens, 900], 16, 180)
        seen = tokens - 100
        for j, block in ((11, 0), (1003, 3), (seen, 1)):
            cache["vs"][table[0, j // 16], 1, block, j % 16] = 0x7F
        cache["ks"][table[1, 20], 0, 2, 5] = 0xFF
        q = queries(rng, 2 * n, 4, dim, "bf16")
        starts = [0, n, 2 * n]
        want, err = oa.attention(q, cache, table, [tokens, 900], starts, 0.05, window)
        assert np.isnan(want[0, 2, 16:32]).all() and np.isnan(want[0, 2, :16]).all() == (window == 0)
        assert not np.isnan(want[:n, 0]).any() and np.isnan(want[n:, 0]).all() == (window == 0)
        got = pd.kv_attention(heads_on_device(q, "bf16"), on_device(cache, dim), i32(table), i32([tokens, 900]),
                              scale=0.05, window=window)
        assert_close(got, want, err, "bf16", f"window {window}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_prompt_among_single_tokens(dim):
    rng = np.random.default_rng(dim)
    counts = np.ones(40, np.int64)
    counts[[5, 39]] = [200, 130]
    lengths = np.where(counts > 1, counts + 100, rng.integers(1, 900, 40))
    check(rng, lengths, counts, 8, 2, dim, 16, "bf16", max_query=200)
    check(rng, lengths, counts, 8, 2, dim, 16, "bf16", max_query=200, window=64, sinks=4, width=70)


@pytest.mark.parametrize("dim", [128, 192, 256])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (65, 64), (500, 1), (7, 300)])
@pytest.mark.parametrize("counts,lengths", [([1, 1, 1], [1, 130, 1500]), ([5, 5], [600, 5]), ([100], [700])])
def test_windows_of_wide_heads(kind, window, sinks, counts, lengths, dim):
    rng = np.random.default_rng(window + sinks + dim)
    check(rng, lengths, counts, 8, 2, dim, 16, kind, window=window, sinks=sinks, uniform=True)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("counts,lengths,width", [
    ([1, 1, 1], [400, 90, 512], 32), ([1, 1, 1], [1500, 700, 2000], 130), ([4, 4, 4], [1500, 700, 2000], 130),
    ([70, 33, 80], [400, 90, 512], 32), ([70, 33, 80], [1500, 700, 2000], 130), ([300, 1, 7], [1500, 700, 2000], 264)])
def test_rows_depend_on_no_value_of_another_sequence(kind, counts, lengths, width):
    """Other queries, keys, values and pages of the sequences beside one, NaN and infinities
    among them, at the same lengths: its rows keep every bit."""
    rng = np.random.default_rng(sum(lengths) + counts[0])
    dim, heads, kv, page, pages = 128, 8, 2, 16, 300
    starts = np.concatenate(([0], np.cumsum(counts)))
    cache = filled(rng, pages, kv, page, dim)
    table, free = tables(rng, lengths, page, pages, width)
    q = queries(rng, starts[-1], heads, dim, kind)

    def call(q, cache, table):
        return pd.kv_attention(heads_on_device(q, kind), on_device(cache, dim), i32(table), i32(lengths),
                               query_starts=i32(starts), max_query=max(counts))

    first = call(q, cache, table)
    for b in range(3):
        mine = table[b, :-(-lengths[b] // page)]
        for special in (False, True):
            other = filled(rng, pages, kv, page, dim, nan=special)
            for n in ("kc", "ks", "vc", "vs"):
                other[n][mine] = cache[n][mine]
            other["kg"], other["vg"] = cache["kg"], cache["vg"]
            t, x = table.copy(), queries(rng, starts[-1], heads, dim, kind)
            for o in range(3):
                if o != b:
                    count = -(-lengths[o] // page)
                    t[o, :count] = rng.permutation(free)[:count] if count <= len(free) and not special else \
                        rng.permutation(t[o, :count])
            t[b], x[starts[b]:starts[b + 1]] = table[b], q[starts[b]:starts[b + 1]]
            if special:
                rows = np.r_[0:starts[b], starts[b + 1]:starts[3]]
                x[rows, ::2, 3], x[rows, 1::2, 9] = np.nan, np.inf
            got = call(x, other, t)
            assert torch.equal(got[starts[b]:starts[b + 1]], first[starts[b]:starts[b + 1]]), f"sequence {b}"
            if special:
                assert bool(got[rows].isnan().any())
