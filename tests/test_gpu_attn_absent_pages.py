"""Attention over sequences whose block tables have holes (entries outside the cache's
pages): what page 0 holds, NaN scales among them, reaches no row, in any of the kernels."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import NAN_SCALES, filled, heads_on_device, i32, on_device, queries
from ffn_util import assert_close
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


# queries a sequence and tokens: one workgroup a sequence, pieces (one row tile and two), tiles
SHAPES = [(1, 400, 512), (1, 1500, 2048), (4, 400, 512), (8, 1500, 2048), (40, 400, 512), (40, 1500, 2048)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("queries_each,tokens,context", SHAPES)
def test_page_0_does_not_reach_rows_with_holes(queries_each, tokens, context, dim, page, window, sinks):
    """Sequence 0 has holes, sequence 1 none of its pages, sequence 2 all; page 0 belongs to none."""
    rng = np.random.default_rng(tokens + dim + page + window)
    kv, heads, batch, width = 2, 8, 3, context // page
    lengths, counts = [tokens, tokens - 7, 100], [queries_each] * batch
    own = -(-tokens // page) + -(-100 // page)
    clean = filled(rng, own + 1, kv, page, dim)
    order = 1 + rng.permutation(own)
    table = np.full((batch, width), -1, np.int32)
    table[0, :own - -(-100 // page)] = order[-(-100 // page):]
    table[2, :-(-100 // page)] = order[:-(-100 // page)]
    last = (tokens - 1) // page
    for hole, entry in ((0, -1), (last // 2, own + 1), (last - 2, 1 << 30), (last, -(1 << 31))):
        table[0, max(hole, 0)] = entry
    starts = np.concatenate(([0], np.cumsum(counts)))
    q = queries(rng, starts[-1], heads, dim, "bf16")
    nan = {n: None if v is None else v.copy() for n, v in clean.items()}
    for n in ("ks", "vs"):
        nan[n][0] = NAN_SCALES[rng.integers(0, 2, nan[n][0].shape)]
    args = (i32(table), i32(lengths))
    kw = dict(scale=0.05, window=window, sinks=sinks)
    qd = heads_on_device(q, "bf16")
    want, err = oa.attention(q, clean, table, lengths, starts, 0.05, window, sinks)
    first = pd.kv_attention(qd, on_device(clean, dim), *args, **kw)
    assert_close(first, want, err, "bf16")
    got = pd.kv_attention(qd, on_device(nan, dim), *args, **kw)
    assert torch.equal(got, first)
    assert bool((got[starts[1]:starts[2]] == 0).all())


def test_page_0_of_another_sequence():
    """Page 0 is another sequence's and holds a NaN block: that sequence's rows are NaN there,
    those of the one with holes are not."""
    rng = np.random.default_rng(1)
    for tokens in (300, 900):
        cache = filled(rng, 60, 1, 16, 64)
        table = np.full((2, 64), -1, np.int32)
        table[0, :57] = 1 + rng.permutation(57)
        table[0, 3:9] = -1
        table[1, 0] = 0
        cache["vs"][0, 0, 2, 5] = 0x7F
        q = queries(rng, 2, 4, 64, "f16")
        want, err = oa.attention(q, cache, table, [tokens, 16], [0, 1, 2], 0.1)
        assert np.isnan(want[1, :, 32:48]).all() and not np.isnan(want[0]).any()
        got = pd.kv_attention(heads_on_device(q, "f16"), on_device(cache, 64), i32(table), i32([tokens, 16]), scale=0.1)
        assert_close(got, want, err, "f16", f"{tokens}")
