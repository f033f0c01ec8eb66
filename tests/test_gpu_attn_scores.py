"""Attention where scores are far from ordinary: finite ones of 2^20 to 2^90, whose
softmax is one or a few tokens, globals that are not finite, and rows of queries whose
elements are very different in size."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import filled, heads_on_device, i32, on_device, tables
from ffn_util import assert_close, rounded
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


# queries and tokens: one workgroup a sequence, pieces of one and two row tiles, tiles
SHAPES = [(1, 400), (1, 3000), (24, 3000), (40, 900)]
# |score| is up to 128 * 60000 * 2688 * scale in fp16: these span 2^20 .. 2^34; bf16 rows reach 2^90
SIZES = [("f16", 6e4, s) for s in (5.3e-5, 1.1e-3, 3.7e-3, 0.0131, 0.0883883, 0.37, 0.9)] + \
    [("bf16", 2.0 ** 60, s) for s in (1e-12, 0.0883883)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,tokens", SHAPES)
@pytest.mark.parametrize("kind,size,scale", SIZES)
def test_large_scores_choose_their_tokens(kind, size, scale, n, tokens, dim):
    """Head 0's queries meet one token with the largest score, head 1's three of equal keys far
    apart; all others reach a quarter of it at most, so that their weight is zero.
    The weights are then 1 or thirds: they err by fp16's rounding where the running
    maximum lies below, 2^-11, and the sums by 2^-20."""
    scale = float(np.float32(scale))                    # equal scores are then equal in 64 bits too
    rng = np.random.default_rng(tokens + dim)
    page, pages = 16, -(-tokens // 16) + 1
    cache = filled(rng, pages, 2, page, dim)
    cache["kg"], cache["vg"] = None, np.array([0.5, 2.0], np.float32)
    cache["kc"][..., :dim // 2] &= 0x55                 # K positive, at most 3
    cache["kc"][..., :dim // 2] |= 0x11                 # and not zero
    cache["ks"][:, :, :dim // 16] = 0x76                # times 224
    table, _ = tables(rng, [tokens], page, pages)
    for h, chosen in ((0, [tokens // 3]), (1, [5, tokens // 2, tokens - n])):
        for j in chosen:
            p, o = table[0, j // page], j % page
            cache["kc"][p, h, o, :dim // 2] = 0x77      # 6 times 448
            cache["ks"][p, h, :dim // 16, o] = 0x7E
    q = rounded(np.full((n, 2, dim), size), kind)
    want, _ = oa.attention(q, cache, table, [tokens], [0, n], scale)
    got = pd.kv_attention(heads_on_device(q, kind), on_device(cache, dim), i32(table), i32([tokens]), scale=scale)
    v = oa.read(cache, table[0, np.arange(tokens) // page].astype(np.int64) * page + np.arange(tokens) % page, dim)[1]
    assert np.allclose(want[0, 0], v[tokens // 3, 0], rtol=1e-12)
    parts = np.abs(v[[5, tokens // 2, tokens - n], 1]).mean(axis=0)
    err = np.stack((np.abs(want[:, 0]), np.broadcast_to(parts, want[:, 1].shape)), axis=1) * (2.0 ** -11 + 2.0 ** -20)
    assert_close(got, want, err, kind)


@pytest.mark.parametrize("n,tokens", SHAPES)
def test_large_scores_of_either_sign(n, tokens):
    """A negative scale and rows of both signs: the row's largest score is a negative one where
    all are negative."""
    rng = np.random.default_rng(n)
    dim, page, pages = 128, 16, -(-tokens // 16) + 1
    cache = filled(rng, pages, 1, page, dim)
    cache["kg"] = cache["vg"] = None
    cache["kc"][..., :dim // 2] = 0x77
    cache["ks"][:, :, :dim // 16] = 0x7E
    table, _ = tables(rng, [tokens], page, pages)
    chosen = tokens // 3                                # the smallest key, half of the others
    cache["ks"][table[0, chosen // page], 0, :, chosen % page] = 0x76
    for scale, size in ((-0.3, 5e4), (0.3, -5e4)):
        q = rounded(np.full((n, 2, dim), size), "f16")
        want, _ = oa.attention(q, cache, table, [tokens], [0, n], scale)
        got = pd.kv_attention(heads_on_device(q, "f16"), on_device(cache, dim), i32(table), i32([tokens]), scale=scale)
        assert_close(got, want, np.abs(want) * (2.0 ** -11 + 2.0 ** -20), "f16")


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("n,tokens,width", [(6, 3, 16), (6, 3, 64), (16, 9, 64), (80, 40, 64)])
def test_globals_that_are_not_finite_leave_rows_without_tokens_zero(n, tokens, width, value):
    """The first n - tokens queries see no token: they are zero whatever the globals are; the
    others are NaN where k_global is not finite."""
    rng = np.random.default_rng(2)
    cache = filled(rng, 8, 2, 16, 64)
    cache["kg"][0] = value
    table, _ = tables(rng, [tokens], 16, 8, width)
    q = heads_on_device(rng.standard_normal((n, 4, 64)), "bf16")
    got = pd.kv_attention(q, on_device(cache, 64), i32(table), i32([tokens]))
    assert bool((got[:n - tokens] == 0).all())
    assert bool(got[n - tokens:, :2].isnan().all()) and bool(got[n - tokens:, 2:].isfinite().all())
    cache["kg"][0], cache["vg"][1] = 1.0, np.nan
    got = pd.kv_attention(q, on_device(cache, 64), i32(table), i32([tokens]))
    assert bool((got[:n - tokens] == 0).all())
    assert bool(got[n - tokens:, 2:].isnan().all()) and bool(got[n - tokens:, :2].isfinite().all())


@pytest.mark.parametrize("power", [20, 27, 31])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("n,tokens", SHAPES)
def test_small_elements_beside_a_large_one_that_meets_zeros(n, tokens, dim, power):
    """Elements of a bf16 row down to 2^-31 of its largest keep their bits: the largest meets
    zeros of K here, so that the scores are those of the others alone."""
    rng = np.random.default_rng(n + dim)
    page, pages = 16, -(-tokens // 16) + 1
    cache = filled(rng, pages, 2, page, dim)
    cache["kc"][..., 0] &= 0xF0
    table, _ = tables(rng, [tokens], page, pages)
    q = rounded(rng.uniform(1.0, 2.0, (n, 4, dim)) * rng.choice([-1.0, 1.0], (n, 4, dim)), "bf16")
    q[..., 0] = 2.0 ** power
    want, err = oa.attention(q, cache, table, [tokens], [0, n], 0.05)
    got = pd.kv_attention(heads_on_device(q, "bf16"), on_device(cache, dim), i32(table), i32([tokens]), scale=0.05)
    assert_close(got, want, err, "bf16")
