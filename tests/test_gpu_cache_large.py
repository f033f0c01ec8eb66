"""Cache reads of next to 2^27 rows, the most that a call takes."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import filled, i64, on_device
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


def test_read_of_rows_that_round_up_to_2_32_threads():
    # 134217724 rows of 32 lanes: one launch would be 2^24 workgroups of 256
    kv, dim, page, tokens = 31, 208, 16, 2164802
    cache = filled(np.random.default_rng(1), 1, kv, page, dim)
    slots = np.arange(tokens) % (page + 1) - 1          # -1 gives zeros
    want = [torch.from_numpy(w).to(torch.bfloat16).cuda() for w in oa.read(cache, slots[:page + 1], dim)]
    got = pd.kv_cache_read(on_device(cache, dim), i64(slots))
    for g, w in zip(got, want):
        assert g.shape == (tokens, kv, dim)
        whole = tokens // (page + 1)
        parts = g[:whole * (page + 1)].view(whole, page + 1, kv, dim)
        for first in range(0, whole, 4096):
            assert bool((parts[first:first + 4096] == w).all()), f"tokens from {first * (page + 1)}"
        assert torch.equal(g[whole * (page + 1):], w[:tokens - whole * (page + 1)])
    del got, g, parts
    torch.cuda.empty_cache()
