"""Calls that the attention operators' documentation allows and that ordinary programs make
less often: negative globals, rows at odd addresses, keys without queries, one weight of
two, shared block tables and broadcast queries, very many heads, one page, graphs of the
cache's writer and reader, another stream."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import back, filled, heads_on_device, i32, i64, on_device, queries, tables
from ffn_util import CODES, TYPES, assert_close, rounded
from oracle import attn as oa
from test_gpu_attn import check
from test_gpu_cache import dev, rope_case, same_cache, slots_of

pytestmark = pytest.mark.gpu
RULES = [pd.NVFP4_ROUND_HALF_STEP, pd.NVFP4_ROUND_NEAREST_EVEN, pd.NVFP4_ROUND_NEAREST_LOWER]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rule", RULES)
def test_negative_globals_and_rows_at_odd_addresses(rule, kind):
    rng = np.random.default_rng(rule)
    n, kv, dim, page = 21, 2, 80, 16
    k, v = (rounded(rng.standard_normal((n, kv, dim)) * 2, kind) for _ in "kv")
    cache = filled(rng, 3, kv, page, dim)
    cache["kg"] = np.array([-0.37, 1.5], np.float32)
    cache["vg"] = np.array([2.0 ** -3, -7.7], np.float32)
    gpu, slots = on_device(cache, dim), slots_of(rng, n, 3, page)
    oa.write(cache, k.astype(np.float32), v.astype(np.float32), slots, rule)
    pd.kv_cache_write(heads_on_device(k, kind, token=kv * dim + 7, offset=3),
                      heads_on_device(v, kind, token=dim + 1, head=n * (dim + 1) + 5, offset=1), gpu, i64(slots), rule=rule)
    same_cache(gpu, cache)
    for g, w in zip(pd.kv_cache_read(gpu, i64(slots), out_dtype=torch.float32), oa.read(cache, slots, dim)):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=True)


@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
def test_reads_to_odd_addresses(y):
    rng = np.random.default_rng(1)
    kv, dim, page, n = 3, 48, 16, 19
    cache = filled(rng, 2, kv, page, dim)
    slots = rng.integers(-1, 33, n)
    out = [torch.full((n * kv * dim + 9,), 7.0, dtype=TYPES[y], device="cuda") for _ in "kv"]
    pd.nvfp4_kv_read_launch(on_device(cache, dim), i64(slots), n, out[0][1:], out[1][3:], CODES[y])
    for o, at, w in zip(out, (1, 3), oa.read(cache, slots, dim)):
        got = o[at:at + n * kv * dim].view(n, kv, dim).cpu()
        assert torch.equal(got, torch.from_numpy(w).to(TYPES[y]))
        assert bool((o[:at] == 7.0).all()) and bool((o[at + n * kv * dim:] == 7.0).all())


def test_attention_with_negative_globals():
    rng = np.random.default_rng(2)
    for n, tokens in ((1, 300), (1, 900), (8, 900), (50, 300)):
        cache = filled(rng, 80, 2, 16, 64)
        cache["kg"], cache["vg"] = np.array([-0.2, 0.3], np.float32), np.array([1.5, -2.5], np.float32)
        check(rng, [tokens], [n], 8, 2, 64, 16, "bf16", cache=cache, spare=80 - -(-tokens // 16), uniform=True)


@pytest.mark.parametrize("rot", [0, 64])
def test_keys_without_queries_and_one_weight_of_two(rot):
    rng = np.random.default_rng(3)
    q, k, table, pos, w = rope_case(rng, 9, 4, 2, 64, rot, "bf16", True)
    qd, kd = heads_on_device(q, "bf16"), heads_on_device(k, "bf16")
    args = (i64(pos) if rot else None, dev(table))
    for wq, wk in ((w[0], None), (None, w[1])):
        got = pd.qk_norm_rope(qd, kd, *args, q_weight=dev(wq), k_weight=dev(wk), eps=0.0)
        for x, y, ww in ((q, got[0], wq), (k, got[1], wk)):
            want, err = oa.norm_rope(x, ww, pos, table, 0.0, False)
            assert_close(y, want, err, "bf16")
    alone = torch.empty_like(kd)
    pd.nvfp4_qk_norm_rope_launch(None, 0, 0, None, None, 0, 0, 0, kd, 128, 64, dev(w[1]), alone, 128, 64, 2, 64,
                                 pd.NVFP4_OUT_BF16, args[0], args[1], 50 if rot else 0, rot, 0, 0.0, 9)
    assert torch.equal(alone, got[1])


@pytest.mark.parametrize("n", [1, 6])
def test_a_shared_table_and_broadcast_queries(n):
    """Every sequence on the same pages, a block table of row stride 0, queries of one token and
    of one head repeated: as with copies."""
    rng = np.random.default_rng(4)
    cache = on_device(filled(rng, 90, 2, 16, 64), 64)
    table, _ = tables(rng, [1300], 16, 90)
    lengths = i32([1300, 900, 40])
    row = i32(table).expand(3, -1)
    assert row.stride(0) == 0
    for q in (heads_on_device(queries(rng, 1, 8, 64, "bf16"), "bf16").expand(3 * n, -1, -1),
              heads_on_device(queries(rng, 3 * n, 1, 64, "bf16"), "bf16").expand(-1, 8, -1)):
        got = pd.kv_attention(q, cache, row, lengths)
        assert torch.equal(got, pd.kv_attention(q.contiguous(), cache, row.contiguous(), lengths))


@pytest.mark.parametrize("heads,kv", [(512, 1), (1024, 1024), (64, 64)])
@pytest.mark.parametrize("tokens", [40, 700])
def test_very_many_heads(heads, kv, tokens):
    check(np.random.default_rng(heads), [tokens], [2], heads, kv, 64, 16, "bf16", uniform=True)


@pytest.mark.parametrize("page", [16, 1024])
def test_one_page_filled_to_its_end(page):
    for n in (1, 16, 60):
        if n <= page:
            check(np.random.default_rng(page), [page], [n], 4, 1, 128, page, "f16", uniform=True, spare=0)


def test_writes_and_reads_captured_and_replayed():
    rng = np.random.default_rng(5)
    n, kv, dim, page, pages = 37, 2, 128, 16, 6
    cache = filled(rng, pages, kv, page, dim)
    gpu = on_device(cache, dim)
    k, v = (torch.zeros((n, kv, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    slots = i64(np.arange(n))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pd.kv_cache_write(k, v, gpu, slots)
        out = pd.kv_cache_read(gpu, slots)
    same_cache(gpu, cache)
    for _ in range(4):
        x = [rounded(rng.standard_normal((n, kv, dim)), "bf16") for _ in "kv"]
        at = slots_of(rng, n, pages, page)
        k.copy_(torch.from_numpy(x[0]))
        v.copy_(torch.from_numpy(x[1]))
        slots.copy_(i64(at))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        oa.write(cache, x[0].astype(np.float32), x[1].astype(np.float32), at, pd.NVFP4_ROUND_NEAREST_EVEN)
        same_cache(gpu, cache)
        for a, b in zip(out, pd.kv_cache_read(gpu, slots)):
            assert torch.equal(a, b) or bool((a.isnan() == b.isnan()).all())
            assert torch.equal(a.nan_to_num(), b.nan_to_num())


def test_writes_and_reads_on_another_stream():
    rng = np.random.default_rng(6)
    n, kv, dim, page = 300, 4, 64, 64
    k, v = (heads_on_device(queries(rng, n, kv, dim, "f16"), "f16") for _ in "kv")
    one, two = (pd.KvCache.empty(6, kv, page, dim) for _ in range(2))
    slots = i64(rng.permutation(6 * page)[:n])
    pd.kv_cache_write(k, v, one, slots)
    want = pd.kv_cache_read(one, slots)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pd.kv_cache_write(k, v, two, slots, stream=s)
    got = pd.kv_cache_read(two, slots, stream=s)
    s.synchronize()
    same_cache(two, back(one))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
