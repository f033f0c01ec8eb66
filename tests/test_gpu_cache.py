"""Head norms with the position rotation, cache writes and reads on the GPU:
quantised blocks bit for bit against the oracle, norms and rotations within its
derived error bounds, and the call that does both against the two calls."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from attn_util import back, filled, heads_on_device, i64, on_device
from ffn_util import TYPES, assert_close, rounded
from oracle import attn as oa

pytestmark = pytest.mark.gpu
RULES = [pd.NVFP4_ROUND_HALF_STEP, pd.NVFP4_ROUND_NEAREST_EVEN, pd.NVFP4_ROUND_NEAREST_LOWER]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


def same_cache(kv, want):
    got = back(kv)
    for n in ("kc", "ks", "vc", "vs"):
        assert np.array_equal(got[n], want[n]), f"{n}: {int((got[n] != want[n]).sum())} bytes differ"


def slots_of(rng, n, pages, page):
    s = rng.permutation(pages * page)[:n].astype(np.int64)
    s[::5] = np.array([-1, pages * page, 1 << 62, -(1 << 63)])[np.arange(len(s[::5])) % 4]   # left out
    return s


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n,kv,dim,page", [(1, 1, 64, 16), (37, 3, 128, 16), (50, 2, 80, 64), (9, 5, 256, 32),
                                           (20, 1, 192, 128), (11, 2, 16, 16)])
def test_write_and_read(rule, kind, n, kv, dim, page):
    rng = np.random.default_rng(n + dim + rule)
    pages = -(-n // page) + 2
    k, v = (rounded(rng.standard_normal((n, kv, dim)) * np.exp2(rng.integers(-12, 9, (n, kv, 1))), kind) for _ in "kv")
    k[0, 0, :16] = 0.0
    k[-1, -1, 3] = -0.0
    cache = filled(rng, pages, kv, page, dim)           # what is not written stays
    kv_gpu = on_device(cache, dim)
    slots = slots_of(rng, n, pages, page)
    oa.write(cache, k.astype(np.float32), v.astype(np.float32), slots, rule)
    pd.kv_cache_write(heads_on_device(k, kind), heads_on_device(v, kind), kv_gpu, i64(slots), rule=rule)
    same_cache(kv_gpu, cache)
    every = np.concatenate((slots, np.arange(pages * page)))
    for y in ("bf16", "f16", "f32"):
        got = pd.kv_cache_read(kv_gpu, i64(every), out_dtype=TYPES[y])
        for g, w in zip(got, oa.read(cache, every, dim)):
            # NaN blocks (a scale past E4M3) read back as NaN
            torch.testing.assert_close(g.cpu(), torch.from_numpy(w).to(TYPES[y]), rtol=0, atol=0, equal_nan=True)


def test_write_of_special_values_and_globals():
    rng = np.random.default_rng(1)
    n, kv, dim, page = 24, 2, 64, 16
    k, v = (rounded(rng.standard_normal((n, kv, dim)), "bf16") for _ in "kv")
    k[0, 0, 5], k[1, 0, 5], k[2, 1, 20] = np.nan, np.inf, -np.inf
    k[3] = 2.0 ** -130                                   # subnormal inputs
    k[4] = rounded(np.full((kv, dim), 3e38), "bf16")
    v[5, :, ::2] = 0.0
    for g in (1.0, 1e-3, 7.7, 2.0 ** 40, 2.0 ** -60, 0.0, np.inf, np.nan):
        cache = filled(rng, 3, kv, page, dim)
        cache["kg"][0] = cache["vg"][1] = g
        for rule in RULES:
            kv_gpu = on_device(cache, dim)
            want = {x: None if y is None else y.copy() for x, y in cache.items()}
            oa.write(want, k.astype(np.float32), v.astype(np.float32), np.arange(n), rule)
            pd.kv_cache_write(heads_on_device(k, "bf16"), heads_on_device(v, "bf16"), kv_gpu, i64(np.arange(n)), rule=rule)
            same_cache(kv_gpu, want)


def test_write_matches_the_activation_quantiser():
    rng = np.random.default_rng(2)
    x = heads_on_device(rounded(rng.standard_normal((64, 1, 128)), "bf16"), "bf16")
    g = torch.tensor([0.37], device="cuda")
    kv = pd.KvCache.empty(1, 1, 64, 128, k_global=g, v_global=g)
    for rule in RULES:
        pd.kv_cache_write(x, x, kv, i64(np.arange(64)), rule=rule)
        codes, scales = pd.quantize_activation(x.reshape(64, 128).contiguous(), g, rule=rule)
        assert torch.equal(kv.tensors[0][0, 0], codes) and torch.equal(kv.tensors[1][0, 0].t(), scales)
        assert torch.equal(kv.tensors[2], kv.tensors[0]) and torch.equal(kv.tensors[3], kv.tensors[1])


def table_of(rng, rows, rot):
    a = rng.uniform(-np.pi, np.pi, (rows, rot // 2))
    return np.concatenate((np.cos(a), np.sin(a)), axis=1).astype(np.float32)


def rope_case(rng, n, heads, kv, dim, rot, kind, norm):
    q, k = (rounded(rng.standard_normal((n, h, dim)) * 3, kind) for h in (heads, kv))
    table = table_of(rng, 50, rot) if rot else None
    pos = rng.integers(0, 50, n)
    w = [rng.uniform(0.5, 1.5, dim).astype(np.float32) if norm else None for _ in "qk"]
    return q, k, table, pos, w


def dev(x):
    return None if x is None else torch.from_numpy(x).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("n,heads,kv,dim,rot", [(1, 8, 2, 64, 64), (13, 5, 1, 128, 128), (40, 3, 3, 80, 32),
                                                (7, 4, 2, 96, 96), (5, 2, 1, 256, 128), (6, 9, 3, 192, 192),
                                                (3, 1, 1, 16, 16), (4, 6, 2, 128, 0), (9, 2, 2, 128, 16)])
def test_norm_rope(interleaved, kind, norm, n, heads, kv, dim, rot):
    rng = np.random.default_rng(n + dim + rot)
    q, k, table, pos, w = rope_case(rng, n, heads, kv, dim, rot, kind, norm)
    args = (i64(pos) if rot else None, dev(table))
    kw = dict(q_weight=dev(w[0]), k_weight=dev(w[1]), eps=1e-5, interleaved=interleaved)
    qd, kd = heads_on_device(q, kind), heads_on_device(k, kind)
    got = pd.qk_norm_rope(qd, kd, *args, **kw)
    for x, y, ww in ((q, got[0], w[0]), (k, got[1], w[1])):
        want, err = oa.norm_rope(x, ww, pos, table, 1e-5, interleaved)
        assert_close(y, want, err, kind)
    # in place, in the parts of one projection at an odd place, and in another layout
    both = heads_on_device(np.concatenate((q, k), axis=1), kind, token=(heads + kv) * dim + 3, offset=1)
    pd.qk_norm_rope(both[:, :heads], both[:, heads:], *args, q_out=both[:, :heads], k_out=both[:, heads:], **kw)
    assert torch.equal(both[:, :heads], got[0]) and torch.equal(both[:, heads:], got[1])
    out = torch.zeros((heads, n, dim), dtype=TYPES[kind], device="cuda").transpose(0, 1)
    pd.qk_norm_rope(qd, kd, *args, q_out=out, **kw)
    assert torch.equal(out, got[0])


def test_positions_outside_the_table_give_nan():
    rng = np.random.default_rng(3)
    q, k, table, _, w = rope_case(rng, 5, 3, 2, 64, 32, "bf16", True)
    pos = np.array([0, -1, 49, 50, 1 << 40])
    got = pd.qk_norm_rope(heads_on_device(q, "bf16"), heads_on_device(k, "bf16"), i64(pos), dev(table),
                          q_weight=dev(w[0]))
    want, err = oa.norm_rope(q, w[0], pos, table, 1e-6, False)
    assert np.isnan(want[[1, 3, 4]]).all()
    assert_close(got[0], want, err, "bf16")


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,kv,dim,rot", [(1, 8, 2, 64, 64), (33, 4, 2, 128, 64), (10, 3, 1, 80, 80),
                                                (6, 2, 2, 256, 256)])
def test_rope_into_the_cache_is_the_two_calls(rule, kind, interleaved, n, heads, kv, dim, rot):
    rng = np.random.default_rng(n + dim)
    q, k, table, pos, w = rope_case(rng, n, heads, kv, dim, rot, kind, True)
    v = rounded(rng.standard_normal((n, kv, dim)), kind)
    page, pages = 16, n // 16 + 2
    cache = filled(rng, pages, kv, page, dim)
    slots = i64(slots_of(rng, n, pages, page))
    qkv = heads_on_device(np.concatenate((q, k, v), axis=1), kind)
    parts = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    kw = dict(q_weight=dev(w[0]), k_weight=dev(w[1]), interleaved=interleaved)
    one, two = on_device(cache, dim), on_device(cache, dim)
    q1, none = pd.qk_norm_rope(parts[0], parts[1], i64(pos), dev(table), v=parts[2], cache=one, slots=slots, rule=rule, **kw)
    q2, k2 = pd.qk_norm_rope(parts[0], parts[1], i64(pos), dev(table), **kw)
    pd.kv_cache_write(k2, parts[2], two, slots, rule=rule)
    assert none is None and torch.equal(q1, q2)
    same_cache(one, back(two))


def test_slots_beyond_32_bits_of_bytes():
    pages, kv, page, dim = 1200000, 2, 64, 128
    kvc = pd.KvCache.empty(pages, kv, page, dim)
    rng = np.random.default_rng(4)
    slots = np.array([pages * page - 1, 0, 70000000, pages * page - 64, 33554432])
    k, v = (rounded(rng.standard_normal((5, kv, dim)), "bf16") for _ in "kv")
    pd.kv_cache_write(heads_on_device(k, "bf16"), heads_on_device(v, "bf16"), kvc, i64(slots))
    small = oa.empty(1, kv, 16, dim)
    oa.write(small, k.astype(np.float32), v.astype(np.float32), np.arange(5), pd.NVFP4_ROUND_NEAREST_EVEN)
    for g, w in zip(pd.kv_cache_read(kvc, i64(slots), out_dtype=torch.float32), oa.read(small, np.arange(5), dim)):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int((kvc.tensors[0] != 0).sum()) == int((small["kc"] != 0).sum())
    del kvc
    torch.cuda.empty_cache()
