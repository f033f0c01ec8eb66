"""Refusals of the attention operators without a GPU: every invalid call returns
the documented status before any HIP call, calls of no tokens do nothing, and the
tensor-level calls raise ValueError on tensors that are not on a device."""
import ctypes
import os

import pytest
import torch

import precision_decode_amd as pd
from precision_decode_amd import _binding

GPU_VISIBLE = os.path.exists("/dev/kfd")
fake_pointers = pytest.mark.skipif(GPU_VISIBLE, reason="fake device addresses are passed to launch calls "
                                   "only on machines without a GPU")
CACHE = dict(k_codes=0x100000000, k_scales=0x110000000, v_codes=0x120000000, v_scales=0x130000000,
             k_global=0x140000000, v_global=0x150000000, pages=8, page_size=16, kv_heads=2, head_dim=64)
CODES, SCALES = 8 * 2 * 16 * 32, 8 * 2 * 16 * 4   # bytes of a buffer
NAN, INF = float("nan"), float("inf")

BAD_CACHES = [dict(pages=0), dict(pages=-1), dict(pages=1 << 27), dict(page_size=8), dict(page_size=2048),
              dict(page_size=24), dict(page_size=0), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0),
              dict(head_dim=8), dict(head_dim=72), dict(head_dim=272)]
MISALIGNED_CACHES = [dict(k_codes=0x100000008), dict(v_codes=0x120000004), dict(k_scales=0x110000008),
                     dict(v_scales=0x130000001), dict(k_global=0x140000002), dict(v_global=0x150000001)]
POINTERS = ["k_codes", "k_scales", "v_codes", "v_scales"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        from precision_decode_amd import build
        build.build()
    return pd.load()


def cache(**kw):
    return ctypes.byref(pd.KvCacheStruct(**dict(CACHE, **kw)))


def write(c=None, no_cache=False, K=0x200000000, kt=128, kh=64, V=0x210000000, vt=128, vh=64, x_type=1,
          slots=0x220000000, tokens=4, rule=0):
    return pd.load().nvfp4_kv_write_launch(None if no_cache else cache(**(c or {})), K, kt, kh, V, vt, vh, x_type,
                                           slots, tokens, rule, None)


def read(c=None, no_cache=False, slots=0x220000000, tokens=4, K=0x200000000, V=0x210000000, y_type=1):
    return pd.load().nvfp4_kv_read_launch(None if no_cache else cache(**(c or {})), slots, tokens, K, V, y_type, None)


def rope(c=None, cached=False, **kw):
    a = dict(Q=0x300000000, qt=256, qh=64, qw=0x310000000, Qo=0x320000000, qot=256, qoh=64, heads=4,
             K=0x330000000, kt=128, kh=64, kw=0x340000000, Ko=None if cached else 0x350000000, kot=128, koh=64, kv=2,
             dim=64, x_type=1, positions=0x360000000, cos_sin=0x370000000, rows=100, rot=64, inter=0, eps=1e-6,
             tokens=4, V=0x380000000 if cached else None, vt=128, vh=64, slots=0x390000000 if cached else None, rule=0)
    a.update(kw)
    return pd.load().nvfp4_qk_norm_rope_launch(
        a["Q"], a["qt"], a["qh"], a["qw"], a["Qo"], a["qot"], a["qoh"], a["heads"], a["K"], a["kt"], a["kh"], a["kw"],
        a["Ko"], a["kot"], a["koh"], a["kv"], a["dim"], a["x_type"], a["positions"], a["cos_sin"], a["rows"],
        a["rot"], a["inter"], a["eps"], a["tokens"], cache(**(c or {})) if cached else None, a["V"], a["vt"],
        a["vh"], a["slots"], a["rule"], None)


def attend(c=None, no_cache=False, **kw):
    a = dict(Q=0x400000000, qt=256, qh=64, out=0x410000000, ot=256, oh=64, heads=4, x_type=1, table=0x420000000,
             stride=4, width=4, lengths=0x430000000, starts=0x440000000, batch=2, tokens=6, max_query=3, scale=0.125,
             window=0, sinks=0, ws=None, bytes=0)
    a.update(kw)
    return pd.load().nvfp4_kv_attention_launch_ws(
        None if no_cache else cache(**(c or {})), a["Q"], a["qt"], a["qh"], a["out"], a["ot"], a["oh"], a["heads"],
        a["x_type"], a["table"], a["stride"], a["width"], a["lengths"], a["starts"], a["batch"], a["tokens"],
        a["max_query"], a["scale"], a["window"], a["sinks"], a["ws"], a["bytes"], None)


@fake_pointers
def test_no_tokens_do_nothing():
    assert write(tokens=0) == read(tokens=0) == rope(tokens=0) == rope(cached=True, tokens=0) == 0
    assert attend(tokens=0) == attend(tokens=0, starts=None) == 0


@fake_pointers
@pytest.mark.parametrize("call", [write, read, attend, lambda c: rope(c, cached=True)])
def test_bad_caches(call):
    for name in POINTERS:
        assert call({name: None}) == pd.NVFP4_GEMV_ERR_NULL_POINTER, name
    for c in BAD_CACHES:
        assert call(c) == pd.NVFP4_GEMV_ERR_BAD_SHAPE, c
    for c in MISALIGNED_CACHES:
        assert call(c) == pd.NVFP4_GEMV_ERR_ALIGNMENT, c


@fake_pointers
def test_null_pointers():
    assert write(no_cache=True) == read(no_cache=True) == attend(no_cache=True) == pd.NVFP4_GEMV_ERR_NULL_POINTER
    for call, names in ((write, ["K", "V", "slots"]), (read, ["K", "V", "slots"]),
                        (rope, ["Q", "Qo", "K", "Ko", "positions", "cos_sin"]),
                        (attend, ["Q", "out", "table", "lengths"])):
        for name in names:
            assert call(**{name: None}) == pd.NVFP4_GEMV_ERR_NULL_POINTER, name
    for name in ("V", "slots"):
        assert rope(cached=True, **{name: None}) == pd.NVFP4_GEMV_ERR_NULL_POINTER
        assert rope(**{name: 0x500000000}) == pd.NVFP4_GEMV_ERR_NULL_POINTER   # without the rest of a cache


@fake_pointers
def test_bad_arguments():
    for call, cases in ((write, [dict(x_type=2), dict(x_type=-1), dict(rule=-1), dict(rule=3)]),
                        (read, [dict(y_type=3), dict(y_type=-1)]),
                        (rope, [dict(x_type=2), dict(inter=2), dict(inter=-1), dict(eps=-1.0), dict(eps=NAN),
                                dict(eps=INF), dict(rule=3), dict(cached=True, Ko=0x350000000)]),
                        (attend, [dict(x_type=2), dict(x_type=-1), dict(scale=NAN), dict(scale=INF)])):
        for kw in cases:
            assert call(**kw) == pd.NVFP4_GEMV_ERR_BAD_ARGUMENT, kw


@fake_pointers
def test_bad_shapes():
    far = (1 << 40) + 8
    for call, cases in (
            (write, [dict(tokens=-1), dict(tokens=1 << 24), dict(kt=-8), dict(kh=-8), dict(vt=far), dict(vh=far),
                     dict(c=dict(kv_heads=1024), kt=1 << 16, vt=1 << 16, tokens=1 << 16)]),
            (read, [dict(tokens=-1), dict(tokens=1 << 24), dict(c=dict(kv_heads=1024), tokens=1 << 16)]),
            (rope, [dict(tokens=-1), dict(tokens=1 << 24), dict(heads=-1), dict(heads=16385), dict(kv=0), dict(dim=72),
                    dict(rot=-16), dict(rot=8), dict(rot=80), dict(rows=0), dict(rows=-1), dict(qt=-1), dict(qoh=-1),
                    dict(kot=far), dict(qoh=63), dict(koh=0), dict(qot=255), dict(qot=0), dict(kot=64),
                    dict(cached=True, kv=1), dict(cached=True, dim=48), dict(cached=True, vt=-1)]),
            (attend, [dict(heads=0), dict(heads=3), dict(heads=16386), dict(tokens=-1), dict(tokens=1 << 24),
                      dict(batch=0), dict(batch=65536), dict(max_query=0), dict(max_query=7), dict(width=0),
                      dict(width=1 << 27), dict(stride=-1), dict(window=-1), dict(sinks=-1), dict(starts=None, tokens=5),
                      dict(starts=None, max_query=2), dict(qt=-1), dict(qh=far), dict(oh=63), dict(ot=255), dict(ot=0),
                      dict(heads=66, tokens=(1 << 24) - 1, ot=66 * 64)])):
        for kw in cases:
            assert call(**kw) == pd.NVFP4_GEMV_ERR_BAD_SHAPE, kw


@fake_pointers
def test_misaligned():
    for call, cases in (
            (write, [dict(K=0x200000001), dict(V=0x210000001), dict(slots=0x220000004)]),
            (read, [dict(K=0x200000001), dict(y_type=2, V=0x210000002), dict(slots=0x220000004)]),
            (rope, [dict(Q=0x300000001), dict(Qo=0x320000001), dict(K=0x330000001), dict(Ko=0x350000001),
                    dict(qw=0x310000004), dict(kw=0x340000008), dict(cos_sin=0x370000004), dict(positions=0x360000004),
                    dict(cached=True, V=0x380000001), dict(cached=True, slots=0x390000004)]),
            (attend, [dict(Q=0x400000001), dict(out=0x410000001), dict(table=0x420000002), dict(lengths=0x430000001),
                      dict(starts=0x440000002)])):
        for kw in cases:
            assert call(**kw) == pd.NVFP4_GEMV_ERR_ALIGNMENT, kw


@fake_pointers
def test_aliases():
    alias = pd.NVFP4_GEMV_ERR_ALIAS
    # inputs against the cache that is written, its buffers against each other
    assert write(K=CACHE["v_codes"] + CODES - 16) == alias
    assert write(slots=CACHE["k_scales"] + SCALES - 8) == alias
    assert write(c=dict(v_codes=CACHE["k_codes"] + CODES - 16)) == alias
    assert write(c=dict(v_global=CACHE["v_scales"])) == alias
    assert read(V=0x200000000 + 4 * 128 * 2 - 2) == alias
    assert read(K=CACHE["k_codes"]) == alias
    assert read(slots=0x210000000) == alias
    # norms and rotation: in place only with the same strides; rows between each other's are apart
    assert rope(Qo=0x300000000, qot=320) == alias
    assert rope(Qo=0x300000000 + 2 * 64) == alias
    assert rope(Ko=0x320000000) == alias
    assert rope(Qo=0x330000000) == alias
    assert rope(Qo=0x360000000) == alias
    assert rope(Ko=0x370000000 + 100 * 64 * 4 - 16) == alias
    assert rope(cached=True, Qo=CACHE["k_codes"]) == alias
    assert rope(cached=True, Qo=0x380000000) == alias
    assert rope(cached=True, positions=CACHE["v_scales"]) == alias
    # attention
    assert attend(out=0x400000000) == alias
    assert attend(out=CACHE["v_codes"] + CODES - 2) == alias
    assert attend(out=0x420000000 + 28) == alias
    assert attend(out=0x430000004) == alias
    assert attend(out=0x440000008) == alias


@fake_pointers
def test_workspace():
    shape = dict(heads=4, batch=2, tokens=2, max_query=1, width=1 << 16)
    need = pd.nvfp4_kv_attention_workspace_size(pd.KvCacheStruct(**CACHE), 4, 2, 2, 1, 1 << 16)
    assert need > 0
    bad = pd.NVFP4_GEMV_ERR_WORKSPACE
    assert attend(**shape) == bad
    assert attend(**shape, ws=0x500000000, bytes=need - 1) == bad
    assert attend(**shape, ws=0x500000080, bytes=need) == pd.NVFP4_GEMV_ERR_ALIGNMENT
    # short contexts need none, invalid shapes say 0
    assert pd.nvfp4_kv_attention_workspace_size(pd.KvCacheStruct(**CACHE), 4, 2, 2, 1, 8) == 0
    assert pd.nvfp4_kv_attention_workspace_size(pd.KvCacheStruct(**CACHE), 3, 2, 2, 1, 1 << 16) == 0
    assert pd.nvfp4_kv_attention_workspace_size(pd.KvCacheStruct(**CACHE), 4, 2, 0, 1, 1 << 16) == 0
    assert pd.nvfp4_kv_attention_workspace_size(None, 4, 2, 2, 1, 1 << 16) == 0


def test_tensor_calls_refuse_host_tensors():
    t = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    codes = torch.zeros((2, 1, 16, 32), dtype=torch.uint8)
    scales = torch.zeros((2, 1, 4, 16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        pd.KvCache(codes, scales, codes, scales, head_dim=64)
    with pytest.raises(ValueError, match="GPU"):
        pd.qk_norm_rope(t, t)
    with pytest.raises(ValueError, match="GPU"):
        pd.kv_cache_write(t, t, None, None)
    with pytest.raises(ValueError, match="GPU"):
        pd.kv_attention(t, None, None, None)
