"""Tensor calls of the attention operators with fake tensors (no GPU): tensors of
another GPU, another shape or type than the call's are refused, and the C call is
made with the tensors' GPU current, on its stream."""
import pytest
import torch

import precision_decode_amd as pd
from test_ffn_devices import BF16, F32, U8, Runtime, fake  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a machine without a GPU: none is called")
I32, I64 = torch.int32, torch.int64


def cache_tensors(fake, gpu):
    return dict(k_codes=fake((8, 2, 16, 32), U8, gpu), k_scales=fake((8, 2, 4, 16), U8, gpu),
                v_codes=fake((8, 2, 16, 32), U8, gpu), v_scales=fake((8, 2, 4, 16), U8, gpu),
                k_global=fake((2,), F32, gpu), v_global=fake((2,), F32, gpu))


def cache(fake, gpu):
    return pd.KvCache(head_dim=64, **cache_tensors(fake, gpu))


def write_tensors(fake, gpu):
    return dict(k=fake((3, 2, 64), BF16, gpu), v=fake((3, 2, 64), BF16, gpu), slots=fake((3,), I64, gpu),
                cache=cache(fake, gpu))


def rope_tensors(fake, gpu):
    return dict(q=fake((3, 4, 64), BF16, gpu), k=fake((3, 2, 64), BF16, gpu), positions=fake((3,), I64, gpu),
                cos_sin=fake((9, 64), F32, gpu), q_weight=fake((64,), F32, gpu), k_weight=fake((64,), F32, gpu),
                q_out=fake((3, 4, 64), BF16, gpu))


def attention_tensors(fake, gpu):
    return dict(q=fake((4, 4, 64), BF16, gpu), cache=cache(fake, gpu), block_table=fake((2, 4), I32, gpu),
                lengths=fake((2,), I32, gpu), query_starts=fake((3,), I32, gpu), out=fake((4, 4, 64), BF16, gpu))


CALLS = [(pd.kv_cache_write, write_tensors), (pd.qk_norm_rope, rope_tensors), (pd.kv_attention, attention_tensors),
         (pd.qk_norm_rope, lambda f, gpu: dict(rope_tensors(f, gpu), v=f((3, 2, 64), BF16, gpu),
                                               cache=cache(f, gpu), slots=f((3,), I64, gpu)))]


@pytest.mark.parametrize("call,tensors", CALLS)
def test_tensors_of_another_gpu(fake, monkeypatch, call, tensors):  # noqa: F811
    runtime = Runtime(monkeypatch)
    for other in tensors(fake, 0):
        t = tensors(fake, 0)
        t[other] = tensors(fake, 1)[other]
        with pytest.raises(ValueError, match="GPU"):
            call(**t)
    assert not runtime.calls


def test_cache_of_several_gpus_or_of_other_shapes(fake):  # noqa: F811
    for other in cache_tensors(fake, 0):
        t = cache_tensors(fake, 0)
        t[other] = cache_tensors(fake, 1)[other]
        with pytest.raises(ValueError, match="GPU"):
            pd.KvCache(head_dim=64, **t)
    for name, shape in (("k_scales", (8, 2, 16, 4)), ("v_scales", (8, 2, 4, 8)), ("v_codes", (7, 2, 16, 32)),
                        ("k_codes", (8, 2, 16, 64)), ("k_global", (3,))):
        with pytest.raises(ValueError):
            pd.KvCache(head_dim=64, **dict(cache_tensors(fake, 0), **{name: fake(shape, U8 if len(shape) > 1 else F32, 0)}))
    with pytest.raises(ValueError):
        pd.KvCache(head_dim=128, **cache_tensors(fake, 0))


@pytest.mark.parametrize("call,tensors,bad", [
    (pd.kv_cache_write, write_tensors, dict(k=((3, 128), BF16), v=((3, 2, 64), torch.float16), slots=((2,), I64))),
    (pd.kv_cache_write, write_tensors, dict(k=((3, 2, 64), F32), v=((2, 2, 64), BF16), slots=((3,), I32))),
    (pd.qk_norm_rope, rope_tensors, dict(q=((3, 256), BF16), k=((3, 2, 32), BF16), positions=((3,), I32),
                                         cos_sin=((9, 64), BF16), q_weight=((32,), F32), q_out=((3, 4, 64), F32))),
    (pd.kv_attention, attention_tensors, dict(q=((4, 4, 32), BF16), block_table=((2, 4), I64), lengths=((3,), I32),
                                              query_starts=((2,), I32), out=((4, 2, 64), BF16)))])
def test_other_shapes_and_types(fake, monkeypatch, call, tensors, bad):  # noqa: F811
    runtime = Runtime(monkeypatch)
    for name, (shape, dtype) in bad.items():
        with pytest.raises(ValueError):
            call(**dict(tensors(fake, 0), **{name: fake(shape, dtype, 0)}))
    assert not runtime.calls


def test_arguments_that_go_together(fake, monkeypatch):  # noqa: F811
    runtime = Runtime(monkeypatch)
    t = rope_tensors(fake, 0)
    v, slots, c = fake((3, 2, 64), BF16, 0), fake((3,), I64, 0), cache(fake, 0)
    for kw in (dict(v=v), dict(cache=c), dict(v=v, cache=c), dict(slots=slots),
               dict(v=v, cache=c, slots=slots, k_out=fake((3, 2, 64), BF16, 0)), dict(positions=None)):
        with pytest.raises(ValueError):
            pd.qk_norm_rope(**dict(t, **kw))
    with pytest.raises(ValueError, match="query_starts"):
        pd.kv_attention(**dict(attention_tensors(fake, 0), query_starts=None, q=fake((3, 4, 64), BF16, 0), out=None))
    # rows with a stride of their own elements
    with pytest.raises(ValueError, match="contiguous"):
        pd.kv_attention(**dict(attention_tensors(fake, 0), q=fake((4, 4, 128), BF16, 0)[:, :, ::2]))
    assert not runtime.calls


@pytest.mark.parametrize("gpu", [0, 1])
def test_calls_are_made_on_the_tensors_gpu(fake, monkeypatch, gpu):  # noqa: F811
    runtime = Runtime(monkeypatch)
    for call, tensors in CALLS:
        call(**tensors(fake, gpu))
    k, _ = pd.kv_cache_read(cache(fake, gpu), fake((3,), I64, gpu), stream=7)
    assert k.get_device() == gpu and runtime.on == [(7, gpu)] * 2
    assert runtime.calls == [("nvfp4_kv_write_launch", gpu, 100 + gpu), ("nvfp4_qk_norm_rope_launch", gpu, 100 + gpu),
                             ("nvfp4_kv_attention_launch", gpu, 100 + gpu),
                             ("nvfp4_qk_norm_rope_launch", gpu, 100 + gpu), ("nvfp4_kv_read_launch", gpu, 7)]
    assert runtime.current == 0
