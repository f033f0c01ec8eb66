"""Tensors of several GPUs in the feed-forward tensor calls, with fake tensors
(no GPU): tensors of another GPU than x are refused, and the C call is made
with x's GPU current, on its stream."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import precision_decode_amd as pd
from precision_decode_amd import _binding

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a machine without a GPU: none is called")


@pytest.fixture
def fake():
    """empty(shape, dtype, gpu) and the C calls made: (name, current GPU, stream handle)."""
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        yield lambda shape, dtype, gpu: torch.empty(shape, dtype=dtype, device=f"cuda:{gpu}")


class Runtime:
    """A stand-in for the library and for torch's current GPU."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        runtime = self

        class Current:
            def __init__(self, device):
                self.device = device

            def __enter__(self):
                self.before, runtime.current = runtime.current, self.device

            def __exit__(self, *_):
                runtime.current = self.before

        class Library:
            def __getattr__(self, name):
                def call(*args):
                    runtime.calls.append((name, runtime.current, args[-1]))
                    return 0
                return call

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                runtime.on.append(self.stream)

            def __exit__(self, *_):
                pass

        self.on = []
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, torch.device(device).index))
        monkeypatch.setattr(torch.cuda, "device", Current)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
        monkeypatch.setattr(_binding, "load", lambda: Library())


U8, BF16, F32 = torch.uint8, torch.bfloat16, torch.float32


def linear_tensors(fake, gpu):
    return dict(x=fake((2, 64), BF16, gpu), codes=fake((8, 32), U8, gpu), scales=fake((8, 4), U8, gpu),
                alpha=fake((1,), F32, gpu), bias=fake((8,), F32, gpu), residual=fake((2, 8), BF16, gpu),
                out=fake((2, 8), BF16, gpu))


def layer_tensors(fake, gpu):
    return dict(router=fake((2, 64), BF16, gpu), codes13=fake((4, 32, 32), U8, gpu),
                scales13=fake((4, 32, 4), U8, gpu), codes2=fake((2, 64, 16), U8, gpu),
                scales2=fake((2, 64, 2), U8, gpu), alpha13=fake((2, 2), F32, gpu), alpha2=fake((2,), F32, gpu),
                route_bias=fake((2,), F32, gpu))


@pytest.mark.parametrize("other", ["codes", "scales", "alpha", "bias", "residual", "out"])
def test_linear_refuses_tensors_of_another_gpu(fake, monkeypatch, other):
    runtime = Runtime(monkeypatch)
    t = linear_tensors(fake, 0)
    t[other] = linear_tensors(fake, 1)[other]
    with pytest.raises(ValueError, match="GPU"):
        pd.linear(m=8, **t)
    assert not runtime.calls


@pytest.mark.parametrize("other", ["codes13", "scales13", "codes2", "scales2", "alpha13", "alpha2", "route_bias"])
def test_moe_layer_refuses_weights_of_another_gpu(fake, other):
    t = layer_tensors(fake, 0)
    t[other] = layer_tensors(fake, 1)[other]
    with pytest.raises(ValueError, match="GPU"):
        pd.MoeLayer(inter=32, topk=1, **t)


@pytest.mark.parametrize("other", ["x", "residual", "out"])
def test_moe_layer_refuses_tokens_of_another_gpu(fake, monkeypatch, other):
    runtime = Runtime(monkeypatch)
    layer = pd.MoeLayer(inter=32, topk=1, **layer_tensors(fake, 0))
    t = {name: fake((2, 64), BF16, 1 if name == other else 0) for name in ("x", "residual", "out")}
    with pytest.raises(ValueError, match="GPU"):
        pd.moe_layer(layer=layer, **t)
    assert not runtime.calls


@pytest.mark.parametrize("gpu", [0, 1])
def test_calls_are_made_on_the_tensors_gpu(fake, monkeypatch, gpu):
    runtime = Runtime(monkeypatch)
    pd.linear(m=8, **linear_tensors(fake, gpu))
    layer = pd.MoeLayer(inter=32, topk=1, **layer_tensors(fake, gpu))
    x = fake((2, 64), BF16, gpu)
    assert pd.moe_layer(x, layer, out=fake((2, 64), BF16, gpu), stream=7).get_device() == gpu
    assert runtime.calls == [("nvfp4_linear_launch", gpu, 100 + gpu), ("nvfp4_moe_layer_launch", gpu, 7)]
    assert runtime.current == 0


def test_outputs_are_allocated_on_a_stream_given_as_a_handle(fake, monkeypatch):
    runtime = Runtime(monkeypatch)
    t = linear_tensors(fake, 0)
    del t["out"]
    pd.linear(m=8, stream=0x7000, **t)
    layer = pd.MoeLayer(inter=32, topk=1, **layer_tensors(fake, 0))
    pd.moe_layer(fake((2, 64), BF16, 0), layer, stream=0x7040)
    pd.linear(m=8, **t)
    assert runtime.on == [(0x7000, 0), (0x7040, 0)]   # handle and GPU
    assert [c[2] for c in runtime.calls] == [0x7000, 0x7040, 100]
