"""Tensors of several GPUs in the GEMV, quantiser and packing tensor calls,
with fake tensors (no GPU): tensors of another GPU are refused, and the C call
is made with the tensors' GPU current."""
import pytest
import torch

import precision_decode_amd as pd
from precision_decode_amd import _binding
from test_ffn_devices import BF16, F32, U8, Runtime, fake  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a machine without a GPU: none is called")


@pytest.fixture
def runtime(monkeypatch):
    r = Runtime(monkeypatch)
    monkeypatch.setattr(_binding, "_stream", lambda s: 100 + r.current if s is None else s)
    return r


def gemv_tensors(fake, gpu):  # noqa: F811
    return dict(A_packed=fake((1, 8, 32), U8, gpu), sfA=fake((1, 8, 4), U8, gpu), x_packed=fake((1, 32), U8, gpu),
                sfx=fake((1, 4), U8, gpu), alpha=fake((1,), F32, gpu), out=fake((1, 8), torch.float16, gpu))


@pytest.mark.parametrize("other", ["sfA", "x_packed", "sfx", "alpha", "out"])
def test_gemv_refuses_tensors_of_another_gpu(fake, runtime, other):  # noqa: F811
    t = gemv_tensors(fake, 0)
    t[other] = gemv_tensors(fake, 1)[other]
    with pytest.raises(ValueError, match="GPU"):
        pd.gemv(**t)
    assert not runtime.calls


def test_quantiser_and_packing_refuse_tensors_of_another_gpu(fake, runtime):  # noqa: F811
    with pytest.raises(ValueError, match="GPU"):
        pd.quantize_activation(fake((2, 64), BF16, 0), fake((1,), F32, 1))
    with pytest.raises(ValueError, match="GPU"):
        pd.pack_weight(fake((8, 32), U8, 0), fake((8, 4), U8, 1))
    assert not [c for c in runtime.calls if "sizes" not in c[0]]


@pytest.mark.parametrize("gpu", [0, 1])
def test_calls_are_made_on_the_tensors_gpu(fake, runtime, gpu):  # noqa: F811
    pd.gemv(**gemv_tensors(fake, gpu))
    pd.quantize_activation(fake((2, 64), BF16, gpu), fake((1,), F32, gpu))
    pd.pack_weight(fake((8, 32), U8, gpu), fake((8, 4), U8, gpu), stream=7)
    calls = [c for c in runtime.calls if "sizes" not in c[0]]
    assert calls == [("nvfp4_gemv_launch", gpu, 100 + gpu), ("nvfp4_quantize_activation", gpu, 100 + gpu),
                     ("nvfp4_mma_pack_weight", gpu, 7)]
    assert runtime.current == 0


def test_outputs_are_allocated_on_a_stream_given_as_a_handle(fake, runtime):  # noqa: F811
    t = gemv_tensors(fake, 0)
    del t["out"]
    pd.gemv(stream=0x7000, **t)
    pd.quantize_activation(fake((2, 64), BF16, 0), fake((1,), F32, 0), stream=0x7040)
    pd.pack_weight(fake((8, 32), U8, 0), fake((8, 4), U8, 0), stream=0x7080)
    assert runtime.on == [(0x7000, 0), (0x7040, 0), (0x7040, 0), (0x7080, 0), (0x7080, 0)]
