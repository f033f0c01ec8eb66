"""Streams of the feed-forward tensor calls on the GPU: an output that the call
allocates belongs to the stream that writes it, also where that is given as a
handle."""
import pytest
import torch

import precision_decode_amd as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


@pytest.mark.parametrize("handle", [False, True])
def test_output_memory_is_of_the_writing_stream(handle):
    x = torch.ones((300, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((4100, 32), 0x22, dtype=torch.uint8, device="cuda")     # 1.0
    scales = torch.full((4100, 4), 0x38, dtype=torch.uint8, device="cuda")     # 1.0
    s = torch.cuda.Stream()
    pd.linear(x, codes, scales, 4100)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free = torch.empty((300, 4100), dtype=torch.bfloat16, device="cuda").data_ptr()   # freed at once
    y = pd.linear(x, codes, scales, 4100)
    assert y.data_ptr() == free        # the current stream may have it
    del y
    torch.cuda.synchronize()
    y = pd.linear(x, codes, scales, 4100, stream=s.cuda_stream if handle else s)
    s.synchronize()
    assert y.data_ptr() != free        # another stream may not
    assert bool((y == 64.0).all())


def test_default_stream_as_a_handle():
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((40, 32), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 4), 0x38, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    y = pd.linear(x, codes, scales, 40, stream=0)
    torch.cuda.synchronize()
    assert bool((y == 64.0).all())
