"""The feed-forward operators on the GPU at the limits of their rules: the
longest rows and the largest values."""
import pytest
import torch

import precision_decode_amd as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()
    yield
    torch.cuda.empty_cache()


def test_linear_longest_rows_keep_their_last_elements():
    """Rows of 2^22 elements, as far apart: 256 of them end at byte 2^31 from the first,
    where a block of 256 tokens still reads its last piece.  Weights are 1, so an output is
    the number of ones in its row, exactly; every row has its ones at its end."""
    n, m, k = 256, 8192, 1 << 22
    x = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    x[:, k - 16:] = 1.0
    codes = torch.full((m, k // 2), 0x22, dtype=torch.uint8, device="cuda")      # 1.0 twice
    scales = torch.full((m, k // 16), 0x38, dtype=torch.uint8, device="cuda")    # 1.0
    y = pd.linear(x, codes, scales, m, out_dtype=torch.float32)
    assert bool((y == 16.0).all())
    x[n - 1, k - 1] = float("nan")
    y = pd.linear(x, codes, scales, m, out_dtype=torch.float32)
    assert bool(y[n - 1].isnan().all()) and bool((y[:n - 1] == 16.0).all())
