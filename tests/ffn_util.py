"""Inputs, calls and comparisons shared by the tests of the feed-forward operators."""
import numpy as np
import torch

import precision_decode_amd as pd

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"f16": pd.NVFP4_OUT_F16, "bf16": pd.NVFP4_OUT_BF16, "f32": pd.NVFP4_OUT_F32}
ACTS = {"none": pd.NVFP4_ACT_NONE, "relu": pd.NVFP4_ACT_RELU, "gelu": pd.NVFP4_ACT_GELU,
        "gelu_tanh": pd.NVFP4_ACT_GELU_TANH, "silu": pd.NVFP4_ACT_SILU}

# finite E4M3 codes, subnormal and negative ones among them, none above 16 in size
FINITE = np.array([c for c in range(256) if (c & 0x7F) <= 0x58], dtype=np.uint8)


def weight(rng, groups, rows, k, scale_codes=FINITE):
    codes = rng.integers(0, 256, size=(groups, rows, k // 2), dtype=np.uint8)
    return codes, scale_codes[rng.integers(0, len(scale_codes), size=(groups, rows, k // 16))]


def rounded(values, kind):
    """float64 array of the values rounded to the type ``kind``."""
    return torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).to(TYPES[kind]).double().numpy()


def device(values, kind, ld=None, offset=0):
    """Device tensor of that type holding the values, rows ``ld`` elements apart and the
    first element ``offset`` elements into its allocation; everything around is NaN."""
    v = torch.from_numpy(np.ascontiguousarray(values, dtype=np.float64)).to(TYPES[kind])
    n, c = v.shape
    ld = c if ld is None else ld
    store = torch.full((offset + n * ld + 16,), float("nan"), dtype=TYPES[kind])
    view = store[offset:offset + n * ld].view(n, ld)
    view[:, :c] = v
    return store.cuda()[offset:offset + n * ld].view(n, ld)[:, :c]


def bytes_at(values, offset=0):
    """Flat uint8 device tensor of the values, ``offset`` bytes past an aligned address."""
    flat = torch.from_numpy(np.ascontiguousarray(values, dtype=np.uint8).reshape(-1))
    store = torch.full((flat.numel() + offset + 16,), 0x7F, dtype=torch.uint8)   # NaN scales around
    store[offset:offset + flat.numel()] = flat
    return store.cuda()[offset:offset + flat.numel()]


def assert_close(got, want, err, kind, what=""):
    """|got - want| within err plus half a step of the output type; NaN, infinities and
    overflow to infinity in the same places."""
    got = got.double().cpu().numpy()
    half = torch.finfo(TYPES[kind]).eps / 2
    tiny = torch.finfo(TYPES[kind]).smallest_normal * half
    top = torch.finfo(TYPES[kind]).max
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions differ"
    fin = np.isfinite(want)
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]), f"{what}: infinities differ"
    got, want, err = got[fin], want[fin], err[fin]
    tol = err + half * (np.abs(want) + err) + tiny
    over = np.abs(want) + tol > top
    bad = ~(np.abs(got - want) <= tol) & ~over
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outputs outside tolerance, worst ratio "
                           f"{float((np.abs(got - want) / tol)[bad].max()):.3g}")
