"""Refusals of the feed-forward operators without a GPU: every invalid call
returns the documented status before any HIP call, and the tensor-level calls
raise ValueError on tensors that are not on a device."""
import ctypes
import os

import pytest
import torch

import precision_decode_amd as pd
from precision_decode_amd import _binding

GPU_VISIBLE = os.path.exists("/dev/kfd")
fake_pointers = pytest.mark.skipif(GPU_VISIBLE, reason="fake device addresses are passed to launch calls "
                                   "only on machines without a GPU")
BASE = dict(X=0x100000000, W=0x200000000, sfW=0x300000000, alpha=0x400000000, bias=0x500000000,
            residual=0x600000000, Y=0x700000000)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        from precision_decode_amd import build
        build.build()
    return pd.load()


def linear(x_type=1, ldx=None, w_layout=0, ldr=None, y_type=1, ldy=None, n=4, m=32, k=128, act=0,
           ws=None, **ptr):
    p = dict(BASE, **ptr)
    args = (p["X"], x_type, k if ldx is None else ldx, p["W"], p["sfW"], w_layout, p["alpha"], p["bias"],
            p["residual"], m if ldr is None else ldr, p["Y"], y_type, m if ldy is None else ldy, n, m, k, act)
    return pd.load().nvfp4_linear_launch_ws(*args, ws, 0, None)


@fake_pointers
@pytest.mark.parametrize("name", ["X", "W", "sfW", "Y"])
def test_linear_null_pointers(name):
    assert linear(**{name: None}) == pd.NVFP4_GEMV_ERR_NULL_POINTER


@fake_pointers
@pytest.mark.parametrize("kw", [dict(x_type=2), dict(x_type=-1), dict(y_type=3), dict(y_type=-1),
                                dict(w_layout=2), dict(w_layout=-1), dict(act=5), dict(act=-1), dict(act=21),
                                dict(act=32)])
def test_linear_bad_arguments(kw):
    assert linear(**kw) == pd.NVFP4_GEMV_ERR_BAD_ARGUMENT


@fake_pointers
@pytest.mark.parametrize("kw", [dict(n=-1), dict(m=0), dict(k=0), dict(k=8), dict(k=40),
                                dict(k=(1 << 22) + 16), dict(w_layout=1, k=144), dict(ldx=127),
                                dict(ldx=(1 << 22) + 1), dict(ldy=31), dict(ldr=31), dict(ldy=(1 << 31) + 1),
                                dict(n=1 << 31), dict(m=1 << 31), dict(n=1 << 20, m=1 << 20)])
def test_linear_bad_shapes(kw):
    assert linear(**kw) == pd.NVFP4_GEMV_ERR_BAD_SHAPE


@fake_pointers
@pytest.mark.parametrize("kw", [dict(X=0x100000001), dict(Y=0x700000001), dict(residual=0x600000001),
                                dict(y_type=2, Y=0x700000002), dict(alpha=0x400000002), dict(bias=0x500000001),
                                dict(w_layout=1, W=0x200000008), dict(w_layout=1, sfW=0x300000002)])
def test_linear_misaligned(kw):
    assert linear(**kw) == pd.NVFP4_GEMV_ERR_ALIGNMENT


@fake_pointers
def test_linear_aliases():
    # the last element of each input against the first of Y, and one past it
    ends = dict(X=4 * 128 * 2, W=32 * 64, sfW=32 * 8, alpha=4, bias=32 * 4, residual=4 * 32 * 2)
    for name, size in ends.items():
        step = 4 if name in ("alpha", "bias") else 2
        assert linear(**{name: BASE["Y"] - size + step}) == pd.NVFP4_GEMV_ERR_ALIAS, name
    # in place needs the same rows: another stride is an overlap
    assert linear(residual=BASE["Y"], ldr=40) == pd.NVFP4_GEMV_ERR_ALIAS


def layer(**kw):
    f = dict(router=0x100000000, route_bias=0x110000000, W13=0x200000000, sf13=0x210000000,
             alpha13=0x220000000, W2=0x300000000, sf2=0x310000000, alpha2=0x320000000, experts=8, hidden=128,
             inter=64, topk=2, x_type=1, w_layout=0, activation=4, scoring=0, renormalize=1, routed_scale=1.0,
             reserved=0)
    f.update(kw)
    return pd.MoeLayerStruct(**f)


def moe(X=0x400000000, ldx=128, residual=0x500000000, ldr=128, Y=0x600000000, y_type=1, ldy=128, tokens=4,
        ws=0x700000000, ws_bytes=1 << 40, null_layer=False, **kw):
    return pd.load().nvfp4_moe_layer_launch_ws(None if null_layer else ctypes.byref(layer(**kw)), X, ldx,
                                               residual, ldr, Y, y_type, ldy, tokens, ws, ws_bytes, None)


@fake_pointers
def test_moe_null_pointers():
    assert moe(null_layer=True) == pd.NVFP4_GEMV_ERR_NULL_POINTER
    for name in ("X", "Y", "router", "W13", "sf13", "W2", "sf2"):
        assert moe(**{name: None}) == pd.NVFP4_GEMV_ERR_NULL_POINTER, name


@fake_pointers
@pytest.mark.parametrize("kw", [dict(x_type=2), dict(y_type=3), dict(w_layout=2), dict(activation=5),
                                dict(activation=20), dict(scoring=2), dict(scoring=-1), dict(renormalize=2),
                                dict(reserved=1)])
def test_moe_bad_arguments(kw):
    assert moe(**kw) == pd.NVFP4_GEMV_ERR_BAD_ARGUMENT


@fake_pointers
@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=65536), dict(experts=0), dict(experts=1025),
                                dict(topk=0), dict(topk=9), dict(experts=100, topk=65), dict(hidden=136),
                                dict(inter=8), dict(inter=0), dict(w_layout=1, inter=80), dict(ldx=127),
                                dict(ldy=127), dict(ldr=100), dict(experts=1024, hidden=1 << 22)])
def test_moe_bad_shapes(kw):
    if kw.get("hidden", 0) > 128:
        kw = dict(kw, ldx=kw["hidden"], ldy=kw["hidden"], ldr=kw["hidden"])
    assert moe(**kw) == pd.NVFP4_GEMV_ERR_BAD_SHAPE


@fake_pointers
@pytest.mark.parametrize("kw", [dict(X=0x400000001), dict(router=0x100000001), dict(Y=0x600000001),
                                dict(y_type=2, Y=0x600000002), dict(residual=0x500000001),
                                dict(route_bias=0x110000002), dict(alpha13=0x220000001),
                                dict(alpha2=0x320000002), dict(w_layout=1, W13=0x200000008),
                                dict(w_layout=1, sf2=0x310000001), dict(ws=0x700000080)])
def test_moe_misaligned(kw):
    assert moe(**kw) == pd.NVFP4_GEMV_ERR_ALIGNMENT


@fake_pointers
def test_moe_aliases_and_workspace():
    y = 0x600000000
    for name, size in dict(X=4 * 128 * 2, router=8 * 128 * 2, route_bias=32, W13=8 * 2 * 64 * 64,
                           sf13=8 * 2 * 64 * 8, W2=8 * 128 * 32, sf2=8 * 128 * 4, alpha13=64, alpha2=32,
                           residual=4 * 128 * 2).items():
        assert moe(**{name: y - size + 4}) == pd.NVFP4_GEMV_ERR_ALIAS, name
    assert moe(residual=y, ldr=136) == pd.NVFP4_GEMV_ERR_ALIAS
    need = pd.nvfp4_moe_layer_workspace_size(layer(), 4)
    assert need > 0
    assert moe(ws_bytes=need - 1) == pd.NVFP4_GEMV_ERR_WORKSPACE
    assert moe(ws=None) == pd.NVFP4_GEMV_ERR_WORKSPACE


def test_workspace_sizes_of_invalid_shapes_are_zero():
    assert pd.nvfp4_moe_layer_workspace_size(layer(topk=0), 4) == 0
    assert pd.nvfp4_moe_layer_workspace_size(layer(w_layout=7), 4) == 0
    assert pd.nvfp4_moe_layer_workspace_size(layer(), -1) == 0
    assert pd.nvfp4_moe_layer_workspace_size(layer(), 0) == 0
    assert pd.nvfp4_linear_workspace_size(4, 32, 40) == 0
    assert pd.load().nvfp4_moe_layer_workspace_size(None, 4) == 0


def test_tensor_calls_refuse_host_tensors_and_wrong_sizes():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pd.linear(x, u8(8, 32), u8(8, 4), 8)
    with pytest.raises(ValueError):
        pd.linear(x[0], u8(8, 32), u8(8, 4), 8)
    with pytest.raises(ValueError):
        pd.linear(x.float(), u8(8, 32), u8(8, 4), 8)
    with pytest.raises(ValueError):
        pd.MoeLayer(torch.zeros((2, 64), dtype=torch.bfloat16), u8(4, 32, 32), u8(4, 32, 4), u8(2, 64, 16),
                    u8(2, 64, 2), inter=32, topk=1)
