"""The feed-forward operators on the GPU at the limits of their rules: the
longest rows and the largest values."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from ffn_util import TYPES, assert_close, rounded, weight
from oracle import ffn
from test_gpu_ffn import linear_case, moe_case

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


def one_call(rng, n, k, x, layout, gated, xv, codes, scales):
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    if layout == "packed":
        dc, ds = pd.pack_weight(dc, ds)
    got = pd.linear(torch.from_numpy(xv).to(TYPES[x]).cuda(), dc, ds, codes.shape[1], gated=gated,
                    packed=layout == "packed", out_dtype=torch.float32)
    want, err = ffn.linear(xv, codes, scales, None, None, None, "none", gated)
    assert_close(got, want, err, "f32", f"n={n} k={k} {x} {layout} gated={gated}")
    return got


@pytest.mark.parametrize("layout,k", [("row", 64), ("row", 80), ("row", 320), ("packed", 64), ("packed", 320)])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_linear_large_inputs_times_small_scales_stay_finite(n, layout, k):
    """Inputs near the largest bf16 value and scales of 2^-9: every product is below 2^122,
    so the sums stay finite, though those of 16 inputs times codes would not."""
    rng = np.random.default_rng(51 + k)
    codes, scales = weight(rng, 1, 40, k, np.array([0x01, 0x81], np.uint8))
    xv = rounded(rng.uniform(0.3, 1.0, (n, k)) * 3.3e38 * rng.choice([-1, 1], (n, k)), "bf16")
    scales[0, 3], codes[0, 3] = 0x01, 0x77        # 6 times 2^-9 everywhere
    xv[0] = np.abs(xv[0]) * 2.0 ** -2             # and all products of a sign
    assert bool(one_call(rng, n, k, "bf16", layout, False, xv, codes, scales).isfinite().all())


@pytest.mark.parametrize("layout", ["row", "packed"])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_linear_small_inputs_keep_their_bits(n, x, layout):
    """Subnormal inputs and the smallest scales: fp32 holds every product."""
    rng = np.random.default_rng(52)
    codes, scales = weight(rng, 1, 40, 192, np.array([0x01, 0x02, 0x09, 0x81], np.uint8))
    tiny = torch.finfo(TYPES[x]).smallest_normal
    xv = rounded(rng.uniform(-2.0, 2.0, (n, 192)) * tiny, x)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    if layout == "packed":
        dc, ds = pd.pack_weight(dc, ds)
    up = 2.0 ** 120 if x == "bf16" else 1.0
    got = pd.linear(torch.from_numpy(xv).to(TYPES[x]).cuda(), dc, ds, 40, packed=layout == "packed",
                    alpha=torch.tensor([up], device="cuda"), out_dtype=torch.float32)
    want, err = ffn.linear(xv, codes, scales, np.array([up]), None, None, "none", False)
    # besides, an addition in fp32's subnormals is off by up to half of 2^-149
    assert_close(got, want, err + 192 * 2.0 ** -150 * up, "f32", f"n={n} {x} {layout}")


@pytest.mark.parametrize("layout,k", [("row", 320), ("row", 336), ("packed", 320)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_special_values_of_one_token(x, gated, layout, k):
    """One token has a kernel of its own: NaN scales stay in their rows, an infinite input
    gives infinities and NaN by the weights' signs and zeros."""
    rng = np.random.default_rng(53)
    codes, scales = weight(rng, 2 if gated else 1, 40, k)
    scales[0, 5, 3] = 0x7F
    codes[0, 7], scales[0, 9] = 0, 0
    xv = rounded(rng.standard_normal((1, k)), x)
    got = one_call(rng, 1, k, x, layout, gated, xv, codes, scales)
    assert bool(got[:, 5].isnan().all()) and int(got.isnan().sum()) == 1
    xv[0, 100] = np.inf
    got = one_call(rng, 1, k, x, layout, gated, xv, codes, scales)
    assert bool(got[:, [5, 7, 9]].isnan().all())
    xv[0] = 0.0
    got = one_call(rng, 1, k, x, layout, gated, xv, codes, scales)
    assert bool((got[0, [0, 1, 7, 9]] == 0).all())


@pytest.mark.parametrize("n", [1, 3, 40, 800])
def test_linear_between_columns_of_one_matrix(n):
    """X, the residual and Y as column ranges of one matrix."""
    rng = np.random.default_rng(54)
    codes, scales = weight(rng, 1, 80, 128)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    both = torch.from_numpy(rng.standard_normal((n, 128 + 80 + 80 + 8))).to(torch.bfloat16).cuda()
    before = both.clone()
    al = torch.tensor([0.01], device="cuda")
    want = pd.linear(both[:, 88:216].contiguous(), dc, ds, 80, alpha=al, residual=both[:, 216:].contiguous()[:, :80])
    pd.linear(both[:, 88:216], dc, ds, 80, alpha=al, residual=both[:, 216:296], out=both[:, 4:84])
    assert torch.equal(both[:, 4:84], want)
    before[:, 4:84] = want
    assert torch.equal(both, before)
    if n > 1:   # a column too far
        with pytest.raises(pd.Nvfp4GemvError) as e:
            pd.linear(both[:, 88:216], dc, ds, 80, out=both[:, 9:89])
        assert e.value.status == pd.NVFP4_GEMV_ERR_ALIAS


def test_moe_layer_between_columns_of_one_matrix():
    rng = np.random.default_rng(55)
    c13, s13 = weight(rng, 12, 64, 128)
    c2, s2 = weight(rng, 6, 128, 64)
    dev = lambda v: torch.from_numpy(v).cuda()
    layer = pd.MoeLayer(dev(rng.standard_normal((6, 128))).to(torch.bfloat16), dev(c13), dev(s13), dev(c2), dev(s2),
                        inter=64, topk=2, alpha13=torch.full((6, 2), 0.01, device="cuda"))
    for n in (1, 5, 50):
        both = dev(rng.standard_normal((n, 256))).to(torch.bfloat16)
        x = both[:, :128].clone()
        want = pd.moe_layer(x, layer)
        pd.moe_layer(both[:, :128], layer, out=both[:, 128:])
        assert torch.equal(both[:, 128:], want) and torch.equal(both[:, :128], x)


def test_linear_large_unaligned_input():
    """More pieces of X than the copy to aligned rows has threads."""
    n, m, k = 40000, 2050, 4096
    rng = np.random.default_rng(56)
    codes, scales = weight(rng, 1, m, k)
    dc, ds = pd.pack_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = torch.randint(-8, 9, (n, k + 1), device="cuda").to(torch.bfloat16)
    got = pd.linear(x[:, 1:], dc, ds, m, packed=True, out_dtype=torch.float32)
    want = pd.linear(x[:, 1:].contiguous(), dc, ds, m, packed=True, out_dtype=torch.float32)
    assert torch.equal(got, want)
    for t in (0, 1, 16384, n - 1):
        w, err = ffn.linear(x[t:t + 1, 1:].double().cpu().numpy(), codes, scales)
        assert_close(got[t:t + 1], w, err, "f32", f"token {t}")


@pytest.mark.parametrize("n,m,k,gated", [(1, 40, 65536, False), (2, 40, 65536, False), (5, 41, 65536, True),
                                         (16, 40, 65536, False), (1, 100, 16400, False), (8, 100, 16400, True)])
def test_linear_few_tokens_with_k_split(n, m, k, gated):
    """Long rows and few of them: the stream kernel's workgroups share K."""
    for layout in (("row",) if k % 64 else ("row", "packed")):
        for x in ("bf16", "f16"):
            linear_case(np.random.default_rng(57 + n), n, m, k, x=x, y="f32", gated=gated, act="silu", bias=True,
                        residual="apart", layout=layout, ws=True, ldy=m + 1)


def test_linear_more_outputs_than_31_bits():
    """n m of 4 10^9: the first and last tokens against a call of their own."""
    n, m, k = 262000, 16000, 64
    rng = np.random.default_rng(58)
    codes, scales = weight(rng, 1, m, k)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    x = torch.randint(-8, 9, (n, k), device="cuda").to(torch.float16)
    al = torch.tensor([0.01], device="cuda")
    y = pd.linear(x, dc, ds, m, alpha=al, activation="relu")
    for first in (0, 134200, n - 300):    # the second: around element 2^31
        part = pd.linear(x[first:first + 300], dc, ds, m, alpha=al, activation="relu")
        assert torch.equal(y[first:first + 300], part)
    want, err = ffn.linear(x[n - 1:].double().cpu().numpy(), codes, scales, al.cpu().numpy(), act="relu")
    assert_close(y[n - 1:], want, err, "f16")
    del y


@pytest.mark.parametrize("packed", [False, True])
def test_moe_layer_weights_past_4_gb(packed):
    """300 experts of 7168 x 2048, 6.6 GB of gate and up codes: the last experts' outputs
    against a layer of these alone."""
    experts, hidden, inter, last = 300, 7168, 2048, 6
    g = torch.Generator(device="cuda").manual_seed(59)
    byte = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)
    scale = lambda *s: torch.randint(0x20, 0x48, s, dtype=torch.uint8, device="cuda", generator=g)
    c13, s13 = byte(2 * experts, inter, hidden // 2), scale(2 * experts, inter, hidden // 16)
    c2, s2 = byte(experts, hidden, inter // 2), scale(experts, hidden, inter // 16)
    a13, a2 = torch.full((experts, 2), 0.01, device="cuda"), torch.full((experts,), 0.01, device="cuda")
    bias = torch.zeros(experts, device="cuda")
    bias[:experts - last] = -float("inf")
    router = torch.randn((experts, hidden), device="cuda", generator=g).to(torch.bfloat16)
    pack = pd.pack_weight if packed else lambda c, s: (c.contiguous(), s.contiguous())
    whole = pd.MoeLayer(router, *pack(c13, s13), *pack(c2, s2), inter=inter, topk=3, alpha13=a13, alpha2=a2,
                        route_bias=bias, scoring="sigmoid", packed=packed)
    f = experts - last
    alone = pd.MoeLayer(router[f:].contiguous(), *pack(c13[2 * f:], s13[2 * f:]), *pack(c2[f:], s2[f:]), inter=inter,
                        topk=3, alpha13=a13[f:], alpha2=a2[f:], route_bias=bias[f:], scoring="sigmoid", packed=packed)
    for tokens in (1, 24):
        x = torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16)
        got, want = (pd.moe_layer(x, v, out_dtype=torch.float32) for v in (whole, alone))
        # sums of other workgroup shapes may round in another order
        assert float((got - want).abs().max()) <= 1e-5 * float(want.abs().max())
        assert bool(got.isfinite().all()) and float(want.abs().max()) > 0


@pytest.mark.parametrize("experts,topk,hidden,inter", [(1024, 64, 16, 16), (70, 33, 128, 64), (100, 16, 128, 64),
                                                       (9, 9, 64, 64)])
def test_moe_layer_few_tokens_many_experts_each(experts, topk, hidden, inter):
    """More experts a token than the down product's workgroup has waves."""
    rng = np.random.default_rng(60 + topk)
    for tokens in (1, 2):
        moe_case(rng, tokens, experts, topk, hidden, inter, residual="apart")
        moe_case(rng, tokens, experts, topk, hidden, inter, x="f16", y="f32", scoring="sigmoid", route_bias=True)


def test_moe_layer_slots_past_2_gb():
    """h of more than 2^31 bytes a plane, past the stream kernel's offsets: against calls of
    fewer tokens."""
    tokens, experts, topk, hidden, inter = 65535, 16, 8, 64, 2064
    rng = np.random.default_rng(61)
    c13, s13 = weight(rng, 2 * experts, inter, hidden)
    c2, s2 = weight(rng, experts, hidden, inter)
    dev = lambda v: torch.from_numpy(v).cuda()
    layer = pd.MoeLayer(dev(rng.standard_normal((experts, hidden))).to(torch.bfloat16), dev(c13), dev(s13), dev(c2), dev(s2),
                        inter=inter, topk=topk, alpha13=torch.full((experts, 2), 0.01, device="cuda"),
                        alpha2=torch.full((experts,), 0.01, device="cuda"))
    assert tokens * topk * inter * 2 > 1 << 31
    x = dev(rng.standard_normal((tokens, hidden))).to(torch.bfloat16)
    got = torch.empty((tokens, hidden), dtype=torch.float32, device="cuda")
    need = pd.nvfp4_moe_layer_workspace_size(layer, tokens)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")    # not the library's, which would keep it
    pd.nvfp4_moe_layer_launch_ws(layer, x, hidden, None, hidden, got, pd.NVFP4_OUT_F32, hidden, tokens, ws, need)
    for first in range(0, tokens, 16384):
        want = pd.moe_layer(x[first:first + 16384], layer, out_dtype=torch.float32)
        part = got[first:first + 16384]
        assert float((part - want).abs().max()) <= 1e-5 * float(want.abs().max()), first
    del ws
