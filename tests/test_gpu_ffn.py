"""The linear layer and the mixture-of-experts layer on the GPU against the
float64 oracle, with the tolerances that oracle/ffn.py derives: sizes from one
up, ragged and odd ones, every type, layout, alignment and activation, strided
operands, special values, empty calls, experts without tokens, ties, graphs
and streams."""
import itertools

import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from ffn_util import ACTS, CODES, FINITE, assert_close, bytes_at, device, rounded, weight
from oracle import ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


# ---------------------------------------------------------------- linear
def linear_case(rng, n, m, k, x="bf16", y=None, act="none", gated=False, bias=False, residual=None,
                layout="row", ldx=0, xoff=0, ldy=0, woff=0, soff=0, scale_codes=FINITE, alpha=True,
                edit=None, ws=False):
    """One call and its check; returns the output tensor."""
    y = y or x
    groups = 2 if gated else 1
    codes, scales = weight(rng, groups, m, k, scale_codes)
    xv = rounded(rng.standard_normal((n, k)), x)
    if edit:
        edit(xv, codes, scales)
    al = (rng.uniform(0.5, 2, groups) / np.sqrt(k) / 8).astype(np.float32) if alpha else None
    bv = rng.standard_normal(groups * m).astype(np.float32) if bias else None
    rv = rounded(rng.standard_normal((n, m)), y) if residual else None
    dx = device(xv, x, ldx or k, xoff)
    if layout == "packed":
        dw, ds = pd.pack_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    else:
        dw, ds = bytes_at(codes, woff), bytes_at(scales, soff)
    dal = None if al is None else torch.from_numpy(al).cuda()
    db = None if bv is None else torch.from_numpy(bv).cuda()
    ld = ldy or m
    if residual == "in place":
        dr = out = device(rv, y, ld)
    else:
        out = device(np.full((n, m), 7.0), y, ld)
        dr = None if rv is None else device(rv, y, ld + 3)
    base = out._base if out._base is not None else out
    before = base.clone()
    code = ACTS[act] | (pd.NVFP4_ACT_GATED if gated else 0)
    args = (dx, CODES[x], ldx or k, dw, ds, pd.NVFP4_W_PACKED if layout == "packed" else pd.NVFP4_W_ROW_MAJOR,
            dal, db, dr, ld if residual == "in place" else ld + 3, out, CODES[y], ld, n, m, k, code)
    if ws:
        need = pd.nvfp4_linear_workspace_size(n, m, k, code)
        w = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
        pd.nvfp4_linear_launch_ws(*args, w, need)
        torch.cuda.synchronize()
        assert bool((w[need:] == 0x7F).all()), "wrote past the workspace"
    else:
        pd.nvfp4_linear_launch(*args)
    torch.cuda.synchronize()
    want, err = ffn.linear(xv, codes, scales, al, bv, rv, act, gated)
    what = f"n={n} m={m} k={k} {x}->{y} {act} gated={gated} {layout}"
    assert_close(out, want, err, y, what)
    # nothing but the m elements of every row is written
    mask = torch.ones_like(base, dtype=torch.bool)
    mask.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(False)
    a, b = base[mask], before[mask]
    assert bool(((a == b) | (a.isnan() & b.isnan())).all()), what + ": wrote outside its rows"
    return out


@pytest.mark.parametrize("layout", ["row", "packed"])
@pytest.mark.parametrize("n,m,k", [(1, 1, 64), (1, 16, 64), (2, 17, 128), (3, 100, 256), (4, 64, 320),
                                   (5, 33, 512), (8, 48, 1088), (9, 31, 832), (16, 160, 2048), (17, 15, 704),
                                   (31, 65, 1024), (33, 129, 768), (64, 96, 576), (65, 300, 1280),
                                   (128, 130, 640), (129, 257, 448), (200, 128, 2176), (257, 513, 384),
                                   (300, 40, 4160), (513, 272, 192)])
def test_linear_sizes(n, m, k, layout):
    print(f"linear {n} {m} {k} {layout}", flush=True)
    rng = np.random.default_rng(n * 1000003 + m * 1009 + k)
    for x, gated in itertools.product(("bf16", "f16"), (False, True)):
        linear_case(rng, n, m, k, x=x, gated=gated, layout=layout)


@pytest.mark.parametrize("n,m,k", [(5377, 2050, 320), (2817, 2050, 320), (1409, 2050, 832), (769, 2050, 1088), (385, 2050, 576),
                                   (97, 2050, 1024), (40, 520, 8192), (17, 80, 16384), (48, 7000, 448)])
def test_linear_every_tile_shape(n, m, k):
    """Weights that take each shape of the tile kernel, largest tiles first, then K split."""
    print(f"linear tiles {n} {m} {k}", flush=True)
    rng = np.random.default_rng(n)
    ld = max(m, 2048) // 8 * 8 + 8   # whole 16-byte pieces
    linear_case(rng, n, m, k, x="bf16", bias=True, residual="in place", act="silu", layout="packed", ldy=ld)
    linear_case(rng, n, m, k, x="f16", y="f32", act="gelu", bias=True, residual="in place", ldx=k + 8, ldy=ld + 4)
    linear_case(rng, n, (m + 1) // 2, k, x="f16", gated=True, bias=True, act="gelu_tanh", layout="packed", ldy=ld + 3)
    linear_case(rng, n, (m + 1) // 2, k, x="bf16", y="f32", gated=True, residual="apart", act="relu", ldx=k + 1)


@pytest.mark.parametrize("n,m,k", [(1, 8200, 320), (2, 8193, 448), (4, 8200, 80), (7, 8230, 640), (16, 8209, 576)])
def test_linear_few_tokens_many_rows(n, m, k):
    """Enough row tiles for the smaller workgroups of the stream kernel."""
    rng = np.random.default_rng(n + 100)
    linear_case(rng, n, m, k, x="bf16", act="silu", bias=True, layout="row" if k % 64 else "packed")
    linear_case(rng, n, m, k, x="f16", y="f32", gated=True, act="gelu", residual="apart", ldx=k + 1, xoff=1)


def test_linear_rows_four_million_elements_apart():
    """Token offsets past 32 bits."""
    rng = np.random.default_rng(18)
    codes, scales = weight(rng, 1, 48, 64)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    far = torch.zeros((300, 1 << 22), dtype=torch.bfloat16, device="cuda")[:, 64:128]
    for n in (5, 40, 300):
        x = torch.from_numpy(rng.standard_normal((n, 64))).to(torch.bfloat16).cuda()
        far[:n] = x
        assert torch.equal(pd.linear(far[:n], dc, ds, 48), pd.linear(x, dc, ds, 48))


@pytest.mark.parametrize("k", [16, 32, 48, 80, 112, 144, 240, 272, 1040, 2064])
def test_linear_row_major_k_of_whole_blocks(k):
    rng = np.random.default_rng(k)
    for n, m in ((1, 5), (7, 40), (40, 70)):
        linear_case(rng, n, m, k, x="f16", y="f32", bias=True)
        linear_case(rng, n, m, k, x="bf16", gated=True, act="silu")


@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", list(ACTS))
def test_linear_epilogues(act, y):
    rng = np.random.default_rng(11)
    for gated, bias, residual in itertools.product((False, True), (False, True), (None, "apart", "in place")):
        for n, layout in ((3, "packed"), (70, "row")):
            linear_case(rng, n, 83, 320, y=y, act=act, gated=gated, bias=bias, residual=residual,
                        layout=layout, ldy=90)


@pytest.mark.parametrize("n", [1, 6, 40, 150])
def test_linear_strides_and_alignment(n):
    rng = np.random.default_rng(12 + n)
    for ldx, xoff in ((328, 0), (321, 0), (325, 3), (320, 1), (336, 8)):
        linear_case(rng, n, 50, 320, ldx=ldx, xoff=xoff, layout="packed", ws=True)
        linear_case(rng, n, 50, 320, ldx=ldx, xoff=xoff, x="f16", gated=True, ws=True)
    for woff, soff in ((1, 0), (4, 1), (8, 2), (0, 3), (16, 4)):
        linear_case(rng, n, 50, 320, woff=woff, soff=soff)


def test_linear_without_alpha():
    linear_case(np.random.default_rng(13), 4, 30, 128, alpha=False, y="f32")


@pytest.mark.parametrize("n", [2, 40, 300])
@pytest.mark.parametrize("layout", ["row", "packed"])
def test_linear_special_values_stay_in_their_row_and_token(n, layout):
    def edit(xv, codes, scales):
        scales[0, 5, 3] = 0x7F            # NaN scale: weight row 5
        xv[1, 100] = np.inf               # infinite input: token 1 (inf or NaN by the weights' signs)
        codes[0, 7] = 0                   # a row of zeros (times infinity: NaN)
        xv[0] = 0.0                       # a token of zeros
        scales[0, 9] = 0                  # a row of zero scales

    out = linear_case(np.random.default_rng(14), n, 40, 320, layout=layout, edit=edit, y="f32")
    assert bool(out[:, 5].isnan().all())
    assert bool((out[0, [0, 1, 7, 9]] == 0).all())


def test_linear_large_values_overflow_to_infinity_only():
    linear_case(np.random.default_rng(15), 3, 20, 64, x="bf16", y="f16", alpha=False,
                edit=lambda xv, c, s: xv.__imul__(4096.0))


def test_linear_empty_call_does_nothing():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((8, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((8, 4), dtype=torch.uint8, device="cuda")
    assert tuple(pd.linear(x, codes, scales, 8).shape) == (0, 8)


def test_linear_tensor_call_matches_c_call():
    rng = np.random.default_rng(16)
    codes, scales = weight(rng, 2, 48, 256)
    x = torch.from_numpy(rng.standard_normal((6, 300))).to(torch.bfloat16).cuda()[:, 20:276]
    al = torch.tensor([0.01, 0.02], device="cuda")
    r = torch.ones((6, 48), device="cuda", dtype=torch.float32)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    got = pd.linear(x, dc, ds, 48, alpha=al, residual=r, activation="silu", gated=True, out_dtype=torch.float32)
    want, err = ffn.linear(x.double().cpu().numpy(), codes, scales, al.cpu().numpy(), None, r.cpu().numpy(),
                           "silu", True)
    assert_close(got, want, err, "f32")
    pc, ps = pd.pack_weight(dc, ds)
    again = pd.linear(x, pc, ps, 48, alpha=al, residual=r, activation="silu", gated=True, packed=True, out=r)
    assert again is r
    assert_close(r, want, err, "f32")


def test_linear_repeats_bit_for_bit():
    rng = np.random.default_rng(17)
    for n in (1, 16, 100, 300):
        codes, scales = weight(rng, 1, 500, 2048)
        dc, ds = pd.pack_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
        x = torch.from_numpy(rng.standard_normal((n, 2048))).to(torch.bfloat16).cuda()
        first = pd.linear(x, dc, ds, 500, packed=True, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(first, pd.linear(x, dc, ds, 500, packed=True, out_dtype=torch.float32))


# ---------------------------------------------------------------- MoE
def moe_case(rng, tokens, experts, topk, hidden, inter, x="bf16", y=None, act="silu", scoring="softmax",
             route_bias=False, renormalize=True, scale=1.0, residual=None, layout="row", ldx=0, xoff=0,
             ldy=0, alpha=True, edit=None, stream=None, ws=False, woff=0):
    y = y or x
    c13, s13 = weight(rng, 2 * experts, inter, hidden)
    c2, s2 = weight(rng, experts, hidden, inter)
    xv = rounded(rng.standard_normal((tokens, hidden)), x)
    rt = rounded(rng.standard_normal((experts, hidden)) / np.sqrt(hidden) * 2, x)
    if edit:
        edit(xv, rt, c13, s13, c2, s2)
    a13 = (rng.uniform(0.5, 2, (experts, 2)) / np.sqrt(hidden) / 8).astype(np.float32) if alpha else None
    a2 = (rng.uniform(0.5, 2, experts) / np.sqrt(inter) / 8).astype(np.float32) if alpha else None
    rb = rng.uniform(-0.2, 0.2, experts).astype(np.float32) if route_bias else None
    rv = rounded(rng.standard_normal((tokens, hidden)), y) if residual else None
    dev = lambda v: None if v is None else torch.from_numpy(v).cuda()
    if layout == "packed":
        w13 = pd.pack_weight(dev(c13), dev(s13))
        w2 = pd.pack_weight(dev(c2), dev(s2))
    else:
        w13, w2 = (bytes_at(c13, woff), bytes_at(s13, woff)), (bytes_at(c2, woff), bytes_at(s2, woff))
    layer = pd.MoeLayer(device(rt, x).contiguous(), *w13, *w2, inter=inter, topk=topk, alpha13=dev(a13),
                        alpha2=dev(a2), route_bias=dev(rb), activation=act, scoring=scoring,
                        renormalize=renormalize, routed_scale=scale, packed=layout == "packed")
    dx = device(xv, x, ldx or hidden, xoff)
    ld = ldy or hidden
    if residual == "in place":
        dr = out = device(rv, y, ld)
    else:
        out = device(np.full((tokens, hidden), 7.0), y, ld)
        dr = None if rv is None else device(rv, y, ld + 1)
    args = (layer, dx, ldx or hidden, dr, ld if residual == "in place" else ld + 1, out, CODES[y], ld, tokens)
    if ws:
        need = pd.nvfp4_moe_layer_workspace_size(layer, tokens)
        w = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
        pd.nvfp4_moe_layer_launch_ws(*args, w, need)
        torch.cuda.synchronize()
        assert bool((w[need:] == 0x7F).all()), "wrote past the workspace"
    else:
        pd.nvfp4_moe_layer_launch(*args)
    torch.cuda.synchronize()
    want, err = ffn.moe(xv, rt, c13, s13, c2, s2, topk, a13, a2, rb, rv, act, scoring, renormalize, scale,
                        planes=3 if y == "f32" else 2)
    assert_close(out, want, err, y, f"moe t={tokens} e={experts} k={topk} {hidden}x{inter} {x}->{y} {layout}")
    return out


@pytest.mark.parametrize("layout", ["row", "packed"])
@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [
    (1, 1, 1, 64, 64), (1, 4, 2, 64, 128), (2, 4, 4, 192, 64), (3, 7, 3, 320, 192), (7, 11, 3, 256, 320),
    (16, 64, 8, 512, 256), (17, 5, 2, 1088, 128), (33, 3, 1, 128, 704), (64, 130, 6, 64, 64),
    (40, 2, 2, 256, 192), (100, 9, 4, 128, 128)])
def test_moe_sizes(tokens, experts, topk, hidden, inter, layout):
    print(f"moe {tokens} {experts} {topk} {hidden} {inter} {layout}", flush=True)
    rng = np.random.default_rng(tokens * 7919 + experts * 31 + hidden)
    moe_case(rng, tokens, experts, topk, hidden, inter, layout=layout)
    moe_case(rng, tokens, experts, topk, hidden, inter, x="f16", y="f32", layout=layout, residual="apart")


@pytest.mark.parametrize("hidden,inter", [(16, 16), (48, 80), (272, 112), (1040, 336)])
def test_moe_row_major_whole_blocks(hidden, inter):
    rng = np.random.default_rng(hidden)
    moe_case(rng, 5, 6, 2, hidden, inter, x="f16", scoring="sigmoid", route_bias=True, scale=2.5)
    moe_case(rng, 1, 6, 2, hidden, inter, y="f32")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("act", list(ACTS))
def test_moe_options(act, scoring):
    rng = np.random.default_rng(21)
    for bias, renorm, residual in itertools.product((False, True), (False, True), (None, "apart", "in place")):
        moe_case(rng, 6, 8, 3, 128, 192, act=act, scoring=scoring, route_bias=bias, renormalize=renorm,
                 scale=1.5, residual=residual, layout="packed" if bias else "row", ldy=131, ldx=133, ws=True)


def test_moe_strided_and_unaligned_input():
    rng = np.random.default_rng(22)
    for ldx, xoff in ((264, 0), (257, 0), (256, 1), (259, 5)):
        for layout in ("row", "packed"):
            moe_case(rng, 9, 5, 2, 256, 128, ldx=ldx, xoff=xoff, layout=layout)


def test_moe_more_than_one_pass_of_tokens_per_expert():
    moe_case(np.random.default_rng(23), 150, 2, 2, 192, 128, layout="packed", alpha=False)


@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [
    (12, 7, 4, 128, 768), (16, 40, 6, 80, 400), (5, 1024, 64, 64, 112), (17, 1000, 3, 64, 64),
    (300, 70, 8, 1024, 256), (90, 130, 5, 1088, 192)])
def test_moe_by_expert(tokens, experts, topk, hidden, inter):
    """Sizes at which slots are sorted by expert: few and many tokens, experts up to the most,
    few and many workgroups, several passes of tokens per expert."""
    print(f"moe by expert {tokens} {experts} {topk} {hidden} {inter}", flush=True)
    rng = np.random.default_rng(tokens + experts)
    odd = hidden % 64 or inter % 64
    moe_case(rng, tokens, experts, topk, hidden, inter, layout="row" if odd else "packed", residual="apart")
    moe_case(rng, tokens, experts, topk, hidden, inter, x="f16", y="f32", scoring="sigmoid", route_bias=True,
             renormalize=False, scale=0.5, ldx=hidden + 1)


@pytest.mark.parametrize("woff", [1, 4])
def test_moe_misaligned_weights(woff):
    rng = np.random.default_rng(28)
    moe_case(rng, 3, 6, 2, 128, 192, woff=woff)
    moe_case(rng, 40, 6, 2, 128, 192, x="f16", y="f32", woff=woff)


def test_moe_rows_four_million_elements_apart():
    """Token offsets past 32 bits: within what the fast kernels can address, and past it."""
    rng = np.random.default_rng(29)
    c13, s13 = weight(rng, 12, 64, 64)
    c2, s2 = weight(rng, 6, 64, 64)
    dev = lambda v: torch.from_numpy(v).cuda()
    layer = pd.MoeLayer(torch.from_numpy(rng.standard_normal((6, 64))).to(torch.bfloat16).cuda(),
                        *pd.pack_weight(dev(c13), dev(s13)), *pd.pack_weight(dev(c2), dev(s2)), inter=64, topk=2,
                        alpha13=torch.full((6, 2), 0.01, device="cuda"), packed=True)
    far = torch.zeros((300, 1 << 22), dtype=torch.bfloat16, device="cuda")[:, 64:128]
    for n in (2, 60, 300):
        x = torch.from_numpy(rng.standard_normal((n, 64))).to(torch.bfloat16).cuda()
        far[:n] = x
        a = pd.moe_layer(far[:n], layer, out_dtype=torch.float32)
        b = pd.moe_layer(x, layer, out_dtype=torch.float32)
        # other kernels may add in another order: some 1e-6 of the largest output
        assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max()), n


def test_moe_ties_go_to_the_lowest_index():
    def edit(xv, rt, *rest):
        rt[1:] = rt[0]                     # every expert scores the same

    moe_case(np.random.default_rng(24), 5, 9, 3, 64, 64, y="f32", edit=edit)
    moe_case(np.random.default_rng(24), 5, 70, 3, 64, 64, y="f32", edit=edit, scoring="sigmoid")


def test_moe_experts_without_tokens_and_all_tokens_on_one():
    def edit(xv, rt, *rest):
        rt[:] = 0.0
        xv[:, 0] = 1.0
        rt[4, 0] = 8.0                     # every token chooses expert 4, then 0

    moe_case(np.random.default_rng(25), 35, 6, 2, 128, 64, edit=edit, layout="packed")
    moe_case(np.random.default_rng(25), 35, 6, 2, 128, 64, edit=edit, layout="row")


def test_moe_nan_token_stays_alone():
    def edit(xv, rt, *rest):
        xv[2, 7] = np.nan

    out = moe_case(np.random.default_rng(26), 5, 6, 2, 128, 64, edit=edit, layout="packed")
    assert bool(out[2].isnan().all()) and not bool(out[[0, 1, 3, 4]].isnan().any())


def test_moe_nan_expert_touches_only_its_tokens():
    def edit(xv, rt, c13, s13, c2, s2):
        s13[2 * 3, 1, 0] = 0x7F            # expert 3's gate

    moe_case(np.random.default_rng(27), 12, 6, 2, 128, 64, edit=edit, layout="packed")


def test_moe_empty_call_does_nothing():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    layer = pd.MoeLayer(torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda"), z(4, 32, 32), z(4, 32, 4),
                        z(2, 64, 16), z(2, 64, 2), inter=32, topk=1)
    assert tuple(pd.moe_layer(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), layer).shape) == (0, 64)


# ---------------------------------------------------------------- graphs and streams
def feed_forward_inputs(seed, tokens=5, hidden=256, inter=192, experts=6):
    rng = np.random.default_rng(seed)
    c13, s13 = weight(rng, 2 * experts, inter, hidden)
    c2, s2 = weight(rng, experts, hidden, inter)
    cl, sl = weight(rng, 1, hidden, hidden)
    dev = lambda v: torch.from_numpy(v).cuda()
    layer = pd.MoeLayer(torch.from_numpy(rng.standard_normal((experts, hidden)) / 16).to(torch.bfloat16).cuda(),
                        *pd.pack_weight(dev(c13), dev(s13)), *pd.pack_weight(dev(c2), dev(s2)), inter=inter,
                        topk=2, alpha13=torch.full((experts, 2), 0.01, device="cuda"),
                        alpha2=torch.full((experts,), 0.01, device="cuda"), packed=True)
    lin = pd.pack_weight(dev(cl), dev(sl))
    x = torch.from_numpy(rng.standard_normal((tokens, hidden))).to(torch.bfloat16).cuda()
    return x, layer, lin, torch.tensor([0.01], device="cuda")


def test_captured_graph_replays_match_eager():
    x, layer, lin, al = feed_forward_inputs(31)

    def step():
        h = pd.linear(x, *lin, 256, alpha=al, residual=x, activation="gelu", packed=True)
        return pd.moe_layer(h, layer, residual=h)

    s = torch.cuda.Stream()
    pd.nvfp4_workspace_reserve(max(pd.nvfp4_moe_layer_workspace_size(layer, x.shape[0]),
                                   pd.nvfp4_linear_workspace_size(x.shape[0], 256, 256)), stream=s)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        assert torch.equal(replayed, step()), f"replay {i}"
        torch.cuda.synchronize()


def test_capture_without_a_reserved_workspace_is_refused():
    x, layer, lin, al = feed_forward_inputs(32, tokens=40)
    out = torch.zeros((40, 256), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out.add_(1.0)
        with pytest.raises(pd.Nvfp4GemvError) as e:
            pd.moe_layer(x, layer, out=out)
        assert e.value.status == pd.NVFP4_GEMV_ERR_WORKSPACE
    g.replay()
    torch.cuda.synchronize()
    assert bool((out == 1.0).all())


def test_streams_do_not_share_workspaces():
    cases = [feed_forward_inputs(40 + i, tokens=3 + 4 * i) for i in range(3)]
    want = [pd.moe_layer(x, layer) for x, layer, _, _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        got = [pd.moe_layer(x, layer, stream=s) for (x, layer, _, _), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_feed_forward_example(tokens, capsys):
    """The example's block, captured and replayed, and its step against the same layers on
    the oracle's weights."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(["--tokens", str(tokens), "--hidden", "512", "--inter", "256", "--experts", "8", "--topk", "2",
                         "--steps", "3"])
    assert "equals" in capsys.readouterr().out
    y = example.Block(512, 256, 8, 2).step(torch.randn((tokens, 512), device="cuda").to(torch.bfloat16),
                                           torch.zeros((tokens, 512), dtype=torch.bfloat16, device="cuda"))
    # unit-size weights and inputs: outputs of unit size
    assert bool(y.isfinite().all()) and 0.2 < float(y.float().std()) < 5.0
