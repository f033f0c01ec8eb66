"""The tile kernel of the linear layer on the GPU against the float64 oracle:
each shape with row-major weights of any k and alignment, with K split, with
special values, far and unaligned rows and every epilogue; and, on every kernel,
the activations' tails and overflow."""
import itertools
import math

import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from ffn_plans import SPLIT_TILES, TILES, WHOLE_TILES
from ffn_util import ACTS, TYPES, rounded, weight
from oracle import ffn
from test_gpu_ffn import linear_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,m,k,gated", list(TILES))
def test_row_major_weights_of_any_k_and_alignment(n, m, k, gated):
    print(f"tiles {n} {m} {k} gated={gated}", flush=True)
    rng = np.random.default_rng(n + m)
    linear_case(rng, n, m, k, x="bf16", gated=gated, act="silu", bias=True, ldx=k + 8, ws=True)
    linear_case(rng, n, m, k, x="f16", y="f32", gated=gated, residual="in place", ldx=k + 1, xoff=1, ldy=m + 3, ws=True)
    # whole rows of 64 whose codes or scales have no more than their own alignment
    k = -(-k // 64) * 64
    linear_case(rng, n, m, k, x="f16", gated=gated, woff=4, ldy=m + 2)
    linear_case(rng, n, m, k, x="bf16", y="f16", gated=gated, soff=1, residual="apart")


@pytest.mark.parametrize("n,m,k,gated", list(SPLIT_TILES))
def test_split_sums_of_ragged_rows(n, m, k, gated):
    print(f"split tiles {n} {m} {k} gated={gated}", flush=True)
    rng = np.random.default_rng(n + m + 1)
    linear_case(rng, n, m, k, x="bf16", gated=gated, act="silu", bias=True, residual="in place", ldy=m + 1, ws=True)
    linear_case(rng, n, m, k, x="f16", y="f32", gated=gated, act="gelu", ldx=k + 3, xoff=1, ws=True)


def special(k):
    def edit(xv, codes, scales):
        scales[0, 5, 3] = 0x7F            # NaN scale: weight row 5
        xv[1, 100] = np.inf               # infinite input: token 1 (inf or NaN by the weights' signs)
        xv[3, k - 1] = np.nan             # and one that is not a number: token 3
        codes[0, 7] = 0                   # a row of zeros (times infinity: NaN)
        xv[0] = 0.0                       # a token of zeros
        scales[0, 9] = 0                  # a row of zero scales
    return edit


@pytest.mark.parametrize("layout", ["row", "packed", "blocks"])
@pytest.mark.parametrize("n,m,k,gated", [c for c in WHOLE_TILES if c[2] == 320])
def test_special_values_stay_in_their_row_and_token(n, m, k, gated, layout):
    k = k + 16 if layout == "blocks" else k
    out = linear_case(np.random.default_rng(61), n, m, k, gated=gated, layout="packed" if layout == "packed" else "row",
                      edit=special(k), y="f32")
    assert bool(out[:, 5].isnan().all()) and bool(out[3].isnan().all())
    assert bool((out[0, [0, 1, 7, 9]] == 0).all())


@pytest.mark.parametrize("n,m,k,gated", [c for c in WHOLE_TILES if c[2] == 64])
def test_rows_four_million_elements_apart(n, m, k, gated):
    rng = np.random.default_rng(62)
    codes, scales = weight(rng, 1, m, k)
    dc, ds = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    far = torch.zeros((n, 1 << 22), dtype=torch.bfloat16, device="cuda")[:, 64:128]
    x = torch.from_numpy(rng.standard_normal((n, k))).to(torch.bfloat16).cuda()
    far.copy_(x)
    assert torch.equal(pd.linear(far, dc, ds, m), pd.linear(x, dc, ds, m))


@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", list(ACTS))
def test_epilogues(act, y):
    rng = np.random.default_rng(63)
    for gated, bias, residual in itertools.product((False, True), (False, True), (None, "apart", "in place")):
        linear_case(rng, 130, 1030, 320, y=y, act=act, gated=gated, bias=bias, residual=residual,
                    layout="packed" if bias else "row", ldy=1037)


# ---------------------------------------------------------------- every kernel
# n, m, k: one token, the stream kernel with few and more tokens, the tile kernel, the simple one
# (codes at an odd address)
KERNELS = {"dot": (1, 40, 64, 0), "stream": (9, 40, 64, 0), "tile": (300, 2050, 64, 0), "simple": (20, 40, 64, 1)}
U24 = 2.0 ** -24


def tail_bound(act, z):
    """Relative error of f(z), z exact, from the fp32 operations in it: the hardware's exp2
    and reciprocal err by one unit in the last place (2 U24), the others by half; exp(a) errs
    by |a| U24 for the product with log2 e and half that for log2 e itself."""
    if act == "silu":
        return 1.5 * U24 * np.abs(z) + 6 * U24
    if act == "gelu_tanh":
        # u from six roundings and two constants, all of one sign
        u = math.sqrt(2 / math.pi) * (np.abs(z) + 0.044715 * np.abs(z) ** 3)
        return 2 * u * (8 + 1.5) * U24 + 6 * U24
    # gelu: the polynomial's fit up to |z| = 8 (1e-7), its evaluation (3.2 times half a unit, from
    # the sizes of its partial sums), its argument (reciprocal, constant and sum, times 2.9, the
    # polynomial's largest logarithmic slope), the exponential of z^2 / 2 and the products
    return 1e-7 + 3.2 * U24 + 2.9 * 5 * U24 + (2.5 * z * z / 2 + 6) * U24


def exact64(act, z):
    if act == "gelu":
        return np.array([0.5 * v * math.erfc(-v / math.sqrt(2.0)) for v in z])
    return ffn.activation(act, z)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("act,low,high", [("silu", -80.0, 80.0), ("gelu", -8.0, 20.0), ("gelu_tanh", -9.0, 20.0)])
def test_activations_keep_their_relative_accuracy(act, low, high, kernel):
    """f of numbers that reach it exactly (one input times 1), in fp32: the negative tails to
    the last bits that the fp32 operations leave."""
    n, m, k, odd = KERNELS[kernel]
    codes = torch.zeros((m, k // 2), dtype=torch.uint8)
    codes[:, 0] = 0x02                                        # 1.0 at element 0
    store = torch.zeros(codes.numel() + odd, dtype=torch.uint8, device="cuda")
    store[odd:] = codes.view(-1).cuda()
    scales = torch.full((m * k // 16,), 0x38, dtype=torch.uint8, device="cuda")
    z = rounded(np.concatenate([np.linspace(low, high, 600), np.linspace(-3.0, 3.0, 600)]), "bf16")
    got = []
    for at in range(0, len(z) // n * n if n > 1 else 128, n):
        x = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
        part = z[at:at + n] if n > 1 else z[at * 9:at * 9 + 1]
        x[:, 0] = torch.from_numpy(part).to(torch.bfloat16).cuda()
        y = pd.linear(x, store[odd:], scales, m, activation=act, out_dtype=torch.float32)
        assert bool((y == y[:, :1]).all())
        got.append((part, y[:, 0].double().cpu().numpy()))
    z, got = (np.concatenate(v) for v in zip(*got))
    want = exact64(act, z)
    bound = tail_bound(act, z) * np.abs(want)
    assert bool((np.abs(got - want) <= bound).all()), float((np.abs(got - want) / np.maximum(bound, 1e-300)).max())


def assert_rounds_to(got, want, err, kind, what):
    """As a value within err of want rounds: to the infinity of want's sign from half a step
    above the largest number on, to neither below it."""
    got = got.double().cpu().numpy()
    info = torch.finfo(TYPES[kind])
    half = info.eps / 2
    top = info.max + 2.0 ** (math.floor(math.log2(info.max)) - 1) * info.eps     # half a step more
    assert np.isfinite(want).all()
    sure = np.abs(want) - err >= top
    assert np.array_equal(got[sure], np.copysign(np.inf, want[sure])), f"{what}: overflow"
    below = np.abs(want) + err < top
    tol = err + half * (np.abs(want) + err) + info.smallest_normal * half
    assert bool((np.abs(got - want) <= tol)[below].all()), f"{what}: finite values"
    # within err of the border: the infinity or a finite value as near as any other
    rest = ~sure & ~below
    near = (got == np.copysign(np.inf, want)) | (np.abs(got - want) <= tol)
    assert bool(near[rest].all()), f"{what}: values at the border"
    return int(sure.sum()), int(below.sum())


@pytest.mark.parametrize("y", ["f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,m,k", [(1, 40, 64), (3, 20, 64), (40, 70, 80), (300, 2050, 64), (70, 2050, 4112)])
def test_overflow_goes_to_the_right_infinity(n, m, k, gated, y):
    """Outputs around the largest number of their type, on the kernels for one token, few
    and many, and with K split."""
    rng = np.random.default_rng(64 + n)
    groups = 2 if gated else 1
    codes, scales = weight(rng, groups, m, k)
    xv = rounded(rng.standard_normal((n, k)), "bf16")
    # alphas that put three outputs in ten above the largest number; a residual where fp32 has
    # room for the sum before it
    target = float(torch.finfo(TYPES[y]).max)
    parts = [xv @ ffn.weights(codes[g], scales[g]).T for g in range(groups)]
    al = np.full(groups, (target / np.quantile(np.abs(np.prod(parts, axis=0)), 0.7)) ** (1.0 / groups), np.float32)
    rv = rounded(rng.uniform(-0.5, 0.5, (n, m)) * target, y) if y == "f16" else None
    got = pd.linear(torch.from_numpy(xv).to(torch.bfloat16).cuda(), torch.from_numpy(codes).cuda(),
                    torch.from_numpy(scales).cuda(), m, alpha=torch.from_numpy(al).cuda(),
                    residual=None if rv is None else torch.from_numpy(rv).to(TYPES[y]).cuda(), gated=gated,
                    out_dtype=TYPES[y])
    want, err = ffn.linear(xv, codes, scales, al, None, rv, "none", gated)
    over, under = assert_rounds_to(got, want, err, y, f"{n} {m} {k} {y} gated={gated}")
    assert over > 0 and under > 0
