"""The choice of experts of the MoE layer on the GPU, on each of its kernels:
saturated scores, ties, NaN and masked experts."""
import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from ffn_util import assert_close, rounded, weight
from oracle import ffn

pytestmark = pytest.mark.gpu

# (tokens, experts, topk, hidden, inter): choice by the up product's workgroups with their own
# logits (a small router) and with logits from memory; by one workgroup with a wave per token;
# by a workgroup per four tokens
SHAPES = [(3, 24, 4, 64, 64), (3, 70, 5, 512, 64), (12, 24, 4, 128, 768), (40, 24, 4, 64, 224)]


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()


def routed(shape, z, scoring="sigmoid", renormalize=True, bias=None, nan_token=None):
    """The layer for tokens whose logits are z (tokens, experts), bf16 numbers: token t is
    the t-th unit vector, and column t of the router is z[t]."""
    tokens, experts, topk, hidden, inter = shape
    rng = np.random.default_rng(tokens * experts + hidden)
    c13, s13 = weight(rng, 2 * experts, inter, hidden)
    c2, s2 = weight(rng, experts, hidden, inter)
    xv, rt = np.zeros((tokens, hidden)), np.zeros((experts, hidden))
    xv[np.arange(tokens), np.arange(tokens)] = 1.0
    rt[:, :tokens] = rounded(z, "bf16").T
    if nan_token is not None:
        xv[nan_token, -1] = np.nan
    assert np.array_equal(rt[:, :tokens].T, z, equal_nan=True)
    dev = lambda v: torch.from_numpy(np.asarray(v)).cuda()
    layer = pd.MoeLayer(dev(rt).to(torch.bfloat16), dev(c13), dev(s13), dev(c2), dev(s2), inter=inter, topk=topk,
                        route_bias=None if bias is None else dev(bias.astype(np.float32)), scoring=scoring,
                        renormalize=renormalize)
    got = pd.moe_layer(dev(xv).to(torch.bfloat16), layer, out_dtype=torch.float32)
    want, err = ffn.moe(xv, rt, c13, s13, c2, s2, topk, route_bias=bias, scoring=scoring, renormalize=renormalize,
                        planes=3)
    assert_close(got, want, err, "f32", f"{shape} {scoring}")
    return got


def logits(shape, lo, hi, step):
    """Logits of every token in an order of its own, all different."""
    tokens, experts = shape[:2]
    rng = np.random.default_rng(tokens)
    values = np.linspace(lo, hi, experts) // step * step
    assert len(np.unique(values)) == experts
    return np.stack([rng.permutation(values) for _ in range(tokens)])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_saturated_scores_are_told_apart_by_their_logits(shape, scoring):
    routed(shape, logits(shape, 30.0, 60.0, 0.25), scoring)
    routed(shape, logits(shape, -4096.0, 4096.0, 32.0), scoring)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_scores_go_to_the_lowest_index(shape, scoring):
    z = np.zeros(shape[:2])
    z[:, 5::3] = 1.0
    routed(shape, z, scoring)
    routed(shape, z + 64.0, scoring)
    routed(shape, np.zeros(shape[:2]), scoring, bias=np.where(np.arange(shape[1]) % 4 == 2, 0.5, 0.25))


@pytest.mark.parametrize("shape", SHAPES)
def test_experts_without_a_number_come_last(shape):
    # a sigmoid's NaN is its expert's alone; topk others are left
    z = logits(shape, -4.0, 4.0, 0.0625)
    z[:, ::2] = np.nan
    out = routed(shape, z)
    assert bool(out.isfinite().all())
    # a score of 0 and a masked expert are ahead of a NaN
    z = np.full(shape[:2], np.nan)
    z[:, 3], z[:, 6] = 1.0, -4096.0
    bias = np.zeros(shape[1])
    bias[8:8 + shape[2]] = -np.inf
    z[:, 8:8 + shape[2]] = 2.0
    out = routed(shape, z, renormalize=False, bias=bias)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("shape", SHAPES)
def test_a_token_without_a_number_stays_alone(shape):
    out = routed(shape, logits(shape, -4.0, 4.0, 0.0625), "softmax", nan_token=1)
    assert bool(out[1].isnan().all()) and bool(out[[0, 2]].isfinite().all())
