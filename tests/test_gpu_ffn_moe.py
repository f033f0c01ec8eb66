"""The MoE layer on the GPU against the float64 oracle: thousands of tokens up
to the most that a call takes, rows between other data, and overflow; and the
feed-forward example's step, layer by layer."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import precision_decode_amd as pd
from ffn_util import CODES, TYPES, assert_close, device, rounded, weight
from oracle import ffn
from test_gpu_ffn_tiles import assert_rounds_to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    pd.load()
    yield
    torch.cuda.empty_cache()


class Case:
    """Weights, tokens and the oracle's outputs of one layer."""

    def __init__(self, seed, tokens, experts, topk, hidden, inter, x="bf16", packed=False, **layer):
        rng = np.random.default_rng(seed)
        self.weights = (*weight(rng, 2 * experts, inter, hidden), *weight(rng, experts, hidden, inter))
        self.xv = rounded(rng.standard_normal((tokens, hidden)), x)
        self.router = rounded(rng.standard_normal((experts, hidden)) / np.sqrt(hidden) * 2, x)
        self.a13 = (rng.uniform(0.5, 2, (experts, 2)) / np.sqrt(hidden) / 8).astype(np.float32)
        self.a2 = (rng.uniform(0.5, 2, experts) / np.sqrt(inter) / 8).astype(np.float32)
        self.rng, self.topk, self.options = rng, topk, layer
        dev = lambda v: torch.from_numpy(v).cuda()
        c13, s13, c2, s2 = (dev(v) for v in self.weights)
        if packed:
            (c13, s13), (c2, s2) = pd.pack_weight(c13, s13), pd.pack_weight(c2, s2)
        self.x = dev(self.xv).to(TYPES[x])
        self.layer = pd.MoeLayer(dev(self.router).to(TYPES[x]), c13, s13, c2, s2, inter=inter, topk=topk,
                                 alpha13=dev(self.a13), alpha2=dev(self.a2), packed=packed, **layer)

    def want(self, planes, residual=None, tokens=slice(None)):
        return ffn.moe(self.xv[tokens], self.router, *self.weights, self.topk, self.a13, self.a2, None,
                       None if residual is None else residual[tokens], planes=planes, **self.options)


@pytest.mark.parametrize("tokens,experts,topk,hidden,inter,packed", [
    (1000, 9, 2, 64, 64, True), (1025, 64, 8, 128, 64, True), (4096, 64, 8, 64, 48, False), (3000, 3, 3, 80, 112, False),
    (2048, 1, 1, 128, 64, True), (65535, 4, 2, 16, 16, False)])
def test_many_tokens(tokens, experts, topk, hidden, inter, packed):
    print(f"moe {tokens} {experts} {topk} {hidden} {inter}", flush=True)
    c = Case(tokens, tokens, experts, topk, hidden, inter, packed=packed)
    got = pd.moe_layer(c.x, c.layer, out_dtype=torch.float32)
    want, err = c.want(3)
    assert_close(got, want, err, "f32")
    again = pd.moe_layer(c.x, c.layer, out_dtype=torch.float32)
    assert torch.equal(got, again)         # whatever order the slots of an expert were sorted in
    got = pd.moe_layer(c.x, c.layer)
    want, err = c.want(2)
    assert_close(got, want, err, "bf16")


def test_more_tokens_than_a_call_takes_are_refused():
    c = Case(71, 2, 4, 2, 16, 16)
    x = torch.zeros((65536, 16), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pd.Nvfp4GemvError) as e:
        pd.moe_layer(x, c.layer)
    assert e.value.status == pd.NVFP4_GEMV_ERR_BAD_SHAPE


@pytest.mark.parametrize("tokens", [1, 5, 12, 40])
@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [None, "apart", "in place"])
def test_nothing_but_the_rows_is_written(tokens, y, residual):
    c = Case(72, tokens, 7, 4, 128, 768, x="f16", scoring="sigmoid")
    ld = 131
    rv = rounded(c.rng.standard_normal((tokens, 128)), y) if residual else None
    out = device(rv if residual == "in place" else np.full((tokens, 128), 7.0), y, ld)
    dr = out if residual == "in place" else None if rv is None else device(rv, y, ld + 1)
    base = out._base if out._base is not None else out
    before = base.clone()
    pd.nvfp4_moe_layer_launch(c.layer, c.x, 128, dr, ld if residual == "in place" else ld + 1, out, CODES[y], ld, tokens)
    torch.cuda.synchronize()
    want, err = c.want(3 if y == "f32" else 2, rv)
    assert_close(out, want, err, y)
    mask = torch.ones_like(base, dtype=torch.bool)
    mask.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(False)
    a, b = base[mask], before[mask]
    assert bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("tokens", [1, 5, 40])
@pytest.mark.parametrize("residual", [False, True])
def test_overflow_goes_to_the_right_infinity(tokens, residual):
    c = Case(73, tokens, 7, 4, 128, 768)
    # three outputs in ten above the largest fp16 value
    plain, _ = c.want(2)
    c.a2 *= np.float32(65504.0 / np.quantile(np.abs(plain), 0.7))
    c.layer.tensors[6].copy_(torch.from_numpy(c.a2))
    rv = rounded(c.rng.uniform(-0.5, 0.5, (tokens, 128)) * 65504.0, "f16") if residual else None
    got = pd.moe_layer(c.x, c.layer, out_dtype=torch.float16,
                       residual=None if rv is None else torch.from_numpy(rv).to(torch.float16).cuda())
    want, err = c.want(2, rv)
    over, under = assert_rounds_to(got, want, err, "f16", f"{tokens} tokens")
    assert over > 0 and under > 0


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_example_step_layer_by_layer(tokens, monkeypatch):
    """Each layer call of the example's step against the oracle on the weights that were
    packed for it and the inputs that the step gave it."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    packed, calls = [], []
    pack, linear, moe_layer = pd.pack_weight, pd.linear, pd.moe_layer
    host = lambda t: None if t is None else t.double().cpu().numpy()

    def record_pack(codes, scales):
        out = pack(codes, scales)
        packed.append((out[0].data_ptr(), codes.cpu().numpy(), scales.cpu().numpy()))
        return out

    def record_linear(x, codes, scales, m, **kw):
        before = host(x), host(kw.get("residual"))
        y = linear(x, codes, scales, m, **kw)
        _, c, s = next(p for p in packed if p[0] == codes.data_ptr())
        calls.append((host(y), ffn.linear(before[0], c, s, host(kw.get("alpha")), None, before[1],
                                          kw.get("activation", "none"), kw.get("gated", False))))
        return y

    def record_moe(x, layer, residual=None, out=None):
        before = host(x), host(residual)
        y = moe_layer(x, layer, residual=residual, out=out)
        router, codes13, _, codes2, _, alpha13, alpha2, _ = layer.tensors
        (c13, s13), (c2, s2) = (next(p[1:] for p in packed if p[0] == t.data_ptr()) for t in (codes13, codes2))
        calls.append((host(y), ffn.moe(before[0], host(router), c13, s13, c2, s2, 2, host(alpha13), host(alpha2), None,
                                       before[1])))
        return y

    monkeypatch.setattr(pd, "pack_weight", record_pack)
    monkeypatch.setattr(pd, "linear", record_linear)
    monkeypatch.setattr(pd, "moe_layer", record_moe)
    block = example.Block(512, 256, 8, 2)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    o, x = (torch.randn((tokens, 512), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    block.step(o, x)
    assert len(packed) == 5 and len(calls) == 4
    for i, (got, (want, err)) in enumerate(calls):
        assert_close(torch.from_numpy(got), want, err, "bf16", f"layer {i}")
