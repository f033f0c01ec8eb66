"""Cases and plain forms of the NVFP4-weight operators: the linear layer with a
fused epilogue and the mixture-of-experts layer for a few tokens.

linear:  Y[t,r] = residual[t,r] + f(z[t,r]),  z[t,r] = alpha sum_k X[t,k] W[r,k] + bias[r]
         or, gated, Y[t,r] = residual[t,r] + f(gate[t,r]) up[t,r], with the weight
         holding a gate and an up matrix, each with its own alpha and bias;
moe:     s[t,:] = softmax or sigmoid of X[t] Wr^T; the topk experts of a token by
         s + route_bias (lowest index first among equals), weighted by s,
         renormalised over the chosen ones if asked, times a constant;
         Y[t] = residual[t] + sum_j w[t,j] down_j( f(gate_j(X[t])) up_j(X[t]) ).

X is bf16 or fp16, the weights are NVFP4 (two E2M1 codes per byte, low nibble
first, one E4M3 scale per 16 elements along k), Y is bf16, fp16 or fp32.

``own`` chooses between elementary torch operations and the library's calls.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _linear(name, n, m, k, x="bf16", y="bf16", act="none", gated=False, bias=False, residual=False,
            pad=0, packed=True):
    return {"op": "linear", **({"name": name} if name else {}), "n": n, "m": m, "k": k, "x": x, "y": y, "act": act,
            "gated": gated, "bias": bias, "residual": residual, "pad": pad, "packed": packed}


def _moe(name, tokens, experts, topk, hidden, inter, x="bf16", y="bf16", act="silu",
         scoring="softmax", route_bias=False, renormalize=True, scale=1.0, residual=False,
         packed=True):
    return {"op": "moe", **({"name": name} if name else {}), "tokens": tokens, "experts": experts, "topk": topk,
            "hidden": hidden, "inter": inter, "x": x, "y": y, "act": act, "scoring": scoring,
            "route_bias": route_bias, "renormalize": renormalize, "scale": scale,
            "residual": residual, "packed": packed}


def listed():
    return [
        # one token through a tiny projection: launch latency
        _linear("linear_tiny", 1, 128, 256, act="silu", bias=True),
        # one decoded token through the decode weight, the residual added on the way out
        _linear("linear_decode_1", 1, 7168, 16384, residual=True),
        # a decode batch through the gate and up matrices of a dense feed-forward block
        _linear("linear_gated_16", 16, 4096, 7168, x="f16", y="f16", act="silu", gated=True),
        # odd everything: ragged rows and tokens, a strided input, row-major weights whose
        # k is no multiple of 64, fp32 out
        _linear("linear_odd", 37, 1001, 2064, x="f16", y="f32", act="gelu", bias=True, pad=5,
                packed=False),
        # speculative tokens or a short prompt through a wide, short weight
        _linear("linear_short_100", 100, 7168, 2048, act="gelu_tanh", bias=True),
        # a prompt: the compute-bound end
        _linear("linear_prompt", 4096, 4096, 7168, act="silu", bias=True, residual=True),
        # a small layer, one token: launch latency
        _moe("moe_tiny", 1, 6, 2, 256, 96, packed=False),
        # odd sizes, sigmoid scores with a selection bias, row-major weights, fp32 out
        _moe("moe_odd", 7, 11, 3, 1040, 336, x="f16", y="f32", act="gelu_tanh", scoring="sigmoid",
             route_bias=True, scale=2.5, residual=True, packed=False),
        # one decoded token through a large layer
        _moe("moe_decode_1", 1, 64, 8, 7168, 2048, residual=True),
        # a decode batch: 128 routed slots over 64 experts
        _moe("moe_decode_16", 16, 64, 8, 7168, 2048, residual=True),
        # a larger batch, weights not renormalised
        _moe("moe_batch_64", 64, 64, 4, 4096, 2048, x="f16", y="f16", renormalize=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer of [lo, hi], its logarithm uniform, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    x = rng.choice(["bf16", "bf16", "f16"])
    y = rng.choice([x, x, "f32"])
    packed = rng.random() < 0.7
    # packed weights come in 64-element pieces of k, row-major ones in whole scale blocks
    step = 64 if packed else 16
    if rng.random() < 0.55:
        k = _log_int(rng, 128, 16384, step)
        m = _log_int(rng, 64, 7168)
        gated = rng.random() < 0.4
        most = 4096 * 4096 * 7168 // (m * k * (2 if gated else 1))
        n = _log_int(rng, 1, max(1, min(4096, most)))
        return _linear(None, n, m, k, x, y, rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                       gated, rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 3, 8]), packed)
    hidden = _log_int(rng, 256, 7168, step)
    inter = _log_int(rng, 64, 2048, step)
    experts = _log_int(rng, 4, 64)
    topk = rng.randint(1, min(8, experts))
    tokens = _log_int(rng, 1, 64)
    while _moe_flops(tokens, topk, hidden, inter) > _moe_flops(64, 4, 4096, 2048):
        tokens = max(1, tokens // 2)
    return _moe(None, tokens, experts, topk, hidden, inter, x, y,
                rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]),
                rng.choice(["softmax", "sigmoid"]), rng.random() < 0.4, rng.random() < 0.6,
                rng.choice([1.0, 2.5]), rng.random() < 0.5, packed)


def _moe_flops(tokens, topk, hidden, inter):
    return 6 * tokens * topk * hidden * inter


def work(case):
    xb, yb = _BYTES[case["x"]], _BYTES[case["y"]]
    if case["op"] == "linear":
        n, m, k = case["n"], case["m"], case["k"]
        rows = m * (2 if case["gated"] else 1)
        b = n * k * xb + rows * k * 9 // 16 + n * m * yb * (2 if case["residual"] else 1)
        b += rows * 4 if case["bias"] else 0
        return {"bytes": b, "flops": 2 * n * rows * k}
    t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inter"]
    # experts that at least one token chooses, as expected of independent choices
    active = e * (1.0 - (1.0 - case["topk"] / e) ** t)
    b = t * h * xb + e * h * xb + int(active * 3 * h * i * 9 / 16) + t * h * yb * (2 if case["residual"] else 1)
    return {"bytes": b, "flops": 2 * t * e * h + _moe_flops(t, case["topk"], h, i)}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weight(g, groups, rows, k):
    """Codes and scales of weights quantised from a normal distribution: the codes take
    16 equally likely levels of one, the scales lie where block maxima put them."""
    levels = torch.tensor([13, 15, 12, 11, 10, 10, 9, 8, 0, 1, 2, 2, 3, 4, 7, 5], dtype=torch.uint8,
                          device="cuda")
    codes = torch.empty((groups, rows, k // 2), dtype=torch.uint8, device="cuda")
    for i in range(groups):
        r = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g).int()
        codes[i] = levels[r & 15] | (levels[r >> 4] << 4)
    scales = torch.randint(0x6A, 0x77, (groups, rows, k // 16), dtype=torch.uint8, device="cuda",
                           generator=g)
    return codes, scales


def _alphas(g, count, k):
    """Global scales that give outputs of about unit size."""
    return (0.75 + 0.5 * torch.rand(count, device="cuda", generator=g)) / (380.0 * math.sqrt(k))


def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _inputs(case, seed):
    g = _gen(seed)
    xt, yt = _TYPES[case["x"]], _TYPES[case["y"]]
    s = {"case": case}
    if case["op"] == "linear":
        n, m, k = case["n"], case["m"], case["k"]
        groups = 2 if case["gated"] else 1
        s["x"] = _normal(g, n, k + case["pad"]).to(xt)[:, :k]
        s["codes"], s["scales"] = _weight(g, groups, m, k)
        s["alpha"] = _alphas(g, groups, k)
        s["bias"] = _normal(g, groups * m) if case["bias"] else None
        s["residual"] = _normal(g, n, m).to(yt) if case["residual"] else None
        return s
    t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inter"]
    s["x"] = _normal(g, t, h).to(xt)
    s["router"] = (_normal(g, e, h) / math.sqrt(h)).to(xt)
    s["route_bias"] = 0.1 * _normal(g, e) if case["route_bias"] else None
    s["codes13"], s["scales13"] = _weight(g, 2 * e, i, h)
    s["codes2"], s["scales2"] = _weight(g, e, h, i)
    s["alpha13"] = _alphas(g, 2 * e, h).view(e, 2)
    s["alpha2"] = 2.0 * _alphas(g, e, i)
    s["residual"] = _normal(g, t, h).to(yt) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import precision_decode_amd as pd

    # what a serving program keeps: the weights, re-laid out once where they can be, and
    # the layer's description
    if case["op"] == "linear":
        if case["packed"]:
            s["codes"], s["scales"] = pd.pack_weight(s["codes"], s["scales"])
        return s
    if case["packed"]:
        s["codes13"], s["scales13"] = pd.pack_weight(s["codes13"], s["scales13"])
        s["codes2"], s["scales2"] = pd.pack_weight(s["codes2"], s["scales2"])
    s["layer"] = pd.MoeLayer(s["router"], s["codes13"], s["scales13"], s["codes2"], s["scales2"],
                             inter=case["inter"], topk=case["topk"], alpha13=s["alpha13"],
                             alpha2=s["alpha2"], route_bias=s["route_bias"], activation=case["act"],
                             scoring=case["scoring"], renormalize=case["renormalize"],
                             routed_scale=case["scale"], packed=case["packed"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        import precision_decode_amd as pd

        if case["op"] == "linear":
            return pd.linear(state["x"], state["codes"], state["scales"], case["m"],
                             alpha=state["alpha"], bias=state["bias"], residual=state["residual"],
                             activation=case["act"], gated=case["gated"], packed=case["packed"],
                             out_dtype=_TYPES[case["y"]])
        return pd.moe_layer(state["x"], state["layer"], residual=state["residual"],
                            out_dtype=_TYPES[case["y"]])
    return _plain_linear(state) if case["op"] == "linear" else _plain_moe(state)


def _decode(codes, scales):
    """float32 weights (without their global scale) of one (rows, k/2) matrix."""
    table = torch.tensor(_MAGNITUDES + tuple(-v for v in _MAGNITUDES), device=codes.device)
    c = codes.int()
    w = torch.stack((table[c & 15], table[c >> 4]), dim=-1)
    s = scales.view(torch.float8_e4m3fn).float()
    return (w.view(codes.shape[0], -1, 16) * s[:, :, None]).view(codes.shape[0], -1)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_linear(state):
    case = state["case"]
    x = state["x"].float()
    m = case["m"]
    z = []
    for i in range(2 if case["gated"] else 1):
        v = state["alpha"][i] * (x @ _decode(state["codes"][i], state["scales"][i]).t())
        if state["bias"] is not None:
            v = v + state["bias"][i * m:(i + 1) * m]
        z.append(v)
    y = _act(case["act"], z[0])
    if case["gated"]:
        y = y * z[1]
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(_TYPES[case["y"]])


def _plain_moe(state):
    case = state["case"]
    e = case["experts"]
    # 64 bits up to the choice: two experts' scores can be very near each other
    z = state["x"].double() @ state["router"].double().t()
    if case["scoring"] == "softmax":
        p = torch.exp(z - z.max(dim=1, keepdim=True).values)
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    key = p if state["route_bias"] is None else p + state["route_bias"].double()
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["topk"]]
    w = torch.zeros_like(p).scatter(1, order, p.gather(1, order))
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = (w * case["scale"]).float()
    x = state["x"].float()
    y = torch.zeros_like(x)
    for i in range(e):
        gate = state["alpha13"][i, 0] * (x @ _decode(state["codes13"][2 * i], state["scales13"][2 * i]).t())
        up = state["alpha13"][i, 1] * (x @ _decode(state["codes13"][2 * i + 1], state["scales13"][2 * i + 1]).t())
        h = _act(case["act"], gate) * up
        y = y + w[:, i:i + 1] * (state["alpha2"][i] * (h @ _decode(state["codes2"][i], state["scales2"][i]).t()))
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(_TYPES[case["y"]])


# ---------------------------------------------------------------- exact values
def _weight64(codes, scales):
    """float64 weights from the formats' definitions: sign, 2-bit exponent and 1-bit
    mantissa of E2M1; sign, 4-bit exponent (bias 7) and 3-bit mantissa of E4M3."""
    rows, half = codes.shape
    w = torch.empty((rows, 2 * half), dtype=torch.float64, device=codes.device)
    for j in range(2):
        c = (codes >> (4 * j)) & 15
        exp, man = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(exp == 0, 0.5 * man, torch.exp2(exp - 1.0) * (1.0 + 0.5 * man))
        w[:, j::2] = torch.where(c >= 8, -mag, mag)
    exp, man = ((scales >> 3) & 15).double(), (scales & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, torch.exp2(exp - 7.0) * (1.0 + man / 8.0))
    s = torch.where(scales >= 128, -mag, mag)
    return w * s.repeat_interleave(16, dim=1)


def _function64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "gelu":
        # z times the normal distribution function
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def exact(case, seed):
    s = _inputs(case, seed)
    x = s["x"].to(torch.float64)
    if case["op"] == "linear":
        m = case["m"]
        part = [torch.matmul(x, _weight64(s["codes"][i], s["scales"][i]).T.contiguous()) * s["alpha"][i].double()
                for i in range(s["codes"].shape[0])]
        if s["bias"] is not None:
            part = [p + s["bias"][i * m:(i + 1) * m].double() for i, p in enumerate(part)]
        y = _function64(case["act"], part[0])
        for p in part[1:]:
            y = y * p
    else:
        logits = torch.matmul(x, s["router"].double().T.contiguous())
        score = torch.softmax(logits, dim=1) if case["scoring"] == "softmax" else torch.sigmoid(logits)
        key = score.clone() if s["route_bias"] is None else score + s["route_bias"].double()
        chosen, weight = [], []
        for _ in range(case["topk"]):
            best = key.argmax(dim=1)
            # the lowest index among equals
            best = (key == key.gather(1, best[:, None])).int().argmax(dim=1)
            chosen.append(best)
            weight.append(score.gather(1, best[:, None])[:, 0])
            key.scatter_(1, best[:, None], -math.inf)
        chosen, weight = torch.stack(chosen, 1), torch.stack(weight, 1)
        if case["renormalize"]:
            weight = weight / weight.sum(dim=1, keepdim=True)
        weight = weight * case["scale"]
        y = torch.zeros_like(x)
        for e in chosen.unique().tolist():
            t, j = (chosen == e).nonzero(as_tuple=True)
            xe = x[t]
            gate = torch.matmul(xe, _weight64(s["codes13"][2 * e], s["scales13"][2 * e]).T.contiguous())
            up = torch.matmul(xe, _weight64(s["codes13"][2 * e + 1], s["scales13"][2 * e + 1]).T.contiguous())
            h = _function64(case["act"], gate * s["alpha13"][e, 0].double()) * (up * s["alpha13"][e, 1].double())
            out = torch.matmul(h, _weight64(s["codes2"][e], s["scales2"][e]).T.contiguous())
            y[t] += out * (s["alpha2"][e].double() * weight[t, j])[:, None]
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return y
