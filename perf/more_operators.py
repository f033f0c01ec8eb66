"""Cases and plain forms of the attention operators on a cache held in NVFP4:
norms of queries and keys with the position rotation, writing keys and values
into the paged cache and reading them back, and attention over it.

rope:   y = w x / sqrt(mean(x^2) + eps) of each head, then pairs (i, i + r/2), or
        (2 i, 2 i + 1) interleaved, of its first r elements turned by the angle that
        row positions[t] of the table holds (r/2 cosines, r/2 sines).  With a cache,
        k (rounded to its type) and v are quantised into it in the same call.
cache:  k and v of a token go to a slot (page * page_size + offset), quantised in
        blocks of 16 along the head: xn = x / g, s = e4m3(max(max |xn|, 1e-8) / 6),
        codes the E2M1 rounding of xn / s; a slot reads back as e2m1 * e4m3 * g.
attn:   softmax(scale q k) v over the visible tokens of the sequence: j <= p and
        (j > p - window, or j < sinks), p = length - queries + i for query i.

The cache: codes (pages, kv heads, page size, dp / 2), two E2M1 codes per byte, low
nibble first, scales (pages, kv heads, dp / 16, page size), dp = the head's
dimension rounded up to 64, the rest zero.

``own`` chooses between elementary torch operations and the library's calls.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-6


def _named(name, **kw):
    return {**({"name": name} if name else {}), **kw}


def _rope(name, tokens, heads, kv, dim, rot=None, x="bf16", interleaved=False, norm=True, table=8192,
          cache=False, page=64, rule=1):
    return _named(name, op="rope", tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rot or dim, x=x,
                  interleaved=interleaved, norm=norm, table=table, cache=cache, page=page, rule=rule)


def _cache(name, tokens, kv, dim, x="bf16", y="bf16", page=64, rule=1, write=True):
    return _named(name, op="cache", tokens=tokens, kv=kv, dim=dim, x=x, y=y, page=page, rule=rule, write=write)


def _attn(name, batch, queries, context, heads, kv, dim, x="bf16", page=64, window=0, sinks=0,
          uneven=False, starts=False):
    return _named(name, op="attn", batch=batch, queries=queries, context=context, heads=heads, kv=kv, dim=dim,
                  x=x, page=page, window=window, sinks=sinks, uneven=uneven, starts=starts)


def listed():
    return [
        # one token of a small layer: launch latency
        _rope("rope_tiny", 1, 8, 2, 64),
        # a prompt through a 7168-wide layer's heads
        _rope("rope_prompt", 4096, 56, 8, 128),
        # a decode batch written into the cache on the way, half of each head rotated, pairs interleaved
        _rope("rope_cache_decode", 64, 32, 8, 128, rot=64, x="f16", interleaved=True, cache=True),
        # a prompt's keys and values into the cache and back
        _cache("cache_prompt", 8192, 8, 128),
        # an odd number of slots of odd heads read back in fp32, from small pages
        _cache("cache_read_odd", 1237, 5, 80, x="f16", y="f32", page=16, write=False),
        # one token with a short history: launch latency
        _attn("attn_tiny", 1, 1, 100, 8, 2, 64, page=16),
        # a decode batch of uneven histories
        _attn("attn_decode_batch", 64, 1, 4096, 32, 8, 128, uneven=True),
        # one token with a long history
        _attn("attn_decode_long", 1, 1, 131072, 56, 8, 128),
        # a decode batch that sees the last 4096 tokens and the first 4
        _attn("attn_decode_window", 16, 1, 32768, 64, 8, 64, x="f16", page=16, window=4096, sinks=4),
        # four speculative tokens a sequence
        _attn("attn_speculative", 16, 4, 8192, 32, 4, 128, page=32, uneven=True),
        # a few prompts of odd lengths at once, odd heads, a window: ragged everything
        _attn("attn_prompts_odd", 5, 701, 1501, 15, 3, 96, x="f16", page=16, window=500, sinks=3, uneven=True,
              starts=True),
        # a prompt: the compute-bound end
        _attn("attn_prompt", 1, 4096, 4096, 32, 8, 128),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], its logarithm uniform."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    x = rng.choice(["bf16", "bf16", "f16"])
    dim = rng.choice([64, 128, 128, 128, 256, 192, 96, 80])
    kv = rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 64, 128])
    rule = rng.choice([0, 1, 1, 2])
    kind = rng.random()
    if kind < 0.25:
        heads = kv * rng.randint(1, 8)
        tokens = _log_int(rng, 1, max(1, 4096 * 64 * 128 // ((heads + kv) * dim)))
        rot = rng.choice([dim, dim, dim // 32 * 16])
        return _rope(None, tokens, heads, kv, dim, rot, x, rng.random() < 0.4, rng.random() < 0.8,
                     8192, rng.random() < 0.5, page, rule)
    if kind < 0.45:
        tokens = _log_int(rng, 1, 8192 * 8 * 128 // (kv * dim))
        return _cache(None, tokens, kv, dim, x, rng.choice([x, x, "f32"]), page, rule, rng.random() < 0.7)
    heads = kv * _log_int(rng, 1, 16)
    window, sinks = (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 64])) if rng.random() < 0.4 else (0, 0)
    uneven = rng.random() < 0.6
    if rng.random() < 0.65:
        queries = rng.choice([1, 1, 1, 2, 4, 8])
        batch = _log_int(rng, 1, 128)
        context = _log_int(rng, queries, max(queries, min(131072, 64 * 4096 * 8 * 128 // (batch * kv * dim))))
    else:
        queries = _log_int(rng, 16, 4096)
        batch = rng.randint(1, 6)
        context = queries + rng.choice([0, 0, _log_int(rng, 1, 4096)])
        while batch * queries * context * heads * dim > 4096 * 4096 * 32 * 128:
            queries = max(16, queries // 2)
            context = max(queries, context // 2)
    return _attn(None, batch, queries, context, heads, kv, dim, x, page, window, sinks, uneven, rng.random() < 0.5)


def _part(context, b, uneven):
    """The share of ``context`` that sequence b has: all, or 25 to 100 percent of it."""
    return max(1, int(context * (0.25 + 0.75 * ((b + 1) * 0.6180339887 % 1.0)))) if uneven else context


def _shape(case):
    """(length, queries) of every sequence; with starts, its own number of queries."""
    got = []
    for b in range(case["batch"]):
        n = _part(case["context"], b, case["uneven"])
        q = _part(case["queries"], b, True) if case["starts"] else case["queries"]
        got.append((max(n, q), q))
    return got


def _visible(n, q, window, sinks):
    """(pairs of a query and a token it sees, tokens that any query sees)."""
    pos = torch.arange(n - q, n, dtype=torch.int64)
    first = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
    pairs = int((pos + 1 - first + first.clamp(max=sinks)).sum())
    lowest = int(first[0])
    return pairs, n - lowest + min(lowest, sinks)


def work(case):
    xb, d = _BYTES[case["x"]], case["dim"]
    if case["op"] == "rope":
        t, heads, kv = case["tokens"], case["heads"], case["kv"]
        b = 2 * t * heads * d * xb + min(t, case["table"]) * case["rot"] * 4 + 8 * t
        b += t * kv * d * 2 * xb
        if case["cache"]:
            # k and v in, their blocks out, and back in as values
            b += t * (2 * kv * d * 9 // 8 + 2 * kv * d * xb + 8)
        return {"bytes": b, "flops": 8 * t * (heads + kv) * d}
    if case["op"] == "cache":
        t, kv = case["tokens"], case["kv"]
        b = 2 * t * kv * d * 9 // 16 + 2 * t * kv * d * _BYTES[case["y"]] + 8 * t
        if case["write"]:
            b += 2 * t * kv * d * xb + 2 * t * kv * d * 9 // 16 + 8 * t
        return {"bytes": b, "flops": 4 * t * kv * d}
    b, f = 0, 0
    for n, q in _shape(case):
        pairs, tokens = _visible(n, q, case["window"], case["sinks"])
        b += 2 * q * case["heads"] * d * xb + tokens * case["kv"] * 2 * d * 9 // 16 + 4 * (n // case["page"] + 1)
        f += 4 * pairs * case["heads"] * d
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _padded(dim):
    return -(-dim // 64) * 64


def _filled(g, pages, kv, page, dim):
    """Codes and scales of a cache that holds normally distributed values: the codes take
    16 equally likely levels, the scales lie where block maxima put them."""
    dp = _padded(dim)
    levels = torch.tensor([13, 15, 12, 11, 10, 10, 9, 8, 0, 1, 2, 2, 3, 4, 7, 5], dtype=torch.uint8, device="cuda")
    r = torch.randint(0, 256, (pages, kv, page, dp // 2), dtype=torch.uint8, device="cuda", generator=g)
    codes = levels[(r & 15).int()] | (levels[(r >> 4).int()] << 4)
    codes[..., dim // 2:] = 0
    scales = torch.randint(0x26, 0x33, (pages, kv, dp // 16, page), dtype=torch.uint8, device="cuda", generator=g)
    scales[:, :, dim // 16:] = 0
    return codes, scales


def _empty(pages, kv, page, dim):
    dp = _padded(dim)
    return (torch.zeros((pages, kv, page, dp // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((pages, kv, dp // 16, page), dtype=torch.uint8, device="cuda"))


def _inputs(case, seed):
    g = _gen(seed)
    xt, d, kv = _TYPES[case["x"]], case["dim"], case["kv"]
    s = {"case": case, "k_global": 0.5 + torch.rand(kv, device="cuda", generator=g),
         "v_global": 0.5 + torch.rand(kv, device="cuda", generator=g)}
    if case["op"] == "attn":
        shape = _shape(case)
        tokens = sum(q for _, q in shape)
        counts = [-(-n // case["page"]) for n, _ in shape]
        # some pages of the cache belong to nobody here
        pages = sum(counts) + 3
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        starts = torch.tensor([0] + counts, device="cuda").cumsum(0)[:-1]
        at = starts[:, None] + torch.arange(max(counts), device="cuda")[None, :]
        s["block_table"] = order[at.clamp(max=pages - 1)].contiguous()
        s["lengths"] = torch.tensor([n for n, _ in shape], dtype=torch.int32, device="cuda")
        s["starts"] = torch.tensor([0] + [q for _, q in shape], device="cuda").cumsum(0).to(torch.int32)
        s["most"] = max(q for _, q in shape)
        s["q"] = _normal(g, tokens, case["heads"], d).to(xt)
        s["cache"] = _filled(g, pages, kv, case["page"], d) + _filled(g, pages, kv, case["page"], d)
        return s
    t = case["tokens"]
    pages = -(-t // case["page"]) + 2
    # whole pages in any order, the first one begun in its middle
    order = torch.randperm(pages, device="cuda", generator=g)
    i = torch.arange(t, device="cuda") + case["page"] // 2
    s["slots"] = order[i // case["page"]] * case["page"] + i % case["page"]
    if case["op"] == "rope":
        # what the QKV projection gives: one row a token, q, k and v side by side
        heads = case["heads"]
        qkv = _normal(g, t, heads + 2 * kv, d).to(xt)
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        s["q_weight"] = 1.0 + 0.1 * _normal(g, d) if case["norm"] else None
        s["k_weight"] = 1.0 + 0.1 * _normal(g, d) if case["norm"] else None
        half = case["rot"] // 2
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * torch.exp2(
            -math.log2(10000.0) / half * torch.arange(half, device="cuda", dtype=torch.float64))
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), dim=1).float()
        s["positions"] = torch.randint(0, case["table"], (t,), device="cuda", generator=g)
    else:
        s["k"] = _normal(g, t, kv, d).to(xt)
        s["v"] = _normal(g, t, kv, d).to(xt)
    fill = case["op"] == "cache" and not case["write"]
    s["cache"] = (_filled(g, pages, kv, case["page"], d) + _filled(g, pages, kv, case["page"], d) if fill else
                  _empty(pages, kv, case["page"], d) + _empty(pages, kv, case["page"], d))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import precision_decode_amd as pd

        # the description of the cache that a serving program keeps
        s["kv"] = pd.KvCache(*s["cache"], head_dim=case["dim"], k_global=s["k_global"], v_global=s["v_global"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        import precision_decode_amd as pd

        if case["op"] == "attn":
            return pd.kv_attention(state["q"], state["kv"], state["block_table"], state["lengths"],
                                   query_starts=state["starts"] if case["starts"] else None,
                                   max_query=state["most"], window=case["window"], sinks=case["sinks"])
        if case["op"] == "cache":
            if case["write"]:
                pd.kv_cache_write(state["k"], state["v"], state["kv"], state["slots"], rule=case["rule"])
            return pd.kv_cache_read(state["kv"], state["slots"], out_dtype=_TYPES[case["y"]])
        kw = {"q_weight": state["q_weight"], "k_weight": state["k_weight"], "eps": _EPS,
              "interleaved": case["interleaved"]}
        if not case["cache"]:
            return pd.qk_norm_rope(state["q"], state["k"], state["positions"], state["cos_sin"], **kw)
        q, _ = pd.qk_norm_rope(state["q"], state["k"], state["positions"], state["cos_sin"], v=state["v"],
                               cache=state["kv"], slots=state["slots"], rule=case["rule"], **kw)
        return q, pd.kv_cache_read(state["kv"], state["slots"], out_dtype=_TYPES[case["x"]])
    if case["op"] == "attn":
        return _plain_attention(state)
    if case["op"] == "cache":
        if case["write"]:
            _plain_write(state, state["k"], state["v"])
        return _plain_read(state, _TYPES[case["y"]])
    q = _plain_rope(state["q"], state["q_weight"], state).to(_TYPES[case["x"]])
    k = _plain_rope(state["k"], state["k_weight"], state).to(_TYPES[case["x"]])
    if not case["cache"]:
        return q, k
    _plain_write(state, k, state["v"])
    return q, _plain_read(state, _TYPES[case["x"]])


def _plain_rope(x, weight, state):
    case = state["case"]
    # 64 bits where the result is quantised: values lie next to the codes' borders
    wide = torch.float64 if case["cache"] else torch.float32
    y = x.to(wide)
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + _EPS) * weight.to(wide)
    r = case["rot"]
    row = state["cos_sin"][state["positions"]].to(wide)[:, None, :]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, y[..., r:]), dim=-1)


def _plain_codes(v, rule):
    a = v.abs()
    if rule == 0:
        table = torch.tensor([0, 1, 2, 3, 4, 4, 5, 5, 6, 6, 6, 7, 7], dtype=torch.int32, device=v.device)
        m = table[(2.0 * a.clamp(max=6.0)).round().int()]
    elif rule == 1:
        m = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
             + (a >= 3.5).int() + (a > 5.0).int())
    else:
        m = ((a > 0.25).int() + (a > 0.75).int() + (a > 1.25).int() + (a > 1.75).int() + (a > 2.5).int()
             + (a > 3.5).int() + (a > 5.0).int())
    return m + 8 * (v < 0).int()


def _plain_one(state, x, scale, codes, scales):
    case = state["case"]
    t, kv, d = x.shape
    xn = (x.float() / scale[:, None]).view(t, kv, d // 16, 16)
    s = (xn.abs().amax(dim=-1).clamp(min=1e-8) / 6.0).to(torch.float8_e4m3fn)
    c = _plain_codes(xn / s.float().clamp(min=1e-8)[..., None], case["rule"]).view(t, kv, d // 2, 2)
    page, off = state["slots"] // case["page"], state["slots"] % case["page"]
    codes[page, :, off, :d // 2] = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)
    scales[page, :, :d // 16, off] = s.view(torch.uint8)


def _plain_write(state, k, v):
    kc, ks, vc, vs = state["cache"]
    _plain_one(state, k, state["k_global"], kc, ks)
    _plain_one(state, v, state["v_global"], vc, vs)


def _values(codes, scales, scale, dim):
    """float32 values (n, kv, dim) of codes (n, kv, dp / 2) and scales (n, kv, dp / 16)."""
    levels = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    table = torch.tensor(levels + tuple(-v for v in levels), device=codes.device)
    c = codes[..., :dim // 2].int()
    w = torch.stack((table[c & 15], table[c >> 4]), dim=-1).view(*c.shape[:2], dim // 16, 16)
    s = scales[..., :dim // 16].contiguous().view(torch.float8_e4m3fn).float()
    return (w * s[..., None]).view(*c.shape[:2], dim) * scale[:, None]


def _plain_read(state, dtype):
    case = state["case"]
    page, off = state["slots"] // case["page"], state["slots"] % case["page"]
    kc, ks, vc, vs = state["cache"]
    return (_values(kc[page, :, off], ks[page, :, :, off], state["k_global"], case["dim"]).to(dtype),
            _values(vc[page, :, off], vs[page, :, :, off], state["v_global"], case["dim"]).to(dtype))


def _plain_attention(state):
    case = state["case"]
    kv, d, most = case["kv"], case["dim"], state["most"]
    kc, ks, vc, vs = state["cache"]
    lengths, starts = state["lengths"].long(), state["starts"].long()
    batch = lengths.shape[0]
    width = state["block_table"].shape[1] * case["page"]
    at = torch.arange(width, device="cuda")
    page = state["block_table"].long()[:, at // case["page"]].reshape(-1)
    off = (at % case["page"]).repeat(batch)
    k = _values(kc[page, :, off], ks[page, :, :, off], state["k_global"], d).view(batch, width, kv, d)
    v = _values(vc[page, :, off], vs[page, :, :, off], state["v_global"], d).view(batch, width, kv, d)
    # queries as one (batch, most) block, those behind a sequence's last one copies of it
    queries = starts[1:] - starts[:-1]
    i = torch.arange(most, device="cuda")
    row = starts[:-1, None] + torch.minimum(i[None, :], queries[:, None] - 1)
    q = state["q"][row.reshape(-1)].float().view(batch, most, kv, -1, d)
    group = q.shape[3]
    q = q.permute(0, 2, 1, 3, 4).reshape(batch, kv, most * group, d)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    pos = (lengths - queries)[:, None] + i[None, :]
    seen = at[None, None, :] <= pos[:, :, None]
    if case["window"]:
        seen = seen & ((at[None, None, :] > pos[:, :, None] - case["window"]) | (at < case["sinks"])[None, None, :])
    z = z.view(batch, kv, most, group, width)
    z = torch.where(seen[:, None, :, None, :], z, torch.full_like(z[:1, :1, :1, :1, :1], -math.inf))
    p = torch.exp(z - z.amax(dim=-1, keepdim=True))
    p = (p / p.sum(dim=-1, keepdim=True)).view(batch, kv, most * group, width)
    y = torch.matmul(p, v.permute(0, 2, 1, 3)).view(batch, kv, most, group, d)
    y = y.permute(0, 2, 1, 3, 4).reshape(batch, most, kv * group, d).to(_TYPES[case["x"]])
    return y[i[None, :] < queries[:, None]]


# ---------------------------------------------------------------- exact values
def _decoded64(codes, scales):
    """float64 values of (n, dp / 2) codes and (n, dp / 16) scales from the formats'
    definitions: sign, 2-bit exponent and 1-bit mantissa of E2M1; sign, 4-bit exponent
    (bias 7) and 3-bit mantissa of E4M3."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    exp, man = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, torch.exp2(exp - 1.0) * (1.0 + 0.5 * man))
    w = torch.where(c >= 8, -mag, mag)
    exp, man = ((scales >> 3) & 15).double(), (scales & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, torch.exp2(exp - 7.0) * (1.0 + man / 8.0))
    return w * torch.where(scales >= 128, -mag, mag).repeat_interleave(16, dim=-1)


def _blocks64(x, scale, rule):
    """Values that the blocks of x (n, kv, d) stand for, times their head's scale."""
    n, kv, d = x.shape
    xn = (x.double() / scale.double()[:, None]).reshape(n, kv, d // 16, 16)
    want = xn.abs().amax(dim=-1).clamp(min=1e-8) / 6.0
    # E4M3: 3 bits below the leading one, steps of 2^-9 under 2^-6
    step = torch.exp2(torch.floor(torch.log2(want)).clamp(min=-6.0) - 3.0)
    s = torch.round(want / step) * step
    v = xn / s.clamp(min=1e-8)[..., None]
    a = v.abs().clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0))) - 1.0)
    if rule == 1:
        m = torch.round(a / step) * step
    elif rule == 2:
        m = torch.ceil(a / step - 0.5) * step
    else:
        h = torch.round(2.0 * a)
        m = torch.where(h <= 4, h / 2, torch.where(h <= 5, 2.0, torch.where(h <= 7, 3.0, torch.where(h <= 10, 4.0, 6.0))))
    return (torch.sign(v) * m * s[..., None]).view(n, kv, d) * scale.double()[:, None]


def _turned64(x, weight, s, case):
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight.double()
    half = case["rot"] // 2
    table = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None, :]
    out = x.clone()
    first, second = (slice(0, case["rot"], 2), slice(1, case["rot"], 2)) if case["interleaved"] else (
        slice(0, half), slice(half, case["rot"]))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    d, page = case["dim"], case["page"]
    if case["op"] == "rope":
        q, k = _turned64(s["q"], s["q_weight"], s, case), _turned64(s["k"], s["k_weight"], s, case)
        if not case["cache"]:
            return q, k
        # the cache is written from k rounded to its type
        k = k.to(_TYPES[case["x"]])
        return q, (_blocks64(k, s["k_global"], case["rule"]), _blocks64(s["v"], s["v_global"], case["rule"]))
    if case["op"] == "cache" and case["write"]:
        return _blocks64(s["k"], s["k_global"], case["rule"]), _blocks64(s["v"], s["v_global"], case["rule"])
    kc, ks, vc, vs = s["cache"]
    if case["op"] == "cache":
        p, o = s["slots"] // page, s["slots"] % page
        return (_decoded64(kc[p, :, o], ks[p, :, :, o])[..., :d] * s["k_global"].double()[:, None],
                _decoded64(vc[p, :, o], vs[p, :, :, o])[..., :d] * s["v_global"].double()[:, None])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv"]
    first = 0
    for b, (n, q) in enumerate(_shape(case)):
        pages = s["block_table"][b, :-(-n // page)].long()
        pos = torch.arange(n - q, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None, :]
        seen = j <= pos
        if case["window"]:
            seen = seen & ((pos - j < case["window"]) | (j < case["sinks"]))
        for h in range(case["kv"]):
            k = _decoded64(kc[pages, h].flatten(0, 1)[:n], ks[pages, h].transpose(1, 2).flatten(0, 1)[:n])[:, :d]
            v = _decoded64(vc[pages, h].flatten(0, 1)[:n], vs[pages, h].transpose(1, 2).flatten(0, 1)[:n])[:, :d]
            kt = (k * s["k_global"][h].double()).T.contiguous()
            for e in range(h * group, (h + 1) * group):
                z = torch.mm(s["q"][first:first + q, e].double(), kt) * d ** -0.5
                p = torch.softmax(z.masked_fill(~seen, -math.inf), dim=1)
                out[first:first + q, e] = torch.mm(p, v) * s["v_global"][h].double()
        first += q
    return out
