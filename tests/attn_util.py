"""Inputs, calls and comparisons shared by the tests of the attention operators."""
import numpy as np
import torch

import precision_decode_amd as pd
from ffn_util import TYPES, rounded
from oracle import attn as oa

# finite E4M3 codes up to 16 in size, subnormal and negative ones among them
FINITE = np.array([c for c in range(256) if (c & 0x7F) <= 0x58], dtype=np.uint8)
NAN_SCALES = np.array([0x7F, 0xFF], dtype=np.uint8)


def filled(rng, pages, kv, page, dim, nan=False, scale_codes=FINITE):
    """A cache whose slots all hold something: finite blocks, or NaN ones."""
    c = oa.empty(pages, kv, page, dim)
    codes = scale_codes if not nan else NAN_SCALES
    for n in ("kc", "vc"):
        c[n][..., :dim // 2] = rng.integers(0, 256, size=c[n][..., :dim // 2].shape, dtype=np.uint8)
    for n in ("ks", "vs"):
        c[n][:, :, :dim // 16] = codes[rng.integers(0, len(codes), size=c[n][:, :, :dim // 16].shape)]
    c["kg"] = rng.uniform(0.05, 0.2, kv).astype(np.float32)
    c["vg"] = rng.uniform(0.5, 2.0, kv).astype(np.float32)
    return c


def tables(rng, lengths, page, pages, width=None):
    """Block tables of sequences whose pages are all different; unused entries lead outside."""
    counts = [-(-int(n) // page) for n in lengths]
    width = max(max(counts), 1) if width is None else width
    assert sum(counts) <= pages and max(counts) <= width
    order = rng.permutation(pages)
    t = np.full((len(lengths), width), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(counts):
        t[b, :n] = order[at:at + n]
        at += n
    return t, order[at:]


def on_device(cache, dim):
    d = {n: None if v is None else torch.from_numpy(v.copy()).cuda() for n, v in cache.items()}
    return pd.KvCache(d["kc"], d["ks"], d["vc"], d["vs"], head_dim=dim, k_global=d["kg"], v_global=d["vg"])


def back(kv):
    """The oracle's form of a cache on the device."""
    names = ("kc", "ks", "vc", "vs", "kg", "vg")
    return {n: None if t is None else t.cpu().numpy() for n, t in zip(names, kv.tensors)}


def heads_on_device(values, kind, token=None, head=None, offset=0):
    """Device tensor (tokens, heads, dim) of the values with those strides, NaN around."""
    v = torch.from_numpy(np.ascontiguousarray(values, dtype=np.float64)).to(TYPES[kind])
    n, hn, d = v.shape
    head = d if head is None else head
    token = hn * head if token is None else token
    size = offset + max(n - 1, 0) * token + (hn - 1) * head + d + 16
    store = torch.full((size,), float("nan"), dtype=TYPES[kind]).cuda()
    view = torch.as_strided(store, (n, hn, d), (token, head, 1), offset)
    view.copy_(v.cuda())
    return view


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def i64(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int64)).cuda()


def queries(rng, tokens, heads, dim, kind, size=1.0):
    return rounded(rng.standard_normal((tokens, heads, dim)) * size, kind)
