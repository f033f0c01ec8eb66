"""CPU oracle of the attention operators on an NVFP4 cache (test infrastructure
only): the cache's layout, head norms with the position rotation, and attention,
in float64 with numpy.

A cache is a dict of codes ``kc``, ``vc`` (pages, kv heads, page size, dp / 2),
scales ``ks``, ``vs`` (pages, kv heads, dp / 16, page size) and globals ``kg``,
``vg`` (kv heads,) or None.  Besides values, the functions return how far a
computation in fp32 may be from them, before the last rounding:

* a score is a sum of d products that are exact in fp32, added 32 at a time into
  an fp32 accumulator, times one factor of three roundings, and enters an exp2
  whose argument is rounded once more: (d / 32 + 12) 2^-23 of scale sum |q k|, plus
  2^-23 of the row's largest |score| (the subtracted maximum), in units of the
  natural logarithm.  A weight then errs by that much relatively, and by 2^-21 of
  its own (exp2, its sum);
* the weight that meets v is rounded to fp16 after scaling the largest to 2^8 at
  least: 2^-11 relatively, and 2^-25 / 2^8 of the largest where it is subnormal;
* sums over n tokens err by (n / 32 + 60) 2^-23 of their absolute sum (each
  rescaling of the running sums among them).
"""
from __future__ import annotations

import numpy as np

from . import quantize as oq
from . import reference as ref

U23 = 2.0 ** -23


def padded(dim):
    return -(-dim // 64) * 64


def empty(pages, kv, page, dim, fill=0):
    dp = padded(dim)
    c = {n: np.full((pages, kv, page, dp // 2), fill, np.uint8) for n in ("kc", "vc")}
    c.update({n: np.full((pages, kv, dp // 16, page), fill, np.uint8) for n in ("ks", "vs")})
    return dict(c, kg=None, vg=None)


def write(cache, k, v, slots, rule):
    """Quantises k and v (tokens, kv, dim) float32 into the slots, in place."""
    pages, kv, page, half = cache["kc"].shape
    dim = k.shape[2]
    for x, codes, scales, g in ((k, "kc", "ks", "kg"), (v, "vc", "vs", "vg")):
        for h in range(kv):
            scale = np.float32(1.0) if cache[g] is None else np.float32(cache[g][h])
            with np.errstate(all="ignore"):
                packed, sf = oq.quantize_with_scale(x[:, h], scale, rule)
            for t, s in enumerate(slots):
                if 0 <= s < pages * page:
                    p, o = divmod(int(s), page)
                    cache[codes][p, h, o] = 0
                    cache[codes][p, h, o, :dim // 2] = packed[t]
                    cache[scales][p, h, :, o] = 0
                    cache[scales][p, h, :dim // 16, o] = sf[t]


def values(codes, scales):
    """float64 (..., dp) of codes (..., dp / 2) and scales (..., dp / 16)."""
    t = ref.e2m1_table()
    w = np.stack((t[codes & 15], t[codes >> 4]), axis=-1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return w * np.repeat(ref.e4m3_table()[scales], 16, axis=-1)


def read(cache, slots, dim):
    """float32 k and v (tokens, kv, dim) of the slots, zeros where one is outside."""
    pages, kv, page, _ = cache["kc"].shape
    out = []
    for codes, scales, g in (("kc", "ks", "kg"), ("vc", "vs", "vg")):
        x = np.zeros((len(slots), kv, dim), np.float32)
        for t, s in enumerate(slots):
            if 0 <= s < pages * page:
                p, o = divmod(int(s), page)
                w = values(cache[codes][p, :, o], cache[scales][p, :, :, o])[:, :dim].astype(np.float32)
                x[t] = w if cache[g] is None else w * np.asarray(cache[g], np.float32)[:, None]
        out.append(x)
    return out


def norm_rope(x, weight, positions, cos_sin, eps, interleaved):
    """(values, error) of rows x (tokens, heads, dim): dim / 2 + 10 roundings at most
    up to the normalised element (the sum of squares counts half in its root), then
    two products and a sum."""
    y, dim = x.astype(np.float64), x.shape[2]
    rel = 0.0
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * weight.astype(np.float64)
        rel = (dim / 2 + 10) * 2.0 ** -24
    out, err = y.copy(), np.abs(y) * rel
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    if rot:
        half = rot // 2
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
        ok = (positions >= 0) & (positions < cos_sin.shape[0])
        row = cos_sin[np.where(ok, positions, 0)].astype(np.float64)[:, None, :]
        c, s = row[..., :half], row[..., half:]
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        err[..., a] = (np.abs(y[..., a] * c) + np.abs(y[..., b] * s)) * (rel + 3 * 2.0 ** -24)
        err[..., b] = (np.abs(y[..., b] * c) + np.abs(y[..., a] * s)) * (rel + 3 * 2.0 ** -24)
        out[~ok] = np.nan
    return out, err


def attention(q, cache, table, lengths, starts, scale, window=0, sinks=0):
    """(values, error) of q (tokens, heads, dim); rows of no sequence are NaN."""
    pages, kv, page, _ = cache["kc"].shape
    tokens, heads, dim = q.shape
    out = np.full(q.shape, np.nan)
    err = np.zeros(q.shape)
    group = heads // kv
    for b, n in enumerate(lengths):
        n, x, y = int(n), int(starts[b]), int(starts[b + 1])
        j = np.arange(n)
        at = np.asarray(table[b], np.int64)[j // page] if n else np.zeros(0, np.int64)
        there = (at >= 0) & (at < pages)
        at = np.where(there, at, 0)
        for h in range(kv):
            k = values(cache["kc"][at, h, j % page], cache["ks"][at, h, :, j % page])[:, :dim]
            v = values(cache["vc"][at, h, j % page], cache["vs"][at, h, :, j % page])[:, :dim]
            k = k if cache["kg"] is None else k * float(cache["kg"][h])
            v = v if cache["vg"] is None else v * float(cache["vg"][h])
            for i in range(y - x):
                p = n - (y - x) + i
                seen = there & (j <= p)
                if window:
                    seen &= (j > p - window) | (j < sinks)
                rows = slice(h * group, (h + 1) * group)
                if not seen.any():
                    out[x + i, rows] = 0.0
                    continue
                qs, ks, vs = q[x + i, rows].astype(np.float64), k[seen], v[seen]
                with np.errstate(all="ignore"):
                    z = scale * qs @ ks.T
                    dz = abs(scale) * np.abs(qs) @ np.abs(ks).T * (dim / 32 + 12) * U23
                    dz = dz + np.abs(z).max(axis=1, keepdims=True) * U23
                    w = np.exp(z - z.max(axis=1, keepdims=True))
                    top = w.max(axis=1, keepdims=True)
                    total = w.sum(axis=1, keepdims=True)
                    out[x + i, rows] = (w / total) @ vs
                    rel = 2 * dz.max(axis=1, keepdims=True) + 2.0 ** -21 + 2.0 ** -11 + \
                        2 * (len(ks) / 32 + 60) * U23
                    err[x + i, rows] = (w / total) @ np.abs(vs) * rel + \
                        (top / total) @ np.abs(vs).sum(axis=0, keepdims=True) * 2.0 ** -33
    return out, err
