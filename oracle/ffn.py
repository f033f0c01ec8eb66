"""CPU oracle of the feed-forward operators on NVFP4 weights (test
infrastructure only): the linear layer with a fused epilogue and the
mixture-of-experts layer, in float64 with numpy.

Besides the values, each function returns how far a computation that sums in
fp32 may be from them, before the last rounding:

* a sum of k products that fp32 holds exactly, added 32 at a time by the matrix
  cores into one fp32 accumulator and then over a few accumulators, errs by at
  most (k / 32 + 40) 2^-23 sum |x w| (one unit in the last place per addition,
  twice the half unit of a correctly rounded one);
* an activation errs by 1.2 times the error of its argument (the largest slope
  of the four, GELU's, is 1.13) and by 2^-20 of |f(z)| + min(|z|, 1) of its own
  (exp, erfc and a handful of fp32 operations around them);
* products and sums of such values follow the usual rules, with one more fp32
  rounding each.
"""
from __future__ import annotations

import math

import numpy as np

from . import reference as ref

U23 = 2.0 ** -23
PLANE_ERROR = {2: 2.0 ** -17, 3: 2.0 ** -24}   # relative error of h kept in 2 or 3 bf16 planes

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def weights(codes, scales) -> np.ndarray:
    """float64 (..., k) from uint8 codes (..., k/2) and scales (..., k/16)."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8)
    t = ref.e2m1_table()
    w = np.stack((t[codes & 15], t[codes >> 4]), axis=-1).reshape(*codes.shape[:-1], -1)
    return w * np.repeat(ref.e4m3_table()[scales], 16, axis=-1)


def activation(name, z):
    if name == "none":
        return z
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2.0))
        if name == "gelu_tanh":
            return z / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1.0 + np.exp(-z))
    raise ValueError(name)


def _product(x, w, dx=0.0):
    """x w^T with |error|, for x known to within dx."""
    a = np.abs(x) @ np.abs(w).T
    err = (x.shape[1] / 32 + 40) * U23 * a
    if np.any(dx):
        err = err + np.asarray(dx) @ np.abs(w).T
    return x @ w.T, err


def _activated(name, z, dz):
    f = activation(name, z)
    if name == "none":
        return f, dz
    return f, 1.2 * dz + 2.0 ** -20 * (np.abs(f) + np.minimum(np.abs(z), 1.0))


def _times(a, da, b, db):
    return a * b, np.abs(a) * db + np.abs(b) * da + da * db + U23 * np.abs(a * b)


def linear(x, codes, scales, alpha=None, bias=None, residual=None, act="none", gated=False):
    """(values, error) of residual + f(alpha x W^T + bias) [* up]; codes and
    scales (groups, m, .), alpha (groups,), bias (groups * m,)."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        parts = []
        m = codes.shape[1]
        for g in range(2 if gated else 1):
            z, dz = _product(x, weights(codes[g], scales[g]))
            a = 1.0 if alpha is None else float(alpha[g])
            z, dz = a * z, abs(a) * dz + U23 * np.abs(a * z)
            if bias is not None:
                z = z + np.asarray(bias[g * m:(g + 1) * m], np.float64)
                dz = dz + U23 * np.abs(z)
            parts.append((z, dz))
        y, dy = _activated(act, *parts[0])
        if gated:
            y, dy = _times(y, dy, *parts[1])
        if residual is not None:
            y = y + np.asarray(residual, np.float64)
            dy = dy + U23 * np.abs(y)
    return y, dy


def route(x, router, topk, route_bias=None, scoring="softmax", renormalize=True, scale=1.0):
    """(experts (tokens, topk), weights (tokens, topk)): the lowest index first
    among equal keys, NaN keys last.  Without a route_bias the keys are the logits,
    which order the experts as the exact scores do."""
    z = np.asarray(x, np.float64) @ np.asarray(router, np.float64).T
    with np.errstate(invalid="ignore", over="ignore"):
        if scoring == "softmax":
            s = np.exp(z - z.max(axis=1, keepdims=True))
            s = s / s.sum(axis=1, keepdims=True)
        else:
            s = 1.0 / (1.0 + np.exp(-z))
        key = z if route_bias is None else s + np.asarray(route_bias, np.float64)
    key = np.where(np.isnan(key), -np.inf, np.maximum(key, -np.finfo(np.float64).max))
    order = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    w = np.take_along_axis(s, order, axis=1)
    if renormalize:
        with np.errstate(invalid="ignore", divide="ignore"):
            w = w / w.sum(axis=1, keepdims=True)
    return order, w * scale


def moe(x, router, codes13, scales13, codes2, scales2, topk, alpha13=None, alpha2=None, route_bias=None,
        residual=None, act="silu", scoring="softmax", renormalize=True, scale=1.0, planes=2):
    """(values, error) of the mixture-of-experts layer."""
    x = np.asarray(x, np.float64)
    order, w = route(x, router, topk, route_bias, scoring, renormalize, scale)
    y = np.zeros((x.shape[0], codes2.shape[1]))
    dy = np.zeros_like(y)
    size = np.zeros_like(y)
    with np.errstate(invalid="ignore", over="ignore"):
        for e in np.unique(order):
            t, j = np.nonzero(order == e)
            parts = []
            for g in range(2):
                z, dz = _product(x[t], weights(codes13[2 * e + g], scales13[2 * e + g]))
                a = 1.0 if alpha13 is None else float(alpha13[e][g])
                parts.append((a * z, abs(a) * dz + U23 * np.abs(a * z)))
            f, df = _activated(act, *parts[0])
            h, dh = _times(f, df, *parts[1])
            dh = dh + PLANE_ERROR[planes] * np.abs(h)
            # one product per plane adds into the same sums
            o, do = _product(h, weights(codes2[e], scales2[e]), dh)
            do = do + (planes - 1) * h.shape[1] / 32 * U23 * (np.abs(h) @ np.abs(weights(codes2[e], scales2[e])).T)
            c = (1.0 if alpha2 is None else float(alpha2[e])) * w[t, j][:, None]
            y[t] += c * o
            dy[t] += np.abs(c) * do + 4 * U23 * np.abs(c * o)
            size[t] += np.abs(c * o)
        dy = dy + topk * U23 * size
        if residual is not None:
            y = y + np.asarray(residual, np.float64)
            dy = dy + U23 * np.abs(y)
    return y, dy
