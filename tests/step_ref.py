"""Plain references, on the CPU, of the operators around a decode step's products:
the rotation by positions (angles in extended precision), the choice of experts
and the experts' layer in binary64, with bounds on what the kernels' roundings
allow. Written from the formulas, not from the kernels."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv_ref as R

U = 2.0 ** -24  # half a step of binary32, relative


def spin(pos, freq, factor):
    """factor * cos and sin of pos * freq, [len(pos)][len(freq)]. The product is
    taken in extended precision (64 bits): positions of 2^31 lose 1e-10."""
    a = np.asarray(pos).astype(np.longdouble)[:, None] * np.asarray(freq).astype(np.longdouble)[None]
    return (np.cos(a) * factor).astype(np.float64), (np.sin(a) * factor).astype(np.float64)


def turn(x, pos, freq, layout, factor=1.0):
    """x [tokens][heads][dim] binary64 -> (turned, tolerance of binary32 kernels).

    Cosine and sine: the angle has 32 bits of a turn, is rounded to binary32 and
    multiplied by a rounded constant (3 U of at most pi / 4, times a slope of at most
    0.71), the series and its last step round by U in all, the factor by U: within
    4 U of the factor. Then a product, a fused multiply-add and their roundings."""
    n = len(freq)
    c, s = (v[:, None] for v in spin(pos, freq, factor))
    i = np.arange(n)
    p, q = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    out, tol = x.copy(), np.zeros_like(x)
    a, b = x[..., p], x[..., q]
    out[..., p], out[..., q] = a * c - b * s, b * c + a * s
    reach = (np.abs(a) + np.abs(b)) * factor * 5 * U
    tol[..., p], tol[..., q] = reach + U * np.abs(out[..., p]), reach + U * np.abs(out[..., q])
    return out, tol * (1 + 1e-6)


def allowed_codes(fmt, y, tol):
    """For values known to +- tol ([..., D]): the least and largest scale byte of
    each block, and codes (as values) of y - tol and y + tol under each."""
    grid, emax = (R.E2M1, 2) if fmt == "mxfp4" else (R.E4M3[:127], 8)
    b, t = y.reshape(y.shape[:-1] + (-1, 32)), tol.reshape(y.shape[:-1] + (-1, 32))

    def exponent(top):
        e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 1 - emax, -127)
        return np.clip(e, -127, 127)

    e0 = exponent(np.maximum(np.abs(b) - t, 0).max(-1))
    e1 = exponent((np.abs(b) + t).max(-1))

    def rounded(v, e):
        m = np.minimum(np.abs(v) / np.ldexp(1.0, e)[..., None], grid[-1])
        hi = np.minimum(np.searchsorted(grid, m), len(grid) - 1)
        lo = np.maximum(hi - 1, 0)
        up, down = grid[hi] - m, m - grid[lo]
        i = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        return np.copysign(grid[i], v) * np.ldexp(1.0, e)[..., None]

    span = [(e, rounded(b - t, e), rounded(b + t, e)) for e in (e0, e1)]
    return e0, e1, span


def check_block(fmt, codes, scales, y, tol, what):
    """Stored codes [..., D or D / 2] and scale bytes [..., D / 32] against y +- tol."""
    if fmt == "mxfp4":
        v = np.stack([R.FP4[codes & 15], R.FP4[codes >> 4]], -1).reshape(y.shape)
    else:
        v = R.FP8[codes].reshape(y.shape)
    e = scales.astype(np.int64) - 127
    v = v.reshape(y.shape[:-1] + (-1, 32)) * np.ldexp(1.0, e)[..., None]
    e0, e1, span = allowed_codes(fmt, y, tol)
    ok = np.zeros(v.shape, bool)
    for ee, lo, hi in span:
        ok |= (e == ee)[..., None] & (lo <= v) & (v <= hi)
    assert ok.all(), "%s: %d of %d codes outside their bounds, first at %s" % (
        what, (~ok).sum(), ok.size, np.argwhere(~ok)[0])


def route(x, w, bias, top, normalize):
    """(ids, weights, least gap between a chosen logit and the next) in binary64."""
    logits = x @ w.T
    if bias is not None:
        logits = logits + bias
    order = np.argsort(-logits, axis=-1, kind="stable")
    ids = order[:, :top]
    val = np.take_along_axis(logits, ids, 1)
    over = val if normalize else logits
    best = over.max(-1, keepdims=True)
    weights = np.exp(val - best) / np.exp(over - best).sum(-1, keepdims=True)
    ranked = np.take_along_axis(logits, order, 1)
    gap = np.diff(-ranked[:, :top + 1], axis=-1).min() if logits.shape[1] > 1 else math.inf
    return ids, weights, gap


def decode(fmt, codes, scales, scale2=None):
    """Experts' weights [experts][rows][k] in binary64."""
    v = np.stack([R.FP4[codes & 15], R.FP4[codes >> 4]], -1).reshape(codes.shape[:-1] + (-1,))
    if fmt == "mxfp4":
        return v * np.repeat(R.e8m0(scales), 32, -1)
    return v * np.repeat(R.FP8[scales], 16, -1) * np.asarray(scale2, np.float64)[:, None, None]


def experts(x, ids, weights, w13, w2):
    """(out [tokens][hidden], tolerance): the layer in binary64, and what binary32
    sums in any order (k U of the sum of magnitudes), the sigmoid (the exponent's
    rounding, |g| 2 U of its value, and 4 U), h in two bfloat16 halves (2^-16) and the
    factors' roundings allow; the output's own rounding to bfloat16 comes last."""
    tokens, inter, hidden = len(x), w13.shape[1] // 2, w2.shape[1]
    out, tol = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for t in range(tokens):
        for e, w in zip(ids[t], weights[t]):
            if not 0 <= e < len(w13):
                continue
            z = w13[e] @ x[t]
            dz = (hidden + 8) * U * (np.abs(w13[e]) @ np.abs(x[t]))
            g, u, dg, du = z[:inter], z[inter:], dz[:inter], dz[inter:]
            with np.errstate(over="ignore"):
                sig = 1 / (1 + np.exp(-g))
            h = g * sig * u
            dh = 1.1 * dg * np.abs(u) + np.abs(g * sig) * du + dg * du + np.abs(h) * (2.0 ** -16 + (2 * np.abs(g) + 8) * U)
            y = w2[e] @ h
            dy = np.abs(w2[e]) @ dh + (2 * inter + 16) * U * (np.abs(w2[e]) @ np.abs(h))
            out[t] += w * y
            tol[t] += abs(w) * (dy + (len(ids[t]) + 8) * U * np.abs(y))
    return out, tol * (1 + 1e-3) + 2.0 ** -8 * (np.abs(out) + tol) + 1e-38


def bf16(rng, *shape, gain=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * gain).astype(np.float32)).to(torch.bfloat16)


def layer(rng, fmt, n, hidden, inter):
    """Random codes and scales of n experts, as numpy arrays (factors None for mxfp4)."""
    out = []
    for rows, k in ((2 * inter, hidden), (hidden, inter)):
        codes = rng.integers(0, 256, (n, rows, k // 2), dtype=np.uint8)
        if fmt == "mxfp4":
            mid = 126 - int(round(math.log2(k) / 2))
            out += [codes, rng.integers(mid - 2, mid + 2, (n, rows, k // 32)).astype(np.uint8), None]
        else:
            out += [codes, rng.integers(0x28, 0x41, (n, rows, k // 16)).astype(np.uint8),
                    (rng.uniform(0.3, 0.6, n) * k ** -0.5).astype(np.float32)]
    return out
