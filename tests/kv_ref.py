"""Plain references of the paged key-value cache, in binary64 on the CPU:
element decoding from the bit fields, the MX quantization by search over the
codes, attention by its definition, and the page bookkeeping one page at a
time."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
E4M3[127] = np.nan
FP4 = np.concatenate([E2M1, -E2M1])
FP8 = np.concatenate([E4M3, -E4M3])


def e8m0(b):
    v = np.ldexp(1.0, np.asarray(b).astype(np.int64) - 127)
    return np.where(np.asarray(b) == 255, np.nan, v)


def decode(fmt, x, s):
    """Elements [..., page, D or D / 2] and scales [..., D / 32, page] -> binary64 [..., page, D]."""
    if fmt == "bf16":
        return x.double().numpy()
    x = x.numpy()
    if fmt == "mxfp4":
        v = np.stack([FP4[x & 15], FP4[x >> 4]], -1).reshape(x.shape[:-1] + (-1,))
    else:
        v = FP8[x]
    return v * np.repeat(np.swapaxes(e8m0(s.numpy()), -1, -2), 32, -1)


def quantize(fmt, x):
    """binary64 [..., D] -> (codes as integers [..., D], scale bytes [..., D / 32])."""
    grid, emax = (E2M1, 2) if fmt == "mxfp4" else (E4M3[:127], 8)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 1 - emax, -127)
    e = np.clip(e, -127, 127)
    y = np.minimum(np.abs(b) / np.ldexp(1.0, e)[..., None], grid[-1])
    hi = np.minimum(np.searchsorted(grid, y), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - y, y - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code + np.where(np.signbit(b), len(E2M1) if fmt == "mxfp4" else 128, 0)
    return code.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8)


def visible(n, pos, window, sinks):
    """Which of n tokens the query at pos sees."""
    j = np.arange(n)
    on = j <= pos
    if window > 0:
        on &= (j > pos - window) | (j < sinks)
    return on


def rows_of(values, table_row, n, kv_head):
    """K or V rows [n][D] of one sequence and head from decoded pages [pages][heads][page][D]."""
    ps = values.shape[2]
    pages = [int(p) for p in table_row[:(n + ps - 1) // ps]]
    # a page that the sequence no longer has stands for tokens that no query may see
    got = [values[p, kv_head] if p >= 0 else np.full(values[0, kv_head].shape, np.nan) for p in pages]
    return np.concatenate(got)[:n] if got else np.zeros((0, values.shape[-1]))


def attention(q, k, v, pos, window, sinks, scale):
    """One query over rows k, v: (out, lse, sum of weight * |v|, the largest
    sum |q k| scale, visible count) in binary64."""
    on = visible(len(k), pos, window, sinks)
    if not on.any():
        return np.zeros(v.shape[-1]), -math.inf, np.zeros(v.shape[-1]), 0.0, 0
    k, v = k[on], v[on]
    s = (k @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    t = p.sum()
    reach = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    return (p @ v) / t, m + math.log(t), (p @ np.abs(v)) / t, reach, int(on.sum())


def attention_tolerance(dim, o, weight, lse, reach, n):
    """What the kernels' roundings allow: the output rounded to bfloat16 (2^-8
    relative), the softmax weights rounded to bfloat16 (2^-8 of each), binary32
    scores (dim products and the scaling, to first order in the exponential)
    and binary32 sums over n tokens; exp2 and log within a few units."""
    score = (dim + 8) * 2.0 ** -24 * reach + 2.0 ** -22
    rel = 2.0 ** -8 + 2 * score + (n + 64) * 2.0 ** -23
    return 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7) + rel * weight + 1e-30, \
        score + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + abs(lse) if math.isfinite(lse) else 1)


class RefPool:
    """The page bookkeeping, one page at a time."""

    def __init__(self, table, lens, refs, ps):
        self.table, self.lens, self.refs, self.ps = table.copy(), lens.copy(), refs.copy(), ps
        self.moves = []

    @property
    def free(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def reserve(self, rows, tokens):
        free, plan, named = self.free, [], set()
        for i, (s, t) in enumerate(zip(rows, tokens)):
            if not 0 <= s < len(self.lens) or s in named or t < 0 or self.lens[s] < 0:
                return i
            named.add(s)
            have, want = -(-self.lens[s] // self.ps), -(-(self.lens[s] + t) // self.ps)
            if want > self.table.shape[1] or want - have > len(free):
                return i
            plan.append((s, t, have, free[:want - have]))
            free = free[want - have:]
        for s, t, have, pages in plan:
            for j, p in enumerate(pages):
                self.table[s, have + j] = p
                self.refs[p] = 1
            self.lens[s] += t
        return -1

    def fork(self, parents, children):
        free, plan, named = self.free, [], set()
        for i, (a, c) in enumerate(zip(parents, children)):
            ok = 0 <= a < len(self.lens) and 0 <= c < len(self.lens) and a != c and c not in named
            if not ok or self.lens[c] != 0 or self.lens[a] < 0 or -(-self.lens[a] // self.ps) > self.table.shape[1]:
                return i
            named.add(c)
            new = None
            if self.lens[a] % self.ps:
                if not 0 <= self.table[a, self.lens[a] // self.ps] < len(self.refs) or not free:
                    return i
                new, free = free[0], free[1:]
            plan.append((a, c, self.lens[a], new))
        for a, c, n, new in plan:
            full = n // self.ps
            row = np.full(self.table.shape[1], -1, self.table.dtype)
            row[:full] = self.table[a, :full]
            for p in row[:full]:
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
            if new is not None:
                self.moves.append((int(self.table[a, full]), new))
                row[full] = new
                self.refs[new] = 1
            self.table[c], self.lens[c] = row, n
        return -1

    def release(self, rows, window=0, sinks=0):
        for s in rows:
            if not 0 <= s < len(self.lens):
                continue
            for j in range(self.table.shape[1]):
                if window > 0 and not (j * self.ps >= sinks and (j + 1) * self.ps <= self.lens[s] - window):
                    continue
                p = self.table[s, j]
                if 0 <= p < len(self.refs):
                    self.refs[p] -= 1
                self.table[s, j] = -1
            if window == 0:
                self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.moves.append((s, d))
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = np.array([[to.get(int(p), p) for p in row] for row in self.table],
                              self.table.dtype).reshape(self.table.shape)
        return live


def torch_table(lens, ps, width, pages, rng):
    """A page table for these lengths: random distinct pages, -1 beyond."""
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // ps)
        table[b, :k] = order[at:at + k]
        at += k
    assert at <= pages
    return torch.from_numpy(table)
