"""Float64 definitions of the serving operators (include/wbserve.h): page planning, cache
writes, attention of one token over a paged cache, the norm with an e4m3 output. Written
from the formulas; nothing is shared with the GPU code."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values of the 1-4-3 format: bias 7, subnormals below 2^-6, no infinities,
    exponent and mantissa all ones NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -v if b & 128 else v
    return out


def e4m3_half_step(x):
    """Half the distance of neighbouring e4m3 values around |x| <= 448."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 0.5 * 2.0 ** (e - 3)


def group_scale(x):
    """Scale of a group along the last axis: max|x| / 448, at least 2^-126 unless all are 0."""
    top = np.max(np.abs(x), axis=-1)
    return np.where(top > 0, np.maximum(top / E4M3_MAX, 2.0 ** -126), 0.0)


def plan(lens, more, table, free, n_free, page, n_slots):
    """(table, slots, starts, lens, n_free, status), one request and token after the other."""
    R, width = table.shape
    none = (table.copy(), np.full(n_slots, -1, np.int64), np.zeros(R + 1, np.int32), np.array(lens), n_free)
    if min(lens) < 0 or min(more) < 0 or not 0 <= n_free <= len(free):
        return none + (1,)
    have = [-(-int(n) // page) for n in lens]
    want = [-(-(int(n) + int(m)) // page) for n, m in zip(lens, more)]
    if max(want) > width:
        return none + (2,)
    if sum(int(m) for m in more) > n_slots:
        return none + (3,)
    if sum(want) - sum(have) > n_free:
        return none + (4,)
    table, slots, starts = none[0], none[1], none[2]
    at = 0
    for r in range(R):
        starts[r] = at
        for j in range(have[r], want[r]):
            n_free -= 1
            table[r, j] = free[n_free]
        for t in range(int(lens[r]), int(lens[r]) + int(more[r])):
            slots[at] = int(table[r, t // page]) * page + t % page
            at += 1
    starts[R] = at
    return table, slots, starts, np.array(lens) + np.array(more), n_free, 0


def release(ended, lens, table, free, n_free, page):
    """(lens, free, n_free, status)."""
    lens, free = np.array(lens), np.array(free)
    if min(lens) < 0 or not 0 <= n_free <= len(free):
        return lens, free, n_free, 1
    pages = [-(-int(n) // page) if e else 0 for n, e in zip(lens, ended)]
    if max(pages) > table.shape[1]:
        return lens, free, n_free, 2
    if n_free + sum(pages) > len(free):
        return lens, free, n_free, 4
    for r, n in enumerate(pages):
        free[n_free:n_free + n] = table[r, :n]
        n_free += n
        if ended[r]:
            lens[r] = 0
    return lens, free, n_free, 0


def attend(q, k, v, scale, window=0):
    """One request: q [Hq, D], k and v [n, H, D] (its stored tokens, in order). Returns
    (o [Hq, D], lse [Hq], mean |v| under the weights [Hq, D], sum |scale q k| at most [Hq])."""
    Hq, D = q.shape
    n, H, _ = k.shape
    first = max(0, n - window) if window else 0
    o, w = np.zeros((Hq, D)), np.zeros((Hq, D))
    lse, size = np.full(Hq, -np.inf), np.zeros(Hq)
    for h in range(Hq):
        kh, vh = k[first:, h // (Hq // H)], v[first:, h // (Hq // H)]
        if n - first <= 0:
            continue
        s = scale * (kh @ q[h])
        size[h] = np.max(abs(scale) * (np.abs(kh) @ np.abs(q[h])))
        top = s.max()
        if top == -np.inf:
            continue
        e = np.exp(s - top)
        o[h] = e @ vh / e.sum()
        w[h] = e @ np.abs(vh) / e.sum()
        lse[h] = top + math.log(e.sum())
    return o, lse, w, size


def norm(x, residual, weight, eps, group):
    """(h, y, scales): h the row that is stored, y its norm, a scale for each group."""
    h = x if residual is None else x + residual
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    D = x.shape[1]
    step = group or D
    scales = np.stack([group_scale(y[:, i:i + step]) for i in range(0, D, step)], axis=1)
    return h, y, scales
