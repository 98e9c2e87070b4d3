"""A paged cache of keys and values, rotary positions and attention, in float64.

TEST INFRASTRUCTURE, NOT PRODUCT CODE: imported only by tests/; shares no code
with the library.

Plain numpy, one token after the other, from the definitions:

* key_index, value_index: where element d of place o stands in a page of one head;
* turn: pair (a, b) becomes (a cos t - b sin t, a sin t + b cos t), t = position of
  the pair's axis times its frequency;
* attend: softmax over the keys that a token sees of cap tanh(scale q k / cap) -
  slope |distance|, times the values; with bounds on a float32 evaluation whose
  weights are rounded to bf16.
"""
from __future__ import annotations

import numpy as np

__all__ = ["key_index", "value_index", "read_cache", "turn", "visible", "attend", "BF16_HALF", "U"]

U = 2.0 ** -23          # one float32 step: matrix instructions may cut where others round
BF16_HALF = 2.0 ** -8   # half a bf16 step, relative


def key_index(o, d, dim):
    return ((o // 32 * (dim // 8) + d // 8) * 32 + o % 32) * 8 + d % 8


def value_index(o, d, dim):
    return ((o // 16 * 2 + o // 4 % 2) * dim + d) * 8 + o // 8 % 2 * 4 + o % 4


def read_cache(cache, table, length, key, absent=np.nan):
    """Rows [length, kv_heads, dim] of a sequence from cache [pages, kv_heads, page, dim]
    (any element type); places whose page is not one of the cache's become `absent`."""
    pages, kv, page, dim = cache.shape
    flat = cache.reshape(pages, kv, page * dim)
    out = np.empty((length, kv, dim), dtype=cache.dtype)
    d = np.arange(dim)
    for p in range(length):
        n = table[p // page] if p // page < len(table) else -1
        at = (key_index if key else value_index)(p % page, d, dim)
        out[p] = flat[n][:, at] if 0 <= n < pages else absent
    return out


def turn(x, angles, adjacent):
    """x [tokens, heads, dim], angles [tokens, pairs]."""
    y = np.array(x, dtype=np.float64)
    pairs = angles.shape[1]
    for j in range(pairs):
        a, b = (2 * j, 2 * j + 1) if adjacent else (j, j + pairs)
        c, s = np.cos(angles[:, j])[:, None], np.sin(angles[:, j])[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
    return y


def visible(i, count, length, window=0, prefix=0, first=0, masks=None):
    """(keys that token i of a sequence sees, their distances).  masks: the sequence's rows
    as whole numbers, bit j for its drafted token j."""
    start = length - count
    position = lambda j: start + bin(masks[j]).count("1") - 1 if masks is not None else start + j  # noqa: E731
    keys, far = [], []
    for k in range(length):
        if masks is None:
            seen = k <= start + i or k < prefix
        else:
            seen = k < start or masks[i] >> (k - start) & 1 == 1
        drafted = masks is not None and 0 <= k - start < count
        distance = position(i) - (position(k - start) if drafted else k)
        if seen and k >= first and (window == 0 or distance < window):
            keys.append(k)
            far.append(distance)
    return np.array(keys, dtype=np.int64), np.array(far, dtype=np.float64)


def attend(q, keys, values, count, length, scale, cap=0.0, window=0, slopes=None, prefix=0, first=None, masks=None,
           y_half=BF16_HALF):
    """One sequence: q [count, heads, dim], keys and values [length, kv_heads, dim] (NaN rows
    of keys: no page).  Returns y, lse and how far float32 results may be off each.

    With u a float32 step, a product of dim terms is off by at most dim u |q||k|, a
    score's further steps by 8 u of their own magnitudes (a capped one's, too, by 8 u of
    the smaller of score and cap, and 4 u of a cap up to 128), so that a weight is off by
    the factor 1 + 2 e, e = the score's error + 4 u.
    Weights are rounded to bf16 (2^-8) before the product with the values, their sum is
    not; sums of n terms are off by n u.  y is rounded once (y_half)."""
    heads, kv = q.shape[1], keys.shape[1]
    y, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    dy, dl = np.zeros(q.shape), np.zeros(q.shape[:2])
    there = ~np.isnan(keys).all(axis=(1, 2))
    for i in range(count):
        at, far = visible(i, count, length, window, prefix, 0 if first is None else first[i], masks)
        far, at = far[there[at]], at[there[at]]
        if len(at) == 0:
            continue
        for h in range(heads):
            k, v = keys[at, h * kv // heads], values[at, h * kv // heads]
            x = scale * (k @ q[i, h])
            e = q.shape[2] * U * scale * (np.abs(k) @ np.abs(q[i, h])) + 8 * U * np.abs(x)
            if cap:
                e += 8 * U * np.minimum(cap, np.abs(x)) + (4 * U * cap if cap <= 128 else 0)
                x = cap * np.tanh(x / cap)
            if slopes is not None:
                x = x - slopes[h] * np.abs(far)
                e += 8 * U * np.abs(slopes[h] * far) + 8 * U * np.abs(x)
            e = e + 4 * U
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            y[i, h] = p @ v / l
            lse[i, h] = m + np.log(l)
            err = 2 * (p @ e) / l + (len(at) + 8) * U
            size = p @ np.abs(v) / l
            dy[i, h] = (p * (BF16_HALF + 2 * e)) @ np.abs(v) / l + size * (err + (len(at) + 8) * U) * 1.01
            dy[i, h] = dy[i, h] * (1 + y_half) + y_half * np.abs(y[i, h])
            dl[i, h] = err + 8 * U * (1 + abs(m) + abs(lse[i, h]))
    return y, lse, dy, dl
