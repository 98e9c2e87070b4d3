"""Routing of tokens to experts and back, and low-rank adapters, in float64.

TEST INFRASTRUCTURE, NOT PRODUCT CODE: imported only by tests/; shares no code
with the library.

Plain numpy, one token after the other, from the definitions:

* route: score s = softmax(l) or 1 / (1 + exp(-l)); choice c = s + bias, or l
  without a bias; the groups of greatest merit stay, then the top_k largest
  choices, equal values by the lowest index; weight = s of the chosen, over
  their sum if renormalised, times a factor;
* group_rows: a stable sort of entries by group, ungrouped ones last;
* dispatch_rows, combine_rows: rows copied to their places and summed back;
* lora: y = base + scale * B (A x) with each token's own adapter.
"""
from __future__ import annotations

import numpy as np

__all__ = ["route", "group_rows", "dispatch_rows", "combine_rows", "lora", "lora_error_bound"]

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def _clean(logits: np.ndarray, largest: float) -> np.ndarray:
    """NaN counts as -inf (no candidate), +inf as the type's largest finite value."""
    v = np.asarray(logits, dtype=np.float64).copy()
    v[np.isnan(v)] = -np.inf
    return np.minimum(v, largest)


def _scores(l: np.ndarray, score: int) -> np.ndarray:
    s = np.zeros(l.shape)
    live = l > -np.inf
    if not live.any():
        return s
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    else:
        e = np.exp(l[live] - l[live].max())
        s[live] = e / e.sum()
    return s


def _order(values) -> list[int]:
    """Indices by descending value, equal values by the lowest index."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))


def route(logits, top_k, score=SOFTMAX, bias=None, groups=1, top_groups=1, group_score=GROUP_MAX, renormalise=True,
          scale=1.0, largest=float(np.finfo(np.float32).max)):
    """(experts [tokens, top_k] int32, weights [tokens, top_k] float64)."""
    logits = _clean(logits, largest)
    tokens, n = logits.shape
    experts = np.full((tokens, top_k), -1, dtype=np.int32)
    weights = np.zeros((tokens, top_k))
    per = n // groups
    for t in range(tokens):
        l = logits[t]
        s = _scores(l, score)
        valued = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        valued = np.where((l > -np.inf) & ~np.isnan(valued), valued, -np.inf)
        choice = l if bias is None else valued
        allowed = list(range(n))
        if groups > 1:
            merit = []
            for g in range(groups):
                if group_score == GROUP_TOP2:
                    two = sorted(valued[g * per:(g + 1) * per], reverse=True)[:2]
                    merit.append(two[0] + (two[1] if len(two) > 1 and two[1] > -np.inf else 0.0))
                else:
                    merit.append(choice[g * per:(g + 1) * per].max())
            kept = _order(merit)[:top_groups]
            allowed = [e for e in range(n) if e // per in kept]
        chosen = [allowed[i] for i in _order([choice[e] for e in allowed])]
        chosen = [e for e in chosen if choice[e] > -np.inf][:top_k]
        w = s[chosen]
        if renormalise and w.sum() > 0:
            w = w / w.sum()
        experts[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    return experts, weights


def group_rows(index, groups):
    """(offsets [groups + 1], order [n], slot (index's shape))."""
    flat = np.asarray(index).reshape(-1)
    lists = [[] for _ in range(groups + 1)]
    for i, g in enumerate(flat):
        lists[g if 0 <= g < groups else groups].append(i)
    offsets = np.cumsum([0] + [len(v) for v in lists[:groups]]).astype(np.int32)
    order = np.array([i for v in lists for i in v], dtype=np.int32)
    slot = np.full(flat.shape, -1, dtype=np.int32)
    for at, i in enumerate(order[:offsets[groups]]):
        slot[i] = at
    return offsets, order, slot.reshape(np.shape(index))


def dispatch_rows(x, slot, xs):
    """A copy of xs with x's rows at their slots."""
    out = np.array(xs)
    for t in range(slot.shape[0]):
        for at in slot[t]:
            if 0 <= at < out.shape[0]:
                out[at] = x[t]
    return out


def combine_rows(ys, slot, weights, base=None):
    """(y, the sum of the magnitudes of its terms), float64."""
    tokens, top_k = slot.shape
    y = np.zeros((tokens, ys.shape[1])) if base is None else base.astype(np.float64)
    size = np.abs(y)
    for t in range(tokens):
        for j in range(top_k):
            if 0 <= slot[t, j] < ys.shape[0]:
                term = float(weights[t, j]) * ys[slot[t, j]].astype(np.float64)
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def lora(x, index, adapters, base):
    """adapters: {slot: (A, B, scale)} of float64 arrays; tokens whose index is not
    among them keep their base."""
    y = np.array(base, dtype=np.float64)
    for t, i in enumerate(index):
        if int(i) in adapters:
            a, b, scale = adapters[int(i)]
            y[t] += scale * (b @ (a @ x[t].astype(np.float64)))
    return y


def lora_error_bound(x, index, adapters, base):
    """How far a float32 evaluation may be off, per element.  With u = 2^-23 (a
    matrix instruction may cut where others round) a sum of m terms is off by at
    most m u times the sum of their magnitudes: v = A x by (cols + 16) u |A||x|
    (up to 16 parts are added up), scale * v by u more, and y, whose terms are
    the base and three exact parts of every rank's product, by (3 rank + 2) u
    (|base| + 3 |scale||B||v|)."""
    u = 2.0 ** -23
    out = np.abs(np.asarray(base, dtype=np.float64)) * u
    for t, i in enumerate(index):
        if int(i) in adapters:
            a, b, scale = adapters[int(i)]
            xt, ab, bb = np.abs(x[t].astype(np.float64)), np.abs(a), abs(scale) * np.abs(b)
            dv = (len(xt) + 16 + 1) * u * (ab @ xt)
            v = np.abs(a @ x[t].astype(np.float64)) + dv
            out[t] = bb @ dv + (3 * len(a) + 2) * u * (np.abs(base[t]) + 3 * (bb @ v))
    return out
