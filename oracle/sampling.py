"""Sampling under a request's parameters, and the acceptance walk with the target distribution so filtered (fp64).

The pages sample from the target's softmax as it is ("EAGLE" notes, EAGLE-2 "Well-Calibrated Draft Model"); what a
serving request adds to that is the usual four parameters, read here in this order:
  * temperature T: weights exp((x - max) / T); T <= 0 (or NaN): all weight on the argmax (lowest id);
  * top-k: the k tokens first in the order (logit descending, id ascending); k <= 0 or k >= V: off;
  * top-p: of those, the fewest first ones whose weights sum to at least p times theirs all (at least one);
    p >= 1 or NaN: off;
  * min-p: of those, the ones whose weight is at least min_p of the largest; <= 0 or NaN: off, > 1: as 1.
The draw is the inverse CDF in id order: the smallest id whose cumulative kept weight exceeds u times the total.
A weight below 2^-45 counts as 0.  NaN logits count as -inf; where some are +inf those alone weigh, equally.

The walk is accept_stochastic's with p = the kept weights, normalised; q stays the draft row's softmax.
"""
from __future__ import annotations

import math
from typing import Dict, List

import numpy as np

from .common import softmax

TINY = 2.0 ** -45
TIE = 1e-8  # relative distance from a border within which a decision is decided by rounding


def filter_row(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row -> (z = (x - max) / T, kept weights, near): near flags a top-p border within TIE of a sum."""
    x = np.asarray(x, dtype=np.float64).copy()
    V = x.shape[0]
    x[np.isnan(x)] = -np.inf
    if np.isposinf(x).any():
        x = np.where(np.isposinf(x), 0.0, -np.inf)
    z = np.full(V, -np.inf)
    alive = np.flatnonzero(x > -np.inf)
    if alive.size == 0:
        return z, np.zeros(V), False
    if not temperature > 0:
        z[int(np.argmax(x))] = 0.0
        return z, np.exp(z), False
    z[alive] = (x[alive] - x.max()) / float(temperature)
    e = np.exp(z)
    e[e < TINY] = 0.0
    order = sorted(range(V), key=lambda i: (-x[i], i))
    chosen = order[:top_k] if 0 < top_k < V else order
    near = False
    if top_p < 1:
        total = math.fsum(e[i] for i in chosen)
        run, count = 0.0, 0
        for i in chosen:
            run += e[i]
            count += 1
            near = near or (0 < top_p and abs(run - top_p * total) <= TIE * total and e[i] > 0)
            if run >= top_p * total or top_p <= 0:
                break
        chosen = chosen[:count]
    kept = np.zeros(V)
    kept[chosen] = e[chosen]
    if min_p > 0:
        kept[e < min(float(min_p), 1.0)] = 0.0
        near = near or bool((np.abs(e[chosen] - min(float(min_p), 1.0)) <= TIE * min_p).any() and min_p < 1)
    return z, kept, near


def draw(weights, u):
    """(smallest id whose cumulative weight exceeds u * total, near): -1 without any weight."""
    u = 0.0 if not u >= 0 else min(float(u), 1.0 - 2.0 ** -24)
    c = np.cumsum(np.asarray(weights, dtype=np.float64))
    if not c[-1] > 0:
        return -1, False
    i = int(np.searchsorted(c, u * c[-1], side="right"))
    lo = c[i - 1] if i > 0 else 0.0
    near = (u > 0 and abs(u * c[-1] - lo) <= TIE * c[-1]) or abs(c[i] - u * c[-1]) <= TIE * c[-1]
    return i, bool(near)


def sample_row(x, u, **params):
    """(token, log-probability among the kept tokens, near)."""
    z, w, near = filter_row(x, **params)
    tok, tie = draw(w, u)
    if tok < 0:
        return -1, -math.inf, False
    return tok, float(z[tok] - math.log(math.fsum(w))), near or tie


def accept_sampling(target, draft, tokens, parents, draft_row, uniforms, max_depth, without_replacement=False,
                    **params) -> Dict:
    """One sequence's walk -> accepted_len, path, bonus, near (some decision lay on a border)."""
    target, draft = np.asarray(target, dtype=np.float64), np.asarray(draft, dtype=np.float64)
    path: List[int] = []
    node, near = 0, False
    while True:
        _, w, tie = filter_row(target[node], **params)
        near |= tie
        if not w.sum() > 0:
            return {"accepted_len": len(path), "path": path + [-1] * (max_depth - len(path)), "bonus": -1, "near": near}
        p = w / w.sum()
        kids = [c + 1 for c in range(len(parents)) if int(parents[c]) == node] if len(path) < max_depth else []
        r = int(draft_row[node])
        if not 0 <= r < draft.shape[0]:
            kids = []
        q = softmax(draft[r]) if kids else None
        moved, spent = 0, False
        for c in kids:
            x = int(tokens[c - 1])
            px, qx = (p[x], q[x]) if 0 <= x < p.shape[0] else (0.0, 0.0)
            u = float(uniforms[0][c])
            near |= abs(u * qx - px) <= TIE * max(px, qx) and px > 0
            if qx > 0 and u * qx < px:
                moved = c
                break
            left = np.maximum(p - q, 0.0)
            if not left.sum() > 0:
                spent = True
                break
            p = left / left.sum()
            if without_replacement:
                q = q.copy()
                if 0 <= x < q.shape[0]:
                    q[x] = 0.0
                if not q.sum() > 0:
                    spent = True
                    break
                q /= q.sum()
        if moved:
            path.append(moved)
            node = moved
            continue
        if spent:
            t = target[node].copy()
            t[np.isnan(t)] = -np.inf
            bonus = int(np.argmax(t))
        else:
            bonus, tie = draw(p, uniforms[1][node])
            near |= tie
        return {"accepted_len": len(path), "path": path + [-1] * (max_depth - len(path)), "bonus": bonus, "near": near}
