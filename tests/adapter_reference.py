"""Plain 64-bit implementations of the low-rank adapters, of the routing to experts and of an expert layer from a given routing, from their definitions.

Nothing here calls the library.  Limits are counted from these roundings:

  * a BF16 rounding is within 2^-8 of its value (half a unit of the last of 8 bits), an fp32 one within 2^-24;
  * an fp32 sum of n exact products is within n 2^-23 of the sum of their magnitudes (n roundings of at most
    2^-24 each, doubled for adders that cut off);
  * an fp32 value as the sum of two BF16 values is within 2^-8 2^-8 = 2^-16 of itself (the first is off by at
    most 2^-8 of it, the second by 2^-8 of that).
"""
from __future__ import annotations

import math

import numpy as np

PARTS = 64  # more additions than the sum over K can be split into parts


def lora(x, a, b, scales, ids, base):
    """float64: (y [m, N], limit).  x [m, K], a [num, R, K], b [num, N, R], scales [num], ids [m] (-1: none), base [m, N] or None."""
    m, K = x.shape
    num, N, R = b.shape
    y = np.zeros((m, N)) if base is None else base.copy()
    err = np.zeros((m, N))
    rounded = np.zeros(m, bool)
    for t in range(m):
        e = ids[t]
        if e == -1:
            continue
        if not 0 <= e < num:
            y[t] = np.nan
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            u, mag = a[e] @ x[t], np.abs(a[e]) @ np.abs(x[t])
            du = (K + PARTS) * 2.0 ** -23 * mag  # the sum over K, by parts
            du = (np.abs(u) + du) * (2.0 ** -16 + 2.0 ** -24) + du  # scaled (one fp32 rounding), as two BF16 values
            delta = scales[e] * (b[e] @ u)
            size = np.abs(scales[e]) * (np.abs(b[e]) @ (np.abs(u) + du))
            y[t] += delta
            err[t] = np.abs(scales[e]) * (np.abs(b[e]) @ du) + (2 * R + 1) * 2.0 ** -23 * size + 2.0 ** -24 * (np.abs(y[t]) + size)
        rounded[t] = True
    return y, np.where(rounded[:, None], err + 2.0 ** -8 * (np.abs(y) + err), 0.0)  # rows without an adapter: exact


def route(logits, topk, scoring="softmax", bias=None, groups=1, topk_groups=None, group_score="top2", renormalize=True, scale=1.0):
    """float64 logits [T, E] -> ids [T, topk] (-1: none), weights float64."""
    T, E = logits.shape
    topk_groups = groups if topk_groups is None else topk_groups
    size = E // groups
    ids, weights = np.full((T, topk), -1), np.zeros((T, topk))
    direct = bias is None
    for t in range(T):
        l = logits[t]
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        free = [e for e in range(E) if l[e] > -np.inf]
        odd = np.isnan(l).any() or (scoring == "softmax" and (l == np.inf).any())
        if not odd:
            if scoring == "softmax":
                top = max((l[e] for e in free), default=0.0)
                total = math.fsum(math.exp(l[e] - top) for e in free)
                s = {e: math.exp(l[e] - top) / total for e in free}
            else:
                s = {e: 1.0 / (1.0 + math.exp(-l[e])) if l[e] > -700 else 0.0 for e in free}
            odd = bool(np.isnan(b).any())
        if odd:
            weights[t] = np.nan
            continue
        c = {e: l[e] if direct else s[e] + b[e] for e in free}
        two = {e: s[e] + b[e] for e in free}
        free = [e for e in free if c[e] > -np.inf]
        if groups > 1:
            of = {}
            for g in range(groups):
                best = sorted(((two if group_score == "top2" else c)[e] for e in free if e // size == g), reverse=True)[:2]
                if best:
                    of[g] = sum(best) if group_score == "top2" else best[0]
            stay = sorted((g for g in of if of[g] > -np.inf), key=lambda g: (-of[g], g))[:topk_groups]
            free = [e for e in free if e // size in stay]
        best = sorted(free, key=lambda e: (-c[e], e))[:topk]
        w = [s[e] for e in best]
        if renormalize:
            total = math.fsum(w)
            w = [v / total if total > 0 else 0.0 for v in w]
        ids[t, :len(best)] = best
        weights[t, :len(best)] = [scale * v for v in w]
    return ids, weights


def experts(x, gate, up, down, mags, ids, weights, resid=None):
    """The expert layer from a given routing in float64: (y, limit).  gate, up [E, I, H], down [E, H, I]; mags: the
    magnitudes behind their sums.  silu's exp and reciprocal are within 2^-18 of their values."""
    T, H = x.shape
    E, I = gate.shape[:2]
    y = np.zeros((T, H)) if resid is None else resid.copy()
    err = np.zeros((T, H))
    for t in range(T):
        if np.isnan(weights[t]).any():
            y[t] = np.nan
            continue
        for e in range(E):
            w = float(np.where(ids[t] == e, weights[t], 0.0).sum())
            if w == 0:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            dg, du = H * 2.0 ** -23 * (mags[0][e] @ np.abs(x[t])), H * 2.0 ** -23 * (mags[1][e] @ np.abs(x[t]))
            s = g / (1 + np.exp(-g))
            h = w * s * u
            dw = 2.0 ** -24 * np.abs(weights[t][ids[t] == e]).sum() * ids.shape[1]  # weights of one expert, added in fp32
            dh = (abs(w) + dw) * (1.1 * dg * (np.abs(u) + du) + np.abs(s) * du) + (2.0 ** -8 + 2.0 ** -16) * np.abs(h) + dw * np.abs(s * u)
            y[t] += down[e] @ h
            err[t] += np.abs(down[e]) @ dh + I * 2.0 ** -23 * (mags[2][e] @ (np.abs(h) + dh))
    return y, err + (ids.shape[1] + 2) * 2.0 ** -23 * np.abs(y) + 2.0 ** -8 * (np.abs(y) + err)
