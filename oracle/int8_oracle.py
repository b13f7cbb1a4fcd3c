"""Plain statement of the 8-bit integer operators and of routing to experts, in NumPy and 64 bits.

Shares no code with the kernels.  A row y is held as codes q in -127 .. 127 and a
scale a / 127, a = max|y|, q the integer nearest to 127 y / a with ties to the even one.
"""
from __future__ import annotations

import numpy as np


def fold(x, act_scale, multiply):
    """The values that are quantized: x, x s or x / s rounded to fp32 (x, s: fp32 values)."""
    x = np.asarray(x, dtype=np.float64)
    if act_scale is None:
        return x
    s = np.asarray(act_scale, dtype=np.float64)
    with np.errstate(all="ignore"):  # 53 bits, then 24: the quotient of two 24-bit numbers is rounded as once
        return (x * s if multiply else x / s).astype(np.float32).astype(np.float64)


def quantize(x, act_scale=None, multiply=False):
    """x [M, K] -> (codes int8 [M, K], scales float64 [M]).  127 y and the quotient's distance from a
    tie are exact enough in 64 bits: 31-bit numerators over 24-bit denominators."""
    y = fold(x, act_scale, multiply)
    codes = np.zeros(y.shape, dtype=np.int8)
    scales = np.zeros(y.shape[0])
    for m, row in enumerate(y):
        if not np.all(np.isfinite(row)):
            scales[m] = np.nan
            continue
        a = np.abs(row).max()
        if a > 0:
            scales[m] = a / 127.0
            codes[m] = np.rint(127.0 * row / a)
    return codes, scales


def gemm(a, sa, w, sw, bias=None):
    """(sum a w) sa sw + bias in 64 bits; the sum of products is exact."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    y = acc * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def scores(x, scoring):
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        out = np.empty_like(x)
        for t, row in enumerate(x):
            top = max((v for v in row if not np.isnan(v)), default=0.0)
            e = np.exp(row - (0.0 if top == -np.inf else top))
            total = sum(e)
            out[t] = e * 0.0 if total == 0 else e / total
        return out


def _rank(keys):
    """Indices by descending key, the lower first among equals, NaN last."""
    return sorted(range(len(keys)), key=lambda i: (1, 0.0, i) if np.isnan(keys[i]) else (0, -keys[i], i))


def _weights(x, s, ids, scoring, renormalize, scale):
    """The weights of the chosen experts of one token."""
    if not renormalize:
        return [scale * s[i] for i in ids]
    with np.errstate(all="ignore"):
        if scoring == "softmax":
            chosen = [x[i] for i in ids]
            top = max((v for v in chosen if not np.isnan(v)), default=0.0)
            v = [np.exp(c - (0.0 if top == -np.inf else top)) for c in chosen]
        else:
            v = [s[i] for i in ids]
        total = sum(v)
        return [0.0 if total == 0 else scale * c / total for c in v]


def route(x, top_k, scoring="softmax", bias=None, groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0):
    """x [T, E] -> (experts int32 [T, top_k], weights float64 [T, top_k])."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    s, per = scores(x, scoring), E // groups
    experts, weights = np.zeros((T, top_k), np.int32), np.zeros((T, top_k))
    for t in range(T):
        if bias is None:
            key = x[t]
        else:
            key = np.where(x[t] == -np.inf, -np.inf, s[t] + np.asarray(bias, np.float64))
        by = key if bias is not None or group_top == 1 else np.where(x[t] == -np.inf, -np.inf, s[t])
        if groups > 1:
            rank = []
            for g in range(groups):
                part = by[g * per:(g + 1) * per]
                best = [part[i] for i in _rank(part)[:group_top]]
                with np.errstate(all="ignore"):
                    rank.append(sum(best[1:], best[0]))
            kept = set(_rank(rank)[:top_groups or groups])
        else:
            kept = {0}
        ids = [i for i in _rank(key) if i // per in kept][:top_k]
        experts[t] = ids
        weights[t] = _weights(x[t], s[t], ids, scoring, renormalize, scale)
    return experts, weights


def route_backward(x, experts, dweights, scoring="softmax", renormalize=True, scale=1.0):
    """dlogits [T, E]: the chain rule through w_c = scale s_c (/ sum of the chosen s)."""
    x, d = np.asarray(x, np.float64), np.asarray(dweights, np.float64)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        ids = [(c, e) for c, e in enumerate(experts[t]) if 0 <= e < x.shape[1]]
        s = scores(x[t:t + 1], scoring)[0]
        rest = scores(-x[t:t + 1], scoring)[0] if scoring == "sigmoid" else np.ones_like(s)  # 1 - s, which would cancel next to 1
        # dw_c - sum p dw as sum p_j (dw_c - dw_j) (the p add up to 1): next to a weight of nearly 1 the former would cancel
        if renormalize:  # by total, with s the weight, times ds / s
            w = _weights(x[t], s, [e for _, e in ids], scoring, True, 1.0)
            for wc, (c, e) in zip(w, ids):
                out[t, e] += scale * wc * sum(wj * (d[t, c] - d[t, j]) for wj, (j, _) in zip(w, ids)) * rest[e]
            continue
        dense = np.zeros_like(s)
        for c, e in ids:
            dense[e] += scale * d[t, c]
        out[t] = s * ((dense[:, None] - dense) @ s) if scoring == "softmax" else dense * s * rest
    return out


def moe(x, experts, weights, up, up_scales, down, down_scales, slack=0.0):
    """(y [T, H], reach [T, H], parts [T, H]): the layer's result; by how much it moves if every code of h within
    `slack` of a tie goes to its other neighbour; and the sum of the magnitudes of what is added up."""
    q, a = quantize(x)
    T, H = q.shape
    E, I2, _ = up.shape
    I = I2 // 2
    y, reach, parts = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for c, e in enumerate(experts[t]):
            if not 0 <= e < E:
                continue
            gu = (up[e].astype(np.float64) @ q[t].astype(np.float64)) * a[t] * np.asarray(up_scales[e], np.float64)
            with np.errstate(over="ignore"):
                h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            top = np.abs(h).max()
            u = 127.0 * h / top if top > 0 else h
            code, step = np.rint(u), top / 127.0
            near = np.abs(np.abs(u - np.trunc(u)) - 0.5) < slack
            d = down[e].astype(np.float64) * np.asarray(down_scales[e], np.float64)[:, None]
            w = float(weights[t, c])
            y[t] += w * step * (d @ code)
            reach[t] += abs(w) * step * (np.abs(d) @ near.astype(np.float64))
            parts[t] += abs(w) * step * (np.abs(d) @ np.abs(code))
    return y, reach, parts
