"""Plain 64-bit forms of routing, its gradient, the gradient of combine and the
experts' 4-bit products, one token (or row) at a time, for the tests to compare
with.  numpy only; nothing here is shared with the library."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scores(l, sigmoid):
    """Scores of one token's logits (fp64, NaN already -inf)."""
    with np.errstate(over="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
    top = l.max()
    if top == -math.inf:
        return np.zeros_like(l)
    e = np.where(l == math.inf, 1.0, 0.0) if top == math.inf else np.exp(l - top)
    return e / e.sum()


def chosen_shares(l, sigmoid):
    """Scores of the chosen logits over their sum, without underflow."""
    if not len(l):
        return l
    if not sigmoid:
        return scores(l, False)
    low = min(0.0, l.max())
    with np.errstate(over="ignore"):
        a = np.exp(np.minimum(l, 0.0) - low) / (1.0 + np.exp(-np.abs(l)))
    return a / a.sum()


def route(logits, k, sigmoid, bias, groups, topk_groups, group_top, renorm, scale):
    logits = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    T, E = logits.shape
    idx, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    size = E // groups
    for t in range(T):
        l = logits[t]
        s = scores(l, sigmoid)
        if bias is not None or (groups > 1 and group_top == 2):
            c = s.astype(np.float32)
            if bias is not None:
                c = c + bias.astype(np.float32)
            c = c.astype(np.float64)
        else:
            c = l.copy()
        c[(l == -np.inf) | np.isnan(c)] = -np.inf
        if groups > 1:
            best = []
            for g in range(groups):
                v = sorted((x for x in c[g * size:(g + 1) * size] if x > -math.inf), reverse=True)[:group_top]
                best.append(float(np.sum(np.array(v, np.float32), dtype=np.float32)) if v else -math.inf)
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
            for g in range(groups):
                if g not in kept:
                    c[g * size:(g + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -math.inf][:k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = scale * (chosen_shares(l[order], sigmoid) if renorm else s[order])
    return idx, w


def route_backward(logits, idx, g, sigmoid, renorm, scale):
    """(gradient, size): size[t, e] is the sum of the magnitudes of the terms
    that make up element [t, e], for an error bound."""
    logits = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    d, size = np.zeros_like(logits), np.zeros_like(logits)
    for t in range(len(logits)):
        l = logits[t]
        slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < len(l) and l[idx[t, j]] > -math.inf]
        if not slots:
            continue
        e, gt, s = idx[t, slots], g[t, slots].astype(np.float64), scores(l, sigmoid)
        if renorm:
            p = chosen_shares(l[e], sigmoid)
            with np.errstate(over="ignore"):
                more = 1.0 / (1.0 + np.exp(l[e])) if sigmoid else 1.0
            np.add.at(d[t], e, scale * p * (gt - (gt * p).sum()) * more)
            np.add.at(size[t], e, abs(scale) * p * (np.abs(gt) + (np.abs(gt) * p).sum()) * more)
        elif sigmoid:
            with np.errstate(over="ignore"):
                v = scale * s[e] / (1.0 + np.exp(l[e]))
            np.add.at(d[t], e, gt * v)
            np.add.at(size[t], e, np.abs(gt * v))
        else:
            here, many = np.zeros_like(l), np.zeros_like(l)
            np.add.at(here, e, gt)
            np.add.at(many, e, np.abs(gt))
            d[t] = scale * s * (here - (gt * s[e]).sum())
            size[t] = abs(scale) * s * (many + (np.abs(gt) * s[e]).sum())
    return d, size


def combine_backward(g, y, row, w):
    """(dy with NaN where no slot maps, dw, sum of |products| of dw)."""
    T, k = row.shape
    dy = np.full(y.shape, np.nan)
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row[t, j]
            if 0 <= r < len(y):
                dy[r] = (1.0 if w is None else float(w[t, j])) * g[t]
                dw[t, j] = (g[t] * y[r]).sum()
                size[t, j] = np.abs(g[t] * y[r]).sum()
    return dy, dw, size


def decode_w4(codes, scales):
    """[..., W, K/2] codes and [..., W, K/32] scales to [..., W, K] values."""
    both = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(both & 8, -1.0, 1.0) * E2M1[both & 7]
    f = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def expert_linear(x, spans, weights, silu):
    """x [rows, K] fp64, spans [(first, count)] per expert, weights [E, W, K]
    fp64: (y with NaN where no expert has the row, error scale)."""
    N = weights.shape[1] // (2 if silu else 1)
    y, size = np.full((len(x), N), np.nan), np.zeros((len(x), N))
    for (first, count), w in zip(spans, weights):
        v = x[first:first + count] @ w.T
        a = np.abs(x[first:first + count]) @ np.abs(w).T
        if silu:
            gate, up = v[:, :N], v[:, N:]
            s = gate / (1.0 + np.exp(-gate))
            y[first:first + count] = s * up
            # |silu'| <= 1.1: the error of gate times |up|, that of up times |silu|.
            size[first:first + count] = 1.1 * a[:, :N] * np.abs(up) + np.abs(s) * a[:, N:]
        else:
            y[first:first + count], size[first:first + count] = v, a
    return y, size
