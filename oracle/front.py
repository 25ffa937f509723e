"""Operators in front of the projections in float64 (TEST INFRASTRUCTURE ONLY -- never imported by the product path).

Definitions (include/fp8q_front.h):
    * norm: h = x (+ residual), rstd = (mean h^2 + eps)^(-1/2), y = h rstd weight, and its gradient;
    * route: the k largest logits of a row (the lower index first where equal), softmax weights, counts, balance loss
      E sum_e f_e P_e and its slope by p; and the gradient with respect to the logits, the counts held constant;
    * dispatch: rows in the order of their experts, each expert's padded to whole tiles of 128.
"""

import numpy as np


def rstd(h, eps):
    h = np.asarray(h, np.float64)
    return 1.0 / np.sqrt((h * h).mean(axis=1) + eps)


def norm(h, weight, eps):
    """y in float64."""
    h = np.asarray(h, np.float64)
    return h * rstd(h, eps)[:, None] * np.asarray(weight, np.float64)[None, :]


def norm_backward(dy, h, weight, r, dh=None):
    """(dx, dw) in float64 from the given 1 / rms."""
    dy, h, r = (np.asarray(v, np.float64) for v in (dy, h, r))
    xhat = h * r[:, None]
    g = dy * np.asarray(weight, np.float64)[None, :]
    dx = r[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return (dx if dh is None else dx + np.asarray(dh, np.float64)), (dy * xhat).sum(axis=0)


def softmax(z):
    """Rows of softmax; zeros for a row of minus infinities."""
    z = np.asarray(z, np.float64)
    m = z.max(axis=1, keepdims=True)
    x = np.exp(z - np.where(np.isfinite(m), m, 0.0))
    s = x.sum(axis=1, keepdims=True)
    return np.divide(x, s, out=np.zeros_like(x), where=s > 0)


def route(z, k, valid=None, renormalize=False):
    """(weights, experts, counts, loss, slope); token by token and expert by expert."""
    z = np.asarray(z, np.float64)
    t, e = z.shape
    weights, experts = np.zeros((t, k)), np.full((t, k), -1, np.int32)
    counts, mass, n = np.zeros(e, np.int64), np.zeros(e), 0
    for i in range(t):
        if valid is not None and not valid[i]:
            continue
        if not np.isfinite(z[i]).any():
            continue
        n += 1
        p = softmax(z[i:i + 1])[0]
        mass += p
        order = [c for c in sorted(range(e), key=lambda c: (-z[i, c], c)) if np.isfinite(z[i, c])][:k]
        total = p[order].sum() if renormalize else 1.0
        for j, c in enumerate(order):
            weights[i, j], experts[i, j] = p[c] / total, c
            counts[c] += 1
    slope = e * counts / (k * float(n) ** 2) if n else np.zeros(e)
    return weights, experts, counts, float((slope * mass).sum()), slope


def route_value(z, experts, slope, dweights, dloss, renormalize):
    """What moe_route_backward differentiates: sum dweights weights + dloss loss, with choice and counts held."""
    p = softmax(z)
    total = 0.0
    for i in range(p.shape[0]):
        if experts[i, 0] < 0:
            continue
        total += dloss * float((p[i] * slope).sum())
        live = [j for j in range(experts.shape[1]) if 0 <= experts[i, j] < p.shape[1]]
        w = np.array([p[i, experts[i, j]] for j in live])
        if renormalize:
            w = w / w.sum()
        total += float((w * dweights[i, live]).sum())
    return total


def route_backward(z, experts, slope, dweights, dloss, renormalize):
    p = softmax(z)
    dz = np.zeros_like(p)
    for i in range(p.shape[0]):
        if experts[i, 0] < 0:
            continue
        dp = dloss * np.asarray(slope, np.float64)
        live = [j for j in range(experts.shape[1]) if 0 <= experts[i, j] < p.shape[1]]
        dc = np.asarray(dweights, np.float64)[i, live]
        chosen = p[i, experts[i, live]]
        if renormalize:
            s = chosen.sum()
            dc = (dc - (dc * chosen).sum() / s) / s
        for j, d in zip(live, dc):
            dp[experts[i, j]] += d
        dz[i] = p[i] * (dp - (p[i] * dp).sum())
    return dz


def dispatch(experts, num_experts, rows):
    """(group_of_mtile, row_of_slot, token_of_row) by counting, slot by slot."""
    t, k = experts.shape
    counts = [int((experts == e).sum()) for e in range(num_experts)]
    start, at = [], 0
    group = np.full(rows // 128, -1, np.int32)
    for e, c in enumerate(counts):
        start.append(at)
        group[at // 128:at // 128 + -(-c // 128)] = e
        at += -(-c // 128) * 128
    row_of_slot, token_of_row, seen = np.full((t, k), -1, np.int32), np.full(rows, -1, np.int32), [0] * num_experts
    for i in range(t):
        for j in range(k):
            e = int(experts[i, j])
            if 0 <= e < num_experts:
                row = start[e] + seen[e]
                seen[e] += 1
                row_of_slot[i, j], token_of_row[row] = row, i
    return group, row_of_slot, token_of_row
