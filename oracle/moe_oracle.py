"""Plain 64-bit statements of the experts' operators (numpy, no product code).

A router's row l of logits over E experts: scores s = softmax(l) or
1 / (1 + exp(-l)), values v = s + bias (the logits themselves without a bias),
groups ranked by the sum of their one or two largest values, the largest v of
the best groups chosen in descending order, equal ones by index; weights s or
s / (sum of the chosen s), times a factor. -inf closes an expert. Choices are
numbered token * top_k + slot and sorted by expert, in their own order.
"""
import numpy as np

from . import block_oracle as bo

U24 = 2.0 ** -24


def route(logits, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0):
    """(experts, weights), one token and one choice at a time."""
    L = np.asarray(logits, np.float64)
    T, E = L.shape
    experts, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    b = None if bias is None else np.asarray(bias, np.float64)
    for t in range(T):
        l = L[t]
        if np.isnan(l).any() or (score == "softmax" and np.isposinf(l).any()) or (b is not None and np.isnan(b).any()):
            experts[t], weights[t] = np.arange(top_k), np.nan
            continue
        closed = np.isneginf(l)
        with np.errstate(over="ignore"):
            if closed.all():
                s = np.zeros(E)
            elif score == "softmax":
                s = np.exp(l - l.max())
                s = s / s.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-l))
        v = l.copy() if b is None else np.where(closed, -np.inf, s + b)
        closed |= np.isneginf(v)
        if n_groups > 1:
            per = E // n_groups
            value = []
            for g in range(n_groups):
                of = s if b is None and group_top == 2 else v
                w = sorted((of[i] for i in range(g * per, (g + 1) * per) if not closed[i]), reverse=True)[:group_top]
                value.append(sum(w) if w else -np.inf)
            best = sorted(range(n_groups), key=lambda g: (-value[g], g))[:top_groups]
            for g in range(n_groups):
                if g not in best:
                    closed[g * per:(g + 1) * per] = True
        order = sorted((i for i in range(E) if not closed[i]), key=lambda i: (-v[i], i))[:top_k]
        experts[t, :len(order)] = order
        weights[t, :len(order)] = s[order]
        if renormalise and order and l[order].max() < -600:  # scores beyond 64 bits: exp(l) (1 + exp(l)) ^ -1 = exp(l) there
            weights[t, :len(order)] = np.exp(l[order] - l[order].max())
        if renormalise:
            total = weights[t].sum()
            weights[t] = weights[t] / total if total > 0 else 0.0
        weights[t] *= scale
    return experts, weights


def plan(experts, E):
    """(order, place, offsets) of the choices."""
    e = np.asarray(experts).reshape(-1)
    lists = [[c for c in range(e.size) if e[c] == x] for x in range(E)]
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    order, place = np.full(e.size, -1, np.int32), np.full(e.size, -1, np.int32)
    for i, c in enumerate(c for x in lists for c in x):
        order[i], place[c] = c, i
    return order, place, offsets


def linear_error(mag, K):
    """What fp32 sums of an e4m3 linear may be off by: a rounding of up to a
    whole step for every product and block, the scale products and the bias."""
    return 2 * (bo.BLOCK + bo.n_blocks(K) + 4) * U24 * mag


def expert_linear(Qx, sx, rows, offsets, q, s, bias=None):
    """(Y, magnitudes) for the activation rows `rows` in plan order; zero rows behind the last."""
    E, N = q.shape[:2]
    Y, A = np.zeros((len(rows), N)), np.zeros((len(rows), N))
    for e in range(E):
        i = slice(offsets[e], offsets[e + 1])
        if i.start < i.stop:
            Y[i], A[i] = bo.fp8_linear(Qx[rows[i]], sx[rows[i]], q[e], s[e], None if bias is None else bias[e])
    return Y, A


def swiglu(g, u, dg, du):
    """(silu(g) u, what it may be off by): dg, du are the errors of g and u;
    silu's slope is within 1.1, its own fp32 arithmetic within a few steps and
    the rounding of the exponent, |g| 2^-24 relative."""
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    return silu * u, 1.1 * np.abs(u) * dg + np.abs(silu) * du + 1.1 * dg * du + np.abs(silu * u) * U24 * (8 + 2 * np.abs(g))


def hidden_slack(h, dh):
    """(codes, scales, slack) of h: slack is what the value of a code may be off
    by, where h is only known to dh. A code may be another where the quotient is
    within its error of a rounding border; the scale has its own error."""
    Q, s = bo.fp8_pack(h.astype(np.float32))
    S = bo.widen(s, *h.shape)
    top = np.concatenate([np.repeat(dh[:, j:j + bo.BLOCK].max(1, keepdims=True), min(bo.BLOCK, h.shape[1] - j), 1)
                          for j in range(0, h.shape[1], bo.BLOCK)], 1) / bo.MAX + S * 2 * U24
    with np.errstate(all="ignore"):
        z = np.where(S > 0, np.abs(h) / S, 0.0)
        dz = np.where(S > 0, (dh + z * top) / S + z * 2 * U24, 0.0)
    grid = bo.e4m3_values()[:127]
    borders = (grid[1:] + grid[:-1]) / 2
    k = np.clip(np.searchsorted(borders, z), 0, len(borders) - 1)
    step = np.exp2(np.floor(np.log2(np.maximum(z + dz, 2.0 ** -6))) - 3.0)
    near = np.minimum(np.abs(z - borders[k]), np.abs(z - borders[np.maximum(k - 1, 0)])) <= dz
    value = np.abs(bo.e4m3_values()[Q])
    return Q, s, np.where(near, step * S, 0.0) + value * top


def combine(rows, place, weights, residual=None):
    """(Y, magnitudes)."""
    T, k = weights.shape
    Y = np.zeros((T, rows.shape[1])) if residual is None else np.array(residual, np.float64)
    A = np.abs(Y)
    for t in range(T):
        for j in range(k):
            p = place.reshape(T, k)[t, j]
            if p >= 0:
                Y[t] += float(weights[t, j]) * rows[p]
                A[t] += abs(float(weights[t, j])) * np.abs(rows[p])
    return Y, A


def moe(X, experts, weights, gate, up, down, residual=None, rows_error=0.0):
    """(Y, what fp32 arithmetic and the codes it may choose can move it by);
    rows_error: the relative rounding of the rows that are summed up."""
    T, k = experts.shape
    Qx, sx = bo.fp8_pack(np.asarray(X, np.float32))
    E = gate[0].shape[0]
    order, place, offsets = plan(experts, E)
    order = order[:offsets[E]]
    rows = order // k
    K, inner = gate[0].shape[2], gate[0].shape[1]
    g, ga = expert_linear(Qx, sx, rows, offsets, *gate)
    u, ua = expert_linear(Qx, sx, rows, offsets, *up)
    h, dh = swiglu(g, u, linear_error(ga, K), linear_error(ua, K))
    Qh, sh, slack = hidden_slack(h, dh)
    y, ya = expert_linear(Qh, sh, np.arange(len(rows)), offsets, *down)
    dy = linear_error(ya, inner)
    val = bo.e4m3_values()
    for e in range(E):
        i = slice(offsets[e], offsets[e + 1])
        if i.start < i.stop:
            dy[i] += slack[i] @ np.abs(val[down[0][e]] * bo.widen(down[1][e], *down[0][e].shape, bo.BLOCK)).T
    Y, A = combine(y, place, weights, residual)
    D, _ = combine(dy + rows_error * np.abs(y) * (1 + 2.0 ** -10), place, np.abs(weights))
    return Y, D + (k + 3) * U24 * A
