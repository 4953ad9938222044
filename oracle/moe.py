"""Oracle for the calls around a mixture of experts: routing with its balance loss, the copy of
tokens into the experts' row order, and the weighted return, with their gradients, in FP64.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product library; it shares no
code with the CUDA path.

The definitions (T tokens, E experts, k per token; l the logits, an open token has mask != 0
and a logit above -inf):

  p_t = softmax(l_t), S_t = the k open experts of the largest logits (ties: the lower expert,
  a NaN first), w_tj = p_t[S_tj] or p_t[S_tj] / sum_i p_t[S_ti], c_e = #{(t, j): S_tj = e},
  R = sum c, n = open tokens, L = coef E sum_e (c_e / R) (sum_t p_te / n),
  row_tj = sum_{e' < e} c_e' + #{t' < t : e in S_t'} for e = S_tj.
"""
from __future__ import annotations

import numpy as np


def route(logits, top_k, normalize, coef, mask=None):
    """expert, weight, row, counts, totals, loss of FP64 logits (T x E)."""
    l = np.array(logits, dtype=np.float64)
    T, E = l.shape
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    expert = np.full((T, top_k), -1, dtype=np.int32)
    weight = np.zeros((T, top_k))
    prob = np.zeros(E)
    live = 0
    for t in range(T):
        open_ = np.flatnonzero(l[t] != -np.inf)   # a NaN is not -inf
        if open_.size == 0:
            continue
        live += 1
        nan = np.isnan(l[t, open_])
        order = open_[np.lexsort((open_, np.where(nan, 0.0, -l[t, open_]), ~nan))][:top_k]
        with np.errstate(invalid="ignore"):
            x = np.exp(l[t] - (np.nan if np.isnan(l[t]).any() else l[t].max()))
        p = x / x.sum()
        prob += p
        w = p[order] / p[order].sum() if normalize else p[order]
        expert[t, :len(order)] = order
        weight[t, :len(order)] = w
    counts = np.bincount(expert[expert >= 0], minlength=E).astype(np.int32)
    first = np.concatenate([[0], np.cumsum(counts)[:-1]])
    row = np.full((T, top_k), -1, dtype=np.int32)
    for e in range(E):
        at = np.argwhere(expert == e)   # by token: an expert occurs once in a row
        row[at[:, 0], at[:, 1]] = first[e] + np.arange(len(at))
    R = int(counts.sum())
    loss = coef * E * float(np.sum(counts / max(R, 1) * (prob / max(live, 1))))
    return dict(expert=expert, weight=weight, row=row, counts=counts, totals=np.array([R, live], dtype=np.int32),
                loss=loss)


def route_loss(logits, weights_dot, d_loss, r, normalize, coef, mask=None):
    """sum(weights_dot * weight) + d_loss * loss as a function of the logits, with the choice r and its
    counts held fixed: what route_backward differentiates."""
    l = np.array(logits, dtype=np.float64)
    E = l.shape[1]
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    R, n = (max(int(v), 1) for v in r["totals"])
    total = 0.0
    for t in range(l.shape[0]):
        if not (l[t] > -np.inf).any():
            continue
        x = np.exp(l[t] - l[t].max())
        p = x / x.sum()
        total += d_loss * coef * E * float(np.sum(r["counts"] / R * p)) / n
        s = r["expert"][t][r["expert"][t] >= 0]
        w = p[s] / p[s].sum() if normalize else p[s]
        total += float(np.sum(weights_dot[t][:len(s)] * w))
    return total


def route_backward(logits, d_weight, d_loss, r, normalize, coef, mask=None):
    """The gradient of route_loss, and per element the sum of the magnitudes it adds up."""
    l = np.array(logits, dtype=np.float64)
    T, E = l.shape
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    R, n = (max(int(v), 1) for v in r["totals"])
    g0 = d_loss * coef * E * r["counts"].astype(np.float64) / (R * n)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if not (l[t] > -np.inf).any():
            continue
        x = np.exp(l[t] - l[t].max())
        p = x / x.sum()
        s = r["expert"][t][r["expert"][t] >= 0]
        dw = d_weight[t][:len(s)]
        g = g0.copy()
        if not normalize:
            g[s] += dw
        out[t] = p * (g - np.sum(p * g))
        size[t] = p * (np.abs(g0) + np.abs(g - g0) + np.sum(p * (np.abs(g0) + np.abs(g - g0))))
        if normalize:
            w = p[s] / p[s].sum()
            out[t, s] += w * (dw - np.sum(w * dw))
            size[t, s] += w * (np.abs(dw) + np.sum(w * np.abs(dw)))
    return out, size


def round_e4m3(v):
    """FP64 -> the nearest e4m3 value (ties to even), saturated to +-448; NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
        q = np.rint(v / 2.0 ** (e - 3)) * 2.0 ** (e - 3)
    return np.where(np.isnan(v), np.nan, np.clip(q, -448.0, 448.0))


def quantize(x):
    """e4m3 values and FP32 scales of FP32 x (T x H) in 1 x 128 tiles, with the FP32 steps of the
    definition: amax at least 2^-96, scale = amax / 448, value = x * (448 / amax)."""
    x = np.asarray(x, dtype=np.float32)
    T, H = x.shape
    blocks = -(-H // 128)
    pad = np.zeros((T, blocks * 128), dtype=np.float32)
    pad[:, :H] = x
    pad = pad.reshape(T, blocks, 128)
    amax = np.maximum(np.abs(pad).max(axis=2), np.float32(2.0 ** -96))
    with np.errstate(invalid="ignore"):
        scale = amax / np.float32(448.0)
        v = pad * (np.float32(448.0) / amax)[:, :, None]
    return round_e4m3(v.astype(np.float64)).reshape(T, blocks * 128)[:, :H], scale


def combine(rows, row, weight=None):
    """out and per element the sum of magnitudes; rows FP64, row T x k (-1: none)."""
    rows = np.asarray(rows, dtype=np.float64)
    T, k = row.shape
    out, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for j in range(k):
        has = row[:, j] >= 0
        v = rows[row[has, j]] * (1.0 if weight is None else np.asarray(weight, dtype=np.float64)[has, j, None])
        out[has] += v
        size[has] += np.abs(v)
    return out, size


def combine_backward(rows, row, weight, d_out):
    """d_rows (NaN where no token names the row), d_weight and the sums of its magnitudes."""
    rows, d_out = np.asarray(rows, dtype=np.float64), np.asarray(d_out, dtype=np.float64)
    T, k = row.shape
    d_rows = np.full(rows.shape, np.nan)
    d_weight, size = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        has = row[:, j] >= 0
        r = row[has, j]
        d_rows[r] = d_out[has] * np.asarray(weight, dtype=np.float64)[has, j, None]
        d_weight[has, j] = np.sum(d_out[has] * rows[r], axis=1)
        size[has, j] = np.sum(np.abs(d_out[has] * rows[r]), axis=1)
    return d_rows, d_weight, size


# ------------------------------------------------------------------ routing by scores
def scores(l, sigmoid):
    """Sigmoid or softmax scores of one token's FP64 logits (-inf: closed, 0)."""
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        x = np.exp(l - (np.nan if np.isnan(l).any() else l.max()))
        return x / x.sum()


def shares(l, sigmoid):
    """Scores over their sum, from the logits where the scores themselves would vanish."""
    if sigmoid and l.max() < -30.0:   # 1 / (1 + e^-l) = e^l (1 + O(e^-30)) / ...: exact to 1e-13
        x = np.exp(l - l.max())
        return x / x.sum()
    s = scores(l, sigmoid)
    return s / s.sum()


def route_scored(logits, top_k, sigmoid, bias=None, groups=1, top_groups=1, best=1, normalize=True, scale=1.0, coef=0.0,
                 mask=None):
    """expert, weight, row, counts, totals, loss of FP64 logits (T x E) by the definition of moe_route_scored."""
    l = np.array(logits, dtype=np.float64)
    T, E = l.shape
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    size = E // groups
    expert = np.full((T, top_k), -1, dtype=np.int32)
    weight, prob, live = np.zeros((T, top_k)), np.zeros(E), 0
    for t in range(T):
        open_ = l[t] != -np.inf
        if not open_.any():
            continue
        live += 1
        s = scores(l[t], sigmoid)
        with np.errstate(invalid="ignore"):
            c = s + b
            if bias is None and not sigmoid and not np.isnan(s).any():
                c = np.exp(l[t] - l[t].max())   # compared before the division
        c = np.where(np.isnan(c), np.inf, c)
        c[~open_] = -np.inf
        prob += np.where(open_, shares(l[t], sigmoid), 0.0)
        value = []
        for g in range(groups):
            top = np.sort(c[g * size:(g + 1) * size])[::-1][:best]
            value.append(top[top > -np.inf].sum() if top[0] > -np.inf else -np.inf)
        keep = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        pool = [e for g in keep for e in range(g * size, (g + 1) * size) if c[e] > -np.inf]
        chosen = sorted(pool, key=lambda e: (-c[e], e))[:top_k]
        if chosen:
            w = shares(l[t, chosen], sigmoid) if normalize else s[chosen]
            expert[t, :len(chosen)] = chosen
            weight[t, :len(chosen)] = w * scale
    counts = np.bincount(expert[expert >= 0], minlength=E).astype(np.int32)
    first = np.concatenate([[0], np.cumsum(counts)[:-1]])
    row = np.full((T, top_k), -1, dtype=np.int32)
    for e in range(E):
        at = np.argwhere(expert == e)
        row[at[:, 0], at[:, 1]] = first[e] + np.arange(len(at))
    R = int(counts.sum())
    loss = coef * E * float(np.sum(counts / max(R, 1) * (prob / max(live, 1)))) if R else 0.0
    return dict(expert=expert, weight=weight, row=row, counts=counts, totals=np.array([R, live], dtype=np.int32), loss=loss)


def route_scored_loss(logits, weights_dot, d_loss, r, sigmoid, normalize, scale, coef, mask=None):
    """sum(weights_dot * weight) + d_loss * loss as a function of the logits, the choice r and its counts fixed: what
    moe_route_scored_backward differentiates."""
    l = np.array(logits, dtype=np.float64)
    E = l.shape[1]
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    R, n = (max(int(v), 1) for v in r["totals"])
    total = 0.0
    for t in range(l.shape[0]):
        if not (l[t] > -np.inf).any():
            continue
        total += d_loss * coef * E * float(np.sum(r["counts"] / R * shares(l[t], sigmoid))) / n
        s = r["expert"][t][r["expert"][t] >= 0]
        if len(s):
            w = shares(l[t, s], sigmoid) if normalize else scores(l[t], sigmoid)[s]
            total += scale * float(np.sum(weights_dot[t][:len(s)] * w))
    return total


def route_scored_backward(logits, d_weight, d_loss, r, sigmoid, normalize, scale, coef, mask=None):
    """The gradient of route_scored_loss, and per element the sum of the magnitudes it adds up."""
    l = np.array(logits, dtype=np.float64)
    T, E = l.shape
    if mask is not None:
        l[np.asarray(mask) == 0] = -np.inf
    R, n = (max(int(v), 1) for v in r["totals"])
    g = d_loss * coef * E * r["counts"].astype(np.float64) / (R * n)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        open_ = l[t] > -np.inf
        if not open_.any():
            continue
        p = np.where(open_, shares(l[t], sigmoid), 0.0)
        u, m = p * (g - np.sum(p * g)), p * (np.abs(g) + np.sum(p * np.abs(g)))
        s = r["expert"][t][r["expert"][t] >= 0]
        if len(s):
            dw = scale * d_weight[t][:len(s)]
            if normalize:
                q = shares(l[t, s], sigmoid)
                u[s] += q * (dw - np.sum(q * dw))
                m[s] += q * (np.abs(dw) + np.sum(q * np.abs(dw)))
            else:
                sc = scores(l[t], sigmoid)[s]
                u[s] += sc * dw
                m[s] += sc * np.abs(dw)
        with np.errstate(over="ignore"):
            rest = 1.0 / (1.0 + np.exp(l[t]))   # 1 - s
        out[t] = u * rest if sigmoid else u - p * u.sum()
        size[t] = m * rest if sigmoid else m + p * m.sum()
        out[t][~open_], size[t][~open_] = 0.0, 0.0
    return out, size


def quantize_int8(x):
    """int8 values and FP32 scales of the rows of FP32 x, with the FP32 steps of the definition."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.maximum(np.abs(x).max(axis=1), np.float32(2.0 ** -96))
    with np.errstate(invalid="ignore"):
        v = x * (np.float32(127.0) / amax)[:, None]
        return np.rint(v), amax / np.float32(127.0)
