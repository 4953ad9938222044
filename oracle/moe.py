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
