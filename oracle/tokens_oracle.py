"""Plain restatement of the operators around the layers, in float64 and whole
numbers, one token, row or group after the other.  Test infrastructure only."""

from __future__ import annotations

import math

import numpy as np


def embed(tokens, table, scale):
    """[T, d]: scale * table[token], zeros for a token outside the table."""
    out = np.zeros((len(tokens), table.shape[1]))
    for t, v in enumerate(tokens):
        if 0 <= v < len(table):
            out[t] = scale * table[v].astype(np.float64)
    return out


def embed_backward(tokens, dout, V, scale):
    """The table's gradient, and for each entry the sum of the terms' sizes and how many there are."""
    grad, size, terms = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros((V, 1))
    for t, v in enumerate(tokens.tolist()):
        if 0 <= v < V:
            grad[v] += scale * dout[t].astype(np.float64)
            size[v] += abs(scale) * np.abs(dout[t].astype(np.float64))
            terms[v] += 1
    return grad, size, terms


def unpack_w4(codes, scales):
    """W [k, n] of codes [n, k / 2] (low four bits first) and scales [k / group, n]."""
    n, half = codes.shape
    k = 2 * half
    group = k // len(scales)
    W = np.zeros((k, n))
    for j in range(k):
        code = codes[:, j // 2] >> 4 if j % 2 else codes[:, j // 2] & 15
        W[j] = scales[j // group].astype(np.float64) * (code.astype(np.float64) - 8)
    return W


def keep(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The tokens that the filters keep of logits z, by index, and their weights."""
    z = np.asarray(z, np.float64)
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), 3.4028234663852886e38)
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if not len(order):
        return [], []
    if not temperature > 0:
        return [int(order[0])], [1.0]
    if top_k > 0:
        order = order[:top_k]
    weight = np.exp((z[order] - z[order[0]]) / temperature)
    if top_p < 1:
        whole, upto, n = math.fsum(weight), 0.0, 0
        while n < len(order) and (n == 0 or upto < top_p * whole):
            upto += weight[n]
            n += 1
        order, weight = order[:n], weight[:n]
    if min_p > 0:
        order, weight = order[weight >= min(min_p, 1.0)], weight[weight >= min(min_p, 1.0)]
    by = np.argsort(order)
    return order[by].tolist(), weight[by].tolist()


def sample(z, u, **settings):
    """(token, its share of the kept weights, how near u is to another token's part)."""
    kept, weight = keep(z, **settings)
    if not kept:
        return -1, 0.0, math.inf
    whole = math.fsum(weight)
    u = min(max(float(u), 0.0), 1.0)
    upto = np.cumsum(np.array(weight)) / whole
    at = int(np.searchsorted(upto, u, side="right"))
    real = [i for i, w in enumerate(weight) if w > 0]
    at = min(at, real[-1])
    near = float(np.abs(u - upto[:-1]).min()) if len(kept) > 1 else math.inf
    return kept[at], weight[at] / whole, near
