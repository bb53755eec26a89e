"""The router in 64 bits (numpy), straight from its formulas: scores, keys,
groups, selection, weights and the gradient of the logits."""
from __future__ import annotations

import numpy as np


def scores(l, score):
    l = np.asarray(l, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    z = e.sum(1, keepdims=True)
    return e / np.where(z == 0, 1.0, z)


def keys(l, score, bias, group_top=1):
    if score == "softmax" and bias is None and group_top == 1:
        return np.asarray(l, np.float64)
    k = scores(l, score)
    return k if bias is None else k + np.asarray(bias, np.float64)[None]


def open_experts(key, groups, topk_groups, group_top):
    """Truth values [T, E]: the expert's group is one of the topk_groups best."""
    T, E = key.shape
    per = np.sort(key.reshape(T, groups, E // groups), axis=2)[:, :, ::-1]
    worth = per[:, :, :group_top].sum(2)
    rank = np.argsort(-worth, axis=1, kind="stable")[:, :topk_groups]
    is_open = np.zeros((T, groups), bool)
    np.put_along_axis(is_open, rank, True, 1)
    return np.repeat(is_open, E // groups, 1)


def select(key, K, is_open):
    """K best keys of the open experts, ties to the lowest index; an open
    expert of key -inf comes before every closed one."""
    out = np.empty((key.shape[0], K), np.int64)
    for t in range(key.shape[0]):
        order = sorted(range(key.shape[1]), key=lambda e: (not is_open[t, e], -key[t, e], e))
        out[t] = order[:K]
    return out


def weights(p, ids, renormalize, scale):
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        s = w.sum(1, keepdims=True)
        w = w / np.where(s == 0, 1.0, s)
    return scale * w


def d_logits(l, ids, dw, ds, score, renormalize, scale):
    """(gradient, a bound of the magnitude of its terms) [T, E]."""
    p = scores(l, score)
    g = np.zeros(ids.shape) if dw is None else scale * np.asarray(dw, np.float64)
    sel = np.take_along_axis(p, ids, 1)
    mag = np.abs(g)
    if renormalize:
        s = sel.sum(1, keepdims=True)
        s = np.where(s == 0, 1.0, s)
        mag = (mag + (np.abs(g) * sel / s).sum(1, keepdims=True)) / s
        g = (g - (g * sel / s).sum(1, keepdims=True)) / s
    dp, dm = np.zeros_like(p), np.zeros_like(p)
    np.put_along_axis(dp, ids, g, 1)
    np.put_along_axis(dm, ids, mag, 1)
    if ds is not None:
        dp, dm = dp + ds, dm + np.abs(ds)
    if score == "sigmoid":
        return dp * p * (1 - p), dm * p
    return p * (dp - (dp * p).sum(1, keepdims=True)), p * (dm + (dm * p).sum(1, keepdims=True))
