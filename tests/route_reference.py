"""Routing by scores, bias and groups by its definition in 64 bits (numpy).
Shares no code with the library."""
import numpy as np


def _descending(v):
    """Indices by descending value, ties to the lowest, NaN last."""
    return np.argsort(np.where(np.isnan(v), np.inf, -v), kind="stable")


def route(logits, k, bias=None, sigmoid=True, groups=1, top_groups=1, group_best=2, renorm=True, scale=1.0):
    """(ids [M, k], weights [M, k], gap): gap is the least difference between
    a chosen score (or group's) and the next one down."""
    M, E = logits.shape
    per = E // groups
    ids, weights, gap = np.zeros((M, k), np.int64), np.zeros((M, k)), np.inf
    for m in range(M):
        l = logits[m]
        if sigmoid:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max())
            s = s / s.sum()
        c = s if bias is None else s + bias
        order = _descending(c)
        if top_groups < groups:
            score = np.array([np.sort(c[g * per:(g + 1) * per])[::-1][:group_best].sum() for g in range(groups)])
            rank = _descending(score)
            gap = min(gap, score[rank[top_groups - 1]] - score[rank[top_groups]])
            order = order[np.isin(order // per, rank[:top_groups])]
        top = c[order]
        if len(top) > 1:
            gap = min(gap, (top[:-1] - top[1:])[:k].min())
        ids[m] = order[:k]
        w = s[ids[m]]
        weights[m] = w * scale / (w.sum() if renorm else 1.0)
    return ids, weights, gap
