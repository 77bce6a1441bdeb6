"""The scored router's definition in numpy float64, token by token (tests only)."""
import numpy as np


def scores(L, sigmoid):
    L = np.asarray(L, np.float64)
    with np.errstate(over="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-L))
        p = np.exp(L - L.max(axis=1, keepdims=True))
    return p / p.sum(axis=1, keepdims=True)


def select(L, balance, k, sigmoid=False, n_groups=1, top_groups=1, group_top=1, renormalise=True, scale=1.0):
    """ids [T][k], weights [T][k] of logits L [T][E]."""
    s = scores(L, sigmoid)
    T, E = s.shape
    gs = E // n_groups
    ids = np.empty((T, k), np.int32)
    w = np.empty((T, k))
    for t in range(T):
        c = s[t] if balance is None else s[t] + np.asarray(balance, np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        allowed = np.ones(E, bool)
        if top_groups < n_groups:
            score = np.array([np.sort(c[g * gs:(g + 1) * gs])[::-1][:group_top].sum() for g in range(n_groups)])
            order = np.argsort(-score, kind="stable")[:top_groups]
            allowed = np.isin(np.arange(E) // gs, order)
        cand = np.nonzero(allowed)[0]
        ids[t] = cand[np.argsort(-c[cand], kind="stable")[:k]]
        g = s[t, ids[t]]
        if renormalise:
            g = g / g.sum() if g.sum() > 0 else np.zeros(k)
        w[t] = g * scale
    return ids, w


def permute(ids, E):
    flat = ids.reshape(-1)
    counts = np.bincount(flat, minlength=E).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    perm = np.argsort(flat, kind="stable").astype(np.int32)
    inv = np.empty_like(perm)
    inv[perm] = np.arange(perm.size, dtype=np.int32)
    return counts, offsets, perm, inv


def decided(L, balance, slack, sigmoid=False, n_groups=1, top_groups=1, group_top=1, k=1):
    """Per token: no logit error up to `slack` changes the kept groups, the choice or its order."""
    s = scores(L, sigmoid)
    err = slack * s * (1 - s) if sigmoid else 2 * slack * s
    T, E = s.shape
    gs = E // n_groups
    out = np.ones(T, bool)
    for t in range(T):
        c = s[t] if balance is None else s[t] + np.asarray(balance, np.float64)
        cand = np.arange(E)
        if top_groups < n_groups:
            score = np.array([np.sort(c[g * gs:(g + 1) * gs])[::-1][:group_top].sum() for g in range(n_groups)])
            e = group_top * np.array([err[t, g * gs:(g + 1) * gs].max() for g in range(n_groups)])
            order = np.argsort(-score, kind="stable")
            kept, rest = order[:top_groups], order[top_groups:]
            out[t] &= (score[kept] - e[kept]).min() > (score[rest] + e[rest]).max()
            cand = np.nonzero(np.isin(np.arange(E) // gs, kept))[0]
        o = cand[np.argsort(-c[cand], kind="stable")[:k + 1]]
        out[t] &= bool(np.all(c[o[:-1]] - err[t, o[:-1]] > c[o[1:]] + err[t, o[1:]]))
    return out
