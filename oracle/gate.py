"""The gate of a routed-expert layer, one token at a time: scores, bias, groups, the k best, weights.

Scores are evaluated in fp64 and rounded once to fp32, keys and group scores are fp32 sums, as the
entry point defines them, so that the choice can be compared exactly.
"""

import numpy as np


def scores(logits, score):
    x = np.asarray(logits, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            p = np.where(x == -np.inf, 0.0, np.exp(x - x.max(axis=1, keepdims=True)))
            s = p / p.sum(axis=1, keepdims=True)
    return np.where(x == -np.inf, 0.0, s).astype(np.float32)


def gate(logits, k, bias=None, score="sigmoid", groups=1, top_groups=None, renormalize=True, scale=1.0):
    """(indices int32 [T, k], weights fp64 [T, k]) of rows without NaN."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    sc = scores(logits, score)
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        key = sc[t] if bias is None else sc[t] + np.asarray(bias, np.float32)
        free = (logits[t] != -np.inf) & (key != -np.inf)
        if groups > 1:
            ranked = []
            for g in range(groups):
                members = [key[e] for e in range(g * E // groups, (g + 1) * E // groups) if free[e]]
                members.sort(reverse=True)
                if not members:
                    continue
                best = members[0] if bias is None or len(members) == 1 else np.float32(members[0] + members[1])
                ranked.append((-best, g))
            kept = {g for _, g in sorted(ranked)[:top_groups]}
            free &= np.array([e // (E // groups) in kept for e in range(E)])
        order = sorted((e for e in range(E) if free[e]), key=lambda e: (-key[e], e))[:k]
        s = [float(sc[t, e]) for e in order]
        total = sum(s)
        for j, e in enumerate(order):
            idx[t, j] = e
            w[t, j] = (s[j] / total if total > 0 else 0.0) * scale if renormalize else s[j] * scale
    return idx, w
