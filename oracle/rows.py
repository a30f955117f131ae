"""What the per-row calls compute (routing, combine, adapters), token by token
in 64 bits from the definitions in include/qlin.h; test infrastructure only.
The dispatch needs nothing of its own: its codes and scales are quant_act's.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = 3.4028234663852886e38
SOFTMAX, SIGMOID = 0, 1
MAX, TOP2 = 0, 1


def _best(values, n):
    """Indices of the n largest values, ties to the lowest index, -inf never."""
    order = sorted(range(len(values)), key=lambda i: (-values[i], i))
    return [i for i in order[:n] if values[i] > -np.inf]


def route(logits, topk, score=SOFTMAX, bias=None, groups=1, topk_groups=1, group_score=MAX, renormalize=1, scale=1.0):
    """logits [T, E] -> (ids [T, k], weights [T, k], offsets [E + 1],
    rows [T k], slots [T, k]); ids -1, weight 0 and slot -1 where fewer than k
    experts are open."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, topk), -1, dtype=np.int32)
    weights = np.zeros((T, topk))
    for t in range(T):
        l = np.minimum(logits[t], FLT_MAX)
        is_open = ~np.isnan(l) & (l > -np.inf)
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == SIGMOID:
                s[is_open] = 1.0 / (1.0 + np.exp(-l[is_open]))
            elif is_open.any():
                e = np.exp(l[is_open] - l[is_open].max())
                s[is_open] = e / e.sum()
        if bias is None and (groups == 1 or group_score == MAX):
            c = np.where(is_open, l, -np.inf)     # the scores' order, where they would round to ties
        else:
            b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
            c = np.where(is_open & ~np.isnan(b) & (b > -np.inf), s + np.where(np.isnan(b), 0.0, b), -np.inf)
        if groups > 1:
            worth = []
            for g in range(groups):
                in_g = sorted((v for v in c[g * (E // groups):(g + 1) * (E // groups)] if v > -np.inf), reverse=True)
                worth.append(-np.inf if not in_g else sum(in_g[:2]) if group_score == TOP2 else
                             in_g[0])
            kept = _best(worth, topk_groups)
            c = np.array([v if e // (E // groups) in kept else -np.inf for e, v in enumerate(c)])
        chosen = _best(c, topk)
        ids[t, :len(chosen)] = chosen
        w = s[chosen]
        if renormalize and len(chosen):
            if score == SOFTMAX:     # the others' exponentials cancel: no underflow
                w = np.exp(l[chosen] - l[chosen].max())
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        weights[t, :len(chosen)] = w * scale
    return (ids, weights) + group_rows(ids, E)


def group_rows(ids, E):
    """Rows of the (token, choice) pairs, in expert then token order."""
    T, k = ids.shape
    pairs = sorted((int(ids[t, j]), t, j) for t in range(T) for j in range(k) if ids[t, j] >= 0)
    offsets = np.zeros(E + 1, dtype=np.int32)
    rows = np.full(T * k, -1, dtype=np.int32)
    slots = np.full((T, k), -1, dtype=np.int32)
    for i, (e, t, j) in enumerate(pairs):
        offsets[e + 1] += 1
        rows[i] = t
        slots[t, j] = i
    return np.cumsum(offsets).astype(np.int32), rows, slots


def combine(h, slots, weights, add=None):
    """(y, sum of the absolute terms): y[t] = add[t] + sum_j w[t,j] h[slots[t,j]]."""
    T, k = slots.shape
    y = np.zeros((T, h.shape[1])) if add is None else np.array(add, dtype=np.float64)
    size = np.abs(y)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < len(h):
                term = float(weights[t, j]) * h[slots[t, j]].astype(np.float64)
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def lora(x, ids, A, B, ranks=None, scales=None, base=None):
    """(y, delta sizes): y[m] = base[m] + s_a B_a (A_a x[m]).  The sizes are
    (sum |B| |v|, sum |B| (sum |A| |x|)), times |s_a|, what rounding errors
    are measured by."""
    M, n = len(x), len(A)
    N = B.shape[1]
    y = np.zeros((M, N)) if base is None else np.array(base, dtype=np.float64)
    of_v, of_terms = np.zeros((M, N)), np.zeros((M, N))
    for m in range(M):
        a = int(ids[m])
        if not 0 <= a < n:
            continue
        r = A.shape[1] if ranks is None else min(max(int(ranks[a]), 0), A.shape[1])
        s = 1.0 if scales is None else float(scales[a])
        Aa, Ba, xm = A[a, :r].astype(np.float64), B[a, :, :r].astype(np.float64), x[m].astype(np.float64)
        v = Aa @ xm
        y[m] += s * (Ba @ v)
        of_v[m] = abs(s) * (np.abs(Ba) @ np.abs(v))
        of_terms[m] = abs(s) * (np.abs(Ba) @ (np.abs(Aa) @ np.abs(xm)))
    return y, of_v, of_terms
