"""Routing in 64 bits, token by token (test infrastructure only)."""
import numpy as np


def route(x, k, score, bias, n_groups, top_groups, group_score, renorm, scale):
    """x [T, E] float64 (finite or -inf), bias [E] or None -> ids [T, k], weights [T, k], span [T] (of the exponentials' arguments)."""
    T, E = x.shape
    size = E // n_groups
    ids, w, span = np.zeros((T, k), np.int64), np.zeros((T, k)), np.zeros(T)
    for t in range(T):
        v = x[t]
        closed = np.isneginf(v)
        if score == "softmax":
            top = v.max() if not closed.all() else 0.0
            e = np.exp(v - top)
            p = e / e.sum() if e.sum() else e
        else:
            with np.errstate(over="ignore"):
                p = 1.0 / (1.0 + np.exp(-v))
        c = np.where(closed, -np.inf, p + bias) if bias is not None else v
        d = p if bias is None and group_score == "top2" and size > 1 else c
        worth = []
        for g in range(n_groups):
            m = [d[i] for i in range(g * size, (g + 1) * size) if not closed[i]]
            m.sort(reverse=True)
            worth.append(-np.inf if not m else m[0] if group_score == "max" else sum(m[:2]))
        kept = sorted(range(n_groups), key=lambda g: (-worth[g], g))[:top_groups]
        among = [i for g in kept for i in range(g * size, (g + 1) * size)]
        among.sort(key=lambda i: (-c[i], i))
        ids[t] = among[:k]
        q = p[ids[t]]
        if renorm:
            m = np.minimum(v[ids[t]], 0) if score == "sigmoid" else v[ids[t]]
            best = m.max()
            if np.isneginf(best):
                q = np.zeros(k)
            else:
                q = np.exp(m - best)
                if score == "sigmoid":
                    q = q / (1 + np.exp(-np.abs(v[ids[t]])))
                q = q / q.sum()
        w[t] = q * scale
        fin = v[~closed]
        span[t] = (fin.max() - fin.min() + np.abs(fin).max()) if fin.size else 0
    return ids, w, span
