"""pa_pool_evict in plain numpy, on a PoolModel."""
import math

import numpy as np


def totals(scores):
    """Exact sums over the heads, rounded to fp32."""
    with np.errstate(invalid="ignore"):
        plain = scores.astype(np.float64).sum(0)
        whole = np.isfinite(scores).all(0)
        plain[whole] = [math.fsum(x) for x in scores[:, whole].T.astype(np.float64)]
        return plain.astype(np.float32)


def choose(scores, n, budget, first, last):
    """Kept places of a row of n tokens; scores [heads, >= n]."""
    if n <= budget:
        return np.arange(n)
    total = totals(scores[:, :n])
    nan = np.isnan(total)  # below every number
    total = np.where(nan, 0, total)
    middle = np.arange(first, n - last)
    order = middle[np.lexsort((middle, -total[middle].astype(np.float64), nan[middle]))]
    return np.sort(np.concatenate([np.arange(first), order[:budget - first - last], np.arange(n - last, n)]))


def evict(model, rows, scores, budget, first, last, apart=None):
    """(kept, scores afterwards), or None (refused); scores [rows, heads, tokens]."""
    bs, out = model.bs, scores.copy() if apart is None else apart.copy()
    kept = np.full((len(rows), budget), -1, np.int32)
    if len(set(rows)) < len(rows) or any(not 0 <= r < len(model.ctx) for r in rows):
        return None
    plan = []
    for i, r in enumerate(rows):
        n = int(model.ctx[r])
        if not 0 <= n <= model.tables.shape[1] * bs:
            return None
        keep = choose(scores[r], n, budget, first, last)
        plan.append((i, r, n, keep))
        if n <= budget:
            continue
        pages = model.tables[r, :-(-n // bs)]
        if (pages < 0).any() or (pages >= len(model.refs)).any() or (model.refs[pages] < 1).any():
            return None
        moved = np.flatnonzero(keep != np.arange(budget))
        if len(moved) and (model.refs[pages[moved[0] // bs:-(-budget // bs)]] != 1).any():
            return None
    for i, r, n, keep in plan:
        kept[i, :len(keep)] = keep
        out[r][:, :len(keep)] = scores[r][:, keep]
        out[r][:, len(keep):n] = 0
        if n <= budget:
            continue
        row = model.tables[r].astype(np.int64)
        k = np.arange(budget)
        for x in model.pages:
            x[:, row[k // bs], k % bs] = x[:, row[keep // bs], keep % bs]
        for x in model.scales:
            x[:, row[k // bs], :, k % bs] = x[:, row[keep // bs], :, keep % bs]
        gone = slice(-(-budget // bs), -(-n // bs))
        for page in model.tables[r, gone]:
            model.refs[page] -= 1
        model.tables[r, gone] = -1
        model.ctx[r] = budget
    return kept, out
