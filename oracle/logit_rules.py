"""Plain CPU form of the rules on logits and of the verification under them.
``ruled`` follows the documented order in a chosen type: binary32 is bit-exact,
binary64 is the formula.  Rules are numpy arrays under the names of the device
struct; missing ones are None."""
from __future__ import annotations

import numpy as np

NONE = dict(history=None, history_offsets=None, n_prompt=None, repetition=None, frequency=None, presence=None,
            bias_ids=None, bias_values=None, bias_offsets=None, mask=None, mask_index=None)


def _span(offsets, i, n):
    lo, hi = (int(min(max(int(v), 0), n)) for v in (offsets[i], offsets[i + 1]))
    return slice(lo, max(lo, hi))


def counts(rules, drafts, i, t, V):
    """(seen [V], generated count [V]) of row t of request i."""
    r = {**NONE, **rules}
    seen, made = np.zeros(V, bool), np.zeros(V, np.int64)
    if r["history"] is not None:
        words = np.asarray(r["history"][_span(r["history_offsets"], i, len(r["history"]))], np.int64)
        n = 0 if r["n_prompt"] is None else int(r["n_prompt"][i])
        for k, v in enumerate(words):
            if 0 <= v < V:
                seen[v] = True
                made[v] += k >= n
    for v in (drafts[i][:t] if t else ()):
        if 0 <= v < V:
            made[v] += 1
    return seen | (made > 0), made


def ruled(logits, rules, drafts, R, T, dtype=np.float32):
    """The ruled logits [R*T, V] in `dtype`."""
    r = {**NONE, **rules}
    x = np.array(logits, dtype)
    V = x.shape[1]
    any_penalty = any(r[k] is not None for k in ("repetition", "frequency", "presence"))
    one = lambda name, i, d: dtype(d if r[name] is None else r[name][i])  # noqa: E731
    with np.errstate(all="ignore"):
        for i in range(R):
            for t in range(T):
                row = x[i * T + t]
                if any_penalty:
                    seen, made = counts(r, drafts, i, t, V)
                    rep = one("repetition", i, 1)
                    row[seen] = np.where(row[seen] > 0, row[seen] / rep, row[seen] * rep)
                    m = made > 0
                    row[m] = row[m] - one("frequency", i, 0) * made[m].astype(dtype)
                    row[m] = row[m] - one("presence", i, 0)
                if r["bias_ids"] is not None:
                    span = _span(r["bias_offsets"], i, len(r["bias_ids"]))
                    last = dict(zip(r["bias_ids"][span].tolist(), r["bias_values"][span].tolist()))
                    for v, b in last.items():
                        if 0 <= v < V:
                            row[v] = row[v] + dtype(b)
                if r["mask"] is not None:
                    at = i * T + t if r["mask_index"] is None else int(r["mask_index"][i * T + t])
                    if at >= len(r["mask"]):
                        row[:] = -np.inf
                    elif at >= 0:
                        words = np.asarray(r["mask"][at]).view(np.uint32)
                        bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                        row[bits == 0] = -np.inf
    return x


def top(row, k):
    """Ids and values of the k best of a row: larger value, then lower id;
    (-1, -inf) past the values above -inf.  NaN is never taken."""
    live = np.nonzero(row > -np.inf)[0]
    best = live[np.lexsort((live, -row[live].astype(np.float64)))][:k]
    ids, val = np.full(k, -1, np.int64), np.full(k, -np.inf, row.dtype)
    ids[: len(best)], val[: len(best)] = best, row[best]
    return ids, val


def lse64(row, tau):
    z = row[row > -np.inf].astype(np.float64)
    if z.size == 0:
        return -np.inf
    m = z.max()
    return m / tau if np.isinf(m) else m / tau + np.log(np.exp((z - m) / tau).sum())


def probability64(row, d, tau, k):
    """The draft's probability among the k best (k >= 1) or the whole row."""
    ids, val = top(row, k if k else len(row))
    if d not in ids[ids >= 0]:
        return 0.0
    z = val[ids >= 0].astype(np.float64)
    e = np.where(z == z[0], 1.0, np.exp(np.where(z == z[0], 0.0, (z - z[0]) / tau)))
    return float(e[ids[ids >= 0] == d][0] / e.sum())
