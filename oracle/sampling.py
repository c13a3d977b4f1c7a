"""Plain CPU form of the sampler: one row at a time, in binary64, from the
definitions.  No arithmetic is shared with the GPU side."""
from __future__ import annotations

import math

import numpy as np


def masses(row, temperature):
    """exp((x - best) / temperature) of a row given in its own type, the
    temperature as binary32 holds it; 0 for -infinity and NaN, 1 for every token
    of an infinite best."""
    temperature = float(np.float32(temperature))
    x = np.where(np.isnan(row), -np.inf, np.asarray(row, np.float64))
    best = x.max()
    if best == -np.inf:
        return np.zeros(len(x))
    with np.errstate(invalid="ignore"):
        z = np.where(x == best, 0.0, (x - best) / (temperature or 1.0))
    return np.exp(z)


def kept(row, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Tokens that stay, in ascending order.  top_p and min_p as binary32 holds
    them."""
    top_p, min_p = float(np.float32(top_p)), min(float(np.float32(min_p)), 1.0)
    if not 0 < temperature < math.inf:
        temperature, top_k, top_p, min_p = 0.0, 1, 1.0, 0.0
    x = np.where(np.isnan(row), -np.inf, np.asarray(row, np.float64))
    m = masses(row, temperature)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1 and len(order):
        whole = math.fsum(m[order])
        before = np.concatenate(([0.0], np.cumsum(m[order])[:-1]))
        n = max(1, int((before < top_p * whole).sum()))
        order = order[:n]
    if min_p > 0:
        order = order[m[order] >= min_p]
    return np.sort(order)


def draw(row, tokens, temperature, u, without=None):
    """(token, its probability) among `tokens` (ascending), one of them left out."""
    tokens = tokens[tokens != without] if without is not None else tokens
    if len(tokens) == 0:
        return -1, 0.0
    m = masses(np.asarray(row)[tokens], temperature if 0 < temperature < math.inf else 0.0)
    if not 0 < temperature < math.inf:
        m = np.ones(len(tokens))
    whole = math.fsum(m)
    c = np.cumsum(m)
    u = min(max(float(u), 0.0), 1 - 2.0 ** -53) if u == u else 0.0
    at = min(int(np.searchsorted(c, u * c[-1], side="right")), len(tokens) - 1)
    return int(tokens[at]), float(m[at] / whole)


def p_draft(row, tokens, temperature, d):
    if d not in tokens:
        return 0.0
    m = masses(np.asarray(row)[tokens], temperature) if 0 < temperature < math.inf else np.ones(len(tokens))
    return float(m[tokens == d][0] / math.fsum(m))
