"""Plain statements of the operators on drafted tokens for the tests, one token at a time."""
from __future__ import annotations

import math

import numpy as np


def chain(n):
    return list(range(-1, n - 1))


def random_tree(rng, n, back=None, roots=1):
    """Parents of n tokens, the first `roots` without one; back: how many tokens before it a parent is at most."""
    return [-1 if i < roots else int(rng.integers(max(0, i - (back or i)), i)) for i in range(n)]


def line(parents, i):
    """Token i and those above it, from the top."""
    got = []
    while i >= 0:
        got.append(i)
        i = parents[i]
    return got[::-1]


def accepted(parents, tokens, targets):
    """Places of the accepted tokens, and what follows the last."""
    if not len(parents):
        return [], -1
    path = [0]
    while True:
        u = path[-1]
        child = [c for c in range(len(parents)) if parents[c] == u and tokens[c] == targets[u]]
        if not child:
            return path, int(targets[u])
        path.append(child[0])


def rules(logits, history, counted_from, path, repetition, presence, frequency, bias, mask):
    """One row's logits after the rules, in 64 bits.  bias: (token, value) entries in order; mask: truth values or None."""
    l = np.array(logits, np.float64)
    V = len(l)
    fine = lambda t: [x for x in t if 0 <= x < V]  # noqa: E731
    seen = np.bincount(fine(list(history) + list(path)), minlength=V) > 0
    n = np.bincount(fine(list(history[counted_from:]) + list(path)), minlength=V)
    with np.errstate(invalid="ignore", over="ignore"):
        l = np.where(seen, np.where(l > 0, l / repetition, l * repetition), l)
        l = np.where(n > 0, l - (frequency * n + presence), l)
        for token, value in dict(bias).items():
            if 0 <= token < V:
                l[token] += value
    if mask is not None:
        l[~np.asarray(mask)] = -math.inf
    return l


def rope(x, angle, amplitude, half):
    """Rows x [rows][heads][hs] turned by angle [rows][pairs], in 64 bits."""
    x = np.array(x, np.float64)
    n = 2 * angle.shape[1]
    a, b = (slice(0, n // 2), slice(n // 2, n)) if half else (slice(0, n, 2), slice(1, n, 2))
    y = x.copy()
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y
