"""The router's balance loss from its definition, in 64 bits (NumPy), for the tests."""
from __future__ import annotations

import numpy as np

ULP = 2.0 ** -23


def choices(l: np.ndarray, k: int) -> np.ndarray:
    """[T][E] 0 / 1: the k largest logits of each row, ties to the lower index, never -inf."""
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    hot = np.zeros(l.shape)
    np.put_along_axis(hot, order, 1.0, 1)
    return hot * (l > -np.inf)


def _softmax(v):
    e = np.exp(v - v.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def scores(l: np.ndarray, scoring: str) -> np.ndarray:
    if scoring == "softmax":
        return _softmax(l)
    return _softmax(np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l))))


def lse(l: np.ndarray) -> np.ndarray:
    m = l.max(1)
    return m + np.log(np.exp(l - m[:, None]).sum(1))


def rows_of(l, lo, hi, mask):
    """The tokens of [lo, hi) that count."""
    t = np.arange(lo, hi)
    if mask is not None:
        t = t[mask[t]]
    with np.errstate(invalid="ignore"):
        return t[~(l[t] == -np.inf).all(1)]


def loss(l, k, offsets, mask, scoring, hot=None):
    """(aux, z, counts, tokens) of each sequence; hot: the choices, held fixed."""
    B, E = len(offsets) - 1, l.shape[1]
    aux, z, counts, tokens = np.zeros(B), np.zeros(B), np.zeros((B, E)), np.zeros(B, int)
    for b in range(B):
        t = rows_of(l, offsets[b], offsets[b + 1], mask)
        tokens[b] = n = len(t)
        if n == 0:
            continue
        c = (choices(l[t], k) if hot is None else hot[t]).sum(0)
        counts[b] = c
        aux[b] = E / (k * n) * (c * scores(l[t], scoring).mean(0)).sum()
        z[b] = (lse(l[t]) ** 2).mean()
    return aux, z, counts, tokens


def gradient(l, k, offsets, mask, scoring, daux, dz):
    """(dlogits, how far a computed gradient may be off).

    In fp32 a score p is off by at most (16 + 4 r) units of 2^-23 of itself,
    where r is the spread of its row: the fast exponential is off by two units
    and 1.2 units per unit of its argument, whose own rounding adds half of
    one more; the sum, the divide and log(sigmoid) add a few.
    """
    T, E = l.shape
    out, tol = np.zeros((T, E)), np.zeros((T, E))
    for b in range(len(offsets) - 1):
        t = rows_of(l, offsets[b], offsets[b + 1], mask)
        n = len(t)
        if n == 0:
            continue
        c = choices(l[t], k).sum(0)
        g = daux[b] * E * (c - k * n / E) / (k * n * n)
        p, q, ls = scores(l[t], scoring), _softmax(l[t]), lse(l[t])
        sg = 1.0 if scoring == "softmax" else 1 / (1 + np.exp(l[t]))
        dot = (p * g).sum(1, keepdims=True)
        out[t] = p * (g - dot) * sg + (dz[b] * 2 / n * ls)[:, None] * q
        fin = np.where(np.isfinite(l[t]), l[t], np.nan)
        r = (np.nanmax(fin, 1) - np.nanmin(fin, 1))[:, None]
        e = (16 + 4 * r) * ULP
        tol[t] = 3 * e * (p * (np.abs(g) + (p * np.abs(g)).sum(1, keepdims=True)) * sg
                          + (np.abs(dz[b]) * 2 / n * (np.abs(ls) + 1))[:, None] * q)
    return out, tol + 1e-37
