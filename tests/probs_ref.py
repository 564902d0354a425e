"""Plain 64-bit forms of the way from logits to probabilities and of the token
history's commit.  CPU only, numpy float64, one row and one token at a time."""
from __future__ import annotations

import numpy as np

from attn_ref import path_of

BIG = float(np.finfo(np.float32).max)


def adjusted(logits, counts, known, rep, freq, pres, bias, allowed):
    """One row's x after penalties, biases and the mask."""
    x = logits.astype(np.float64).copy()
    for y in np.nonzero(known | (counts > 0))[0]:
        v = x[y] / rep if x[y] > 0 else x[y] * rep
        v = v - freq * counts[y] - (pres if counts[y] > 0 else 0.0)
        x[y] = min(max(v, -BIG), BIG) if np.isfinite(x[y]) else v
    for y, b in bias:
        x[y] += b
    if allowed is not None:
        x = np.where(allowed, x, -np.inf)
    return x


def probabilities(x, temperature):
    if np.isnan(x).any():
        return np.full(len(x), np.nan)
    if not (x > -np.inf).any():
        return np.zeros(len(x))
    if not temperature > 0:
        p = np.zeros(len(x))
        p[int(np.argmax(x))] = 1.0
        return p
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(np.where(x == -np.inf, -np.inf, (x - x.max()) / temperature))
    return e / e.sum()


def history_of(h):
    """(counts, prompt) of a row of 16-bit history."""
    h = h.astype(np.int64) & 0xffff
    return h & 0x7fff, h >= 0x8000


def row_counts(history_row, tokens, par, i, V):
    counts, prompt = history_of(history_row[:V]) if history_row is not None else (np.zeros(V, np.int64), np.zeros(V, bool))
    counts = counts.copy()
    for x in path_of(par, i):
        counts[tokens[x]] = min(counts[tokens[x]] + 1, 0x7fff)
    return counts, prompt


def allowed_of(words, V):
    bits = np.unpackbits(np.ascontiguousarray(words).view(np.uint8), bitorder="little")
    return bits[:V].astype(bool)
