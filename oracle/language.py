"""fp64 oracle of the language-model operators: the embedding, the gated
recurrence, activation checkpoints in 8 bits, cross-entropy, and their
gradients.  Everything is evaluated in fp64, row after row, and nothing is
rounded but the e4m3 codes."""

from __future__ import annotations

import numpy as np

from . import feedforward as F

BLOCK = 32
MIN_EXP, MAX_EXP = -116, 120


def embedding(tokens, table, scale=1.0):
    tokens, table = np.asarray(tokens), np.asarray(table, np.float64)
    known = (tokens >= 0) & (tokens < len(table))
    return np.where(known[:, None], table[np.where(known, tokens, 0)] * scale, 0.0)


def embedding_backward(tokens, dy, vocab, scale=1.0):
    out = np.zeros((vocab, np.shape(dy)[1]))
    for t, row in zip(np.asarray(tokens), np.asarray(dy, np.float64)):
        if 0 <= t < vocab:
            out[t] += row * scale
    return out


def equal_starts(rows, sequences):
    return np.arange(sequences + 1) * (rows // sequences)


def recurrence(x, gate, starts, h0=None):
    """(y, hT, h before each row); rows outside of the sequences are NaN."""
    x, c = np.asarray(x, np.float64), F.sigmoid(gate)
    y, before = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    hT = np.zeros((len(starts) - 1, x.shape[1])) if h0 is None else np.array(h0, np.float64)
    for s in range(len(starts) - 1):
        h = hT[s].copy()
        for t in range(starts[s], starts[s + 1]):
            before[t] = h
            h = h + c[t] * (x[t] - h)
            y[t] = h
        hT[s] = h
    return y, hT, before


def recurrence_backward(dy, x, gate, starts, h0=None, dhT=None):
    """(dx, dgate, dh0, the gradient of each row's h); rows outside of the
    sequences are NaN."""
    x, dy, gate = np.asarray(x, np.float64), np.asarray(dy, np.float64), np.asarray(gate, np.float64)
    c, keep = F.sigmoid(gate), F.sigmoid(-gate)
    before = recurrence(x, gate, starts, h0)[2]
    lam = np.full(x.shape, np.nan)
    dh0 = np.zeros((len(starts) - 1, x.shape[1])) if dhT is None else np.array(dhT, np.float64)
    for s in range(len(starts) - 1):
        g = dh0[s].copy()
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            lam[t] = dy[t] + g
            g = keep[t] * lam[t]
        dh0[s] = g
    return c * lam, c * keep * lam * (x - before), dh0, lam


def checkpoint_save(x):
    """(q, exponents): values of e4m3 codes, and e of each block's 2^e."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    q, e = np.empty(x.shape), np.empty((rows, blocks), int)
    for b in range(blocks):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.max(np.where(np.isfinite(part), np.abs(part), 0.0), axis=1)
        amax = np.maximum(amax, 2.0 ** -140)
        k = np.ceil(np.log2(amax / 448.0))
        k += amax > 448.0 * np.exp2(k)              # log2 may be off by a rounding
        k -= amax <= 448.0 * np.exp2(k - 1)
        e[:, b] = np.maximum(k, MIN_EXP).astype(int)
        v = np.where(np.isfinite(part), part, np.nan) * np.exp2(-e[:, b, None].astype(float))
        v = np.where(e[:, b, None] == MAX_EXP, np.clip(v, -240.0, 240.0), v)       # 256 * 2^120 is no finite number
        q[:, b * BLOCK:(b + 1) * BLOCK] = F.e4m3_rne(v)
    return q, e


def checkpoint_restore(q, e):
    q = np.asarray(q, np.float64)
    return q * np.exp2(np.repeat(np.asarray(e, np.float64), BLOCK, axis=1)[:, :q.shape[1]])


def cross_entropy(logits, labels, scale=1.0, weight=None):
    """(loss, lse, dlogits)."""
    x, labels = np.asarray(logits, np.float64), np.asarray(labels)
    rows, cols = x.shape
    known = (labels >= 0) & (labels < cols)
    at = np.where(known, labels, 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.max(x, axis=1)
        anchor = np.where(top == -np.inf, 0.0, top)
        p = np.exp(x - anchor[:, None])
        total = p.sum(axis=1)
        lse = np.log(total) + anchor
        loss = np.where(known, np.where(total == 0, np.inf, lse - x[np.arange(rows), at]), 0.0)
        g = np.where(total[:, None] == 0, 0.0, p / total[:, None])
    g[np.arange(rows), at] -= total != 0
    w = np.full(rows, scale, np.float64) if weight is None else scale * np.asarray(weight, np.float64)
    return loss, lse, np.where(known[:, None], g * w[:, None], 0.0)
