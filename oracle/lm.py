"""Plain float64 oracle of dropout, embedding and softmax cross entropy (include/psgd_lm.h):
numpy, one formula after the other.  Shapes are (workers, rows, dim) for activations,
(workers, rows) for tokens and targets and (vocab, dim) for the table."""

from __future__ import annotations

import numpy as np


def philox4x32(counter, key):
    """Philox4x32-10 (Salmon et al. 2011): (n, 4) words from (n, 4) counters and two key words."""
    c = [np.asarray(counter, dtype=np.uint64)[:, i] for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def kept(shape, p, seed, step, first=0):
    """Which entries of an array of this shape (row-major) dropout keeps; the array may be the
    part of a larger one that starts at entry `first`, a multiple of 4."""
    n = int(np.prod(shape, dtype=np.int64))
    i = np.arange((n + 3) // 4, dtype=np.uint64) + np.uint64(first // 4)
    step = int(step) & 0xFFFFFFFFFFFFFFFF
    counter = np.stack([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), np.full_like(i, step & 0xFFFFFFFF),
                        np.full_like(i, step >> 32)], 1)
    words = philox4x32(counter, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n].reshape(shape)
    return words >= np.uint64(int(p * 2.0 ** 32))


def dropout(x, drop=None):
    """drop: (p, seed, step), or None."""
    x = np.asarray(x, dtype=np.float64)
    if drop is None or drop[0] == 0:
        return x
    if drop[0] == 1:
        return np.zeros_like(x)
    return np.where(kept(x.shape, *drop), x / (1 - drop[0]), 0.0)


def _valid(tokens, vocab):
    return (tokens >= 0) & (tokens < vocab)


def embed(table, tokens, drop=None):
    ok = _valid(tokens, len(table))
    rows = np.asarray(table, dtype=np.float64)[np.where(ok, tokens, 0)]
    return dropout(np.where(ok[..., None], rows, 0.0), drop)


def embed_grad(vocab, tokens, dout, drop=None):
    dy = dropout(dout, drop)
    g = np.zeros((tokens.shape[0], vocab, dy.shape[-1]))
    ok = _valid(tokens, vocab)
    for w in range(tokens.shape[0]):
        np.add.at(g[w], tokens[w][ok[w]], dy[w][ok[w]])
    return g


def scores(x, table, targets, drop=None):
    """(drop(x), zero in the rows that do not count; scores; rows that count)."""
    ok = _valid(targets, len(table))
    h = np.where(ok[..., None], dropout(x, drop), 0.0)
    return h, h @ np.asarray(table, dtype=np.float64).T, ok


def loss(x, table, targets, drop=None):
    """(losses, lse, mean)."""
    _, s, ok = scores(x, table, targets, drop)
    top = s.max(-1, keepdims=True)
    lse = top[..., 0] + np.log(np.exp(s - top).sum(-1))
    hit = np.take_along_axis(s, np.where(ok, targets, 0)[..., None], -1)[..., 0]
    losses = np.where(ok, lse - hit, 0.0)
    return losses, np.where(ok, lse, 0.0), losses.sum(1) / np.maximum(1, ok.sum(1))


def score_grad(x, table, targets, lse, scale=None, drop=None):
    """(g, drop(x)): g is the gradient of the sum over workers of scale * mean by the scores."""
    h, s, ok = scores(x, table, targets, drop)
    g = np.exp(s - np.asarray(lse, dtype=np.float64)[..., None])
    w, t = np.nonzero(ok)
    g[w, t, targets[w, t]] -= 1.0
    c = ok / np.maximum(1, ok.sum(1, keepdims=True))
    if scale is not None:
        c = c * np.asarray(scale, dtype=np.float64)[:, None]
    return np.where(ok[..., None], g * c[..., None], 0.0), h


def loss_grad(x, table, targets, lse, scale=None, drop=None):
    """(dx, table gradients (workers, vocab, dim))."""
    g, h = score_grad(x, table, targets, lse, scale, drop)
    return dropout(g @ np.asarray(table, dtype=np.float64), drop), np.swapaxes(g, 1, 2) @ h
