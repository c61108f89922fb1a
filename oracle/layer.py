"""fp64 oracle of the norms, dropout and the batched router with its balance loss, and their
backward passes.  NumPy only; written from the formulas, independent of the product's code.

Dropout's numbers are those of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
as easy as 1, 2, 3", 2011): block g of eight consecutive elements of the matrix takes the eight 16-bit
halves, low first, of the four words for counter (g, offset) and key seed.
"""
from __future__ import annotations

import numpy as np


def philox4x32(counter: np.ndarray, key, rounds: int = 10) -> np.ndarray:
    """uint32 [n, 4] of counters [n, 4] under a key of two words."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        first, second = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(second >> s32) ^ c[1] ^ np.uint64(k[0]), second & low, (first >> s32) ^ c[3] ^ np.uint64(k[1]), first & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, axis=1).astype(np.uint32)


def dropout_numbers(rows: int, d: int, seed: int, offset: int, first_row: int = 0) -> np.ndarray:
    """The 16-bit numbers of rows first_row .. first_row + rows - 1 of a matrix of d columns."""
    g = np.arange(rows * d // 8, dtype=np.uint64) + np.uint64(first_row * d // 8)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    counter = np.stack([g % np.uint64(2 ** 32), g // np.uint64(2 ** 32), np.full_like(g, offset % 2 ** 32),
                        np.full_like(g, offset // 2 ** 32)], axis=1).astype(np.uint32)
    words = philox4x32(counter, (seed % 2 ** 32, seed // 2 ** 32))
    halves = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], axis=2)
    return halves.reshape(rows, d).astype(np.int64)


def dropout_mask(rows: int, d: int, p: float, seed: int, offset: int, first_row: int = 0):
    """(kept, scale)"""
    least = int(np.rint(p * 65536.0))
    return dropout_numbers(rows, d, seed, offset, first_row) >= least, 65536.0 / (65536 - least) if least < 65536 else 0.0


def dropout(x, p: float, seed: int, offset: int, residual=None, first_row: int = 0):
    kept, scale = dropout_mask(*x.shape, p, seed, offset, first_row)
    y = np.zeros_like(x)
    y[kept] = x[kept] * scale
    return y if residual is None else residual + y


def norm(h, weight, bias, kind: str, eps: float):
    """(y, mean, rstd)"""
    mean = h.mean(axis=1) if kind == "layer" else np.zeros(h.shape[0])
    centred = h - mean[:, None]
    rstd = 1.0 / np.sqrt((centred ** 2).mean(axis=1) + eps)
    y = centred * rstd[:, None]
    if weight is not None:
        y = y * weight
    return (y if bias is None else y + bias), mean, rstd


def norm_backward(dy, h, mean, rstd, weight, dhidden, kind: str):
    """(dh, dweight, dbias), mean and rstd as given"""
    xhat = (h - (mean[:, None] if kind == "layer" else 0.0)) * rstd[:, None]
    t = dy if weight is None else dy * weight
    dh = t - xhat * (t * xhat).mean(axis=1, keepdims=True)
    if kind == "layer":
        dh = dh - t.mean(axis=1, keepdims=True)
    dh = dh * rstd[:, None]
    return (dh if dhidden is None else dh + dhidden), (dy * xhat).sum(axis=0), dy.sum(axis=0)


def softmax_rows(z):
    """Probabilities; a row without an open expert (all -inf) is all zeros."""
    p = np.zeros_like(z)
    for t, row in enumerate(z):
        open_ = row > -np.inf
        if open_.any():
            e = np.where(open_, np.exp(np.where(open_, row, 0.0) - row[open_].max()), 0.0)
            p[t] = e / e.sum()
    return p


def route(z, k: int, renorm: bool, valid=None):
    """(idx, gate, counts, prob, loss, used)"""
    rows, E = z.shape
    p = softmax_rows(z)
    idx, gate = np.full((rows, k), -1, np.int64), np.zeros((rows, k))
    counts, prob, used = np.zeros(E, np.int64), np.zeros(E), 0
    for t in range(rows):
        open_ = [e for e in range(E) if z[t, e] > -np.inf]
        if not open_ or (valid is not None and not valid[t]):
            continue
        used += 1
        prob += p[t]
        picks = sorted(open_, key=lambda e: (-z[t, e], e))[:k]
        idx[t, : len(picks)] = picks
        gate[t, : len(picks)] = p[t, picks] / p[t, picks].sum() if renorm else p[t, picks]
        counts[picks] += 1
    n = max(used, 1)
    prob /= n
    return idx, gate, counts, prob, float(E * np.sum(counts / (k * n) * prob)), used


def route_backward(z, idx, gate, counts, used: int, dgate, dloss, renorm: bool):
    rows, E = z.shape
    k = idx.shape[1]
    p = softmax_rows(z)
    n = max(used, 1)
    dz = np.zeros_like(z)
    for t in range(rows):
        if idx[t, 0] < 0:
            continue
        dp = np.zeros(E) if dloss is None else dloss * E * counts / (k * n * n)
        picks = [j for j in range(k) if 0 <= idx[t, j] < E]
        if dgate is not None:
            if renorm:
                along = sum(gate[t, j] * dgate[t, j] for j in picks)
                for j in picks:
                    dz[t, idx[t, j]] += gate[t, j] * (dgate[t, j] - along)
            else:
                for j in picks:
                    dp[idx[t, j]] += dgate[t, j]
        dz[t] += p[t] * (dp - np.sum(p[t] * dp))
    return dz
