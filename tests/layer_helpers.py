"""Inputs and error bounds of the norm, dropout and router tests.

Bounds, derived from the arithmetic (u = 2^-24; r = eps/2 of the storage type: 2^-8 bf16, 2^-24
fp32; inputs are exact in the storage type):
  * a sum over a row: at most 32 terms one after the other on a lane, then 6 steps across lanes
    and 16 across waves: off by at most DEPTH u of the sum of magnitudes, DEPTH = 64;
  * a sum over rows: rows + 64 additions at the most, in whatever order: (rows + 64) u of the magnitudes;
  * h = residual + x s: 2 u (|x s| + |h|), exact without dropout and residual;
  * xhat: the error of h, of the mean, and xhat times the error of rstd, which is half the
    relative error of the variance and 3 u for the division and the square root;
  * exp(z - m): (|z - m| + 4) u of the value (the argument's rounding, the function, its product);
  * one rounding of a result: r times the value, and the smallest normal number for what underflows.
Bounds of first order, doubled for what they leave out.
"""
from __future__ import annotations

import numpy as np
import torch

from linear_helpers import TD, TINY, U, assert_within, f64, half_step, normal, strided  # noqa: F401
from oracle import layer as OL

DEPTH = 64


def rounded(err, value, dtype: str):
    """The bound behind the rounding to the storage type of a value that is off by err."""
    r = half_step(dtype)
    return 2 * err * (1 + r) + r * np.abs(value) + TINY


def dropout_bound(y, dropped, residual, dtype: str):
    err = U * np.abs(dropped)
    if residual is not None:
        err = err + U * (np.abs(y) + err)
    return rounded(err, y, dtype)


def mean_rows(v):
    return v.mean(axis=1, keepdims=True)


def norm_bounds(h, eh, w, b, kind: str, eps: float, dtype: str):
    """(y, mean, rstd bounds) for the h of the oracle, off by eh where the kernel forms it."""
    _, mean, rstd = OL.norm(h, w, b, kind, eps)
    mean, rstd = mean[:, None], rstd[:, None]
    a = h - mean
    em = np.zeros_like(mean) if kind == "rms" else mean_rows(eh) + (DEPTH + 2) * U * mean_rows(np.abs(h))
    ea = eh + em + 2 * U * (np.abs(a) + em)
    evar = mean_rows(2 * np.abs(a) * ea + ea * ea) + (DEPTH + 4) * U * mean_rows(a * a)
    rel = 0.5 * evar * rstd * rstd + 3 * U
    ex = ea * rstd + np.abs(a) * rstd * rel + 2 * U * np.abs(a) * rstd
    weight = np.ones(h.shape[1]) if w is None else w
    y = a * rstd * weight
    ey = ex * np.abs(weight) + 2 * U * np.abs(y)
    if b is not None:
        y = y + b
        ey = ey + U * (np.abs(y) + ey)
    return rounded(ey, y, dtype), 2 * em[:, 0] + U * np.abs(mean[:, 0]) + TINY, 2 * (rel * rstd)[:, 0] + TINY


def norm_grad_bounds(dy, h, mean, rstd, w, dhidden, kind: str):
    """(error of dh, of dw, of db) before the roundings to the storage type."""
    weight = np.ones(h.shape[1]) if w is None else w
    m, s = (mean if kind == "layer" else 0 * mean)[:, None], rstd[:, None]
    xhat, t = (h - m) * s, dy * weight
    ex, et = 3 * U * np.abs(xhat), U * np.abs(t)
    e1 = (DEPTH + 3) * U * mean_rows(np.abs(t)) if kind == "layer" else 0.0
    c1 = mean_rows(t) if kind == "layer" else 0.0
    c2 = mean_rows(t * xhat)
    e2 = mean_rows(et * np.abs(xhat) + np.abs(t) * ex) + (DEPTH + 3) * U * mean_rows(np.abs(t * xhat))
    inner = et + e1 + np.abs(xhat) * e2 + np.abs(c2) * ex + 3 * U * (np.abs(t) + np.abs(c1) + np.abs(xhat * c2))
    dh = s * (t - c1 - xhat * c2)
    eh = s * inner + 2 * U * np.abs(dh)
    if dhidden is not None:
        eh = eh + U * (np.abs(dh + dhidden) + eh)
    rows = h.shape[0]
    ew = (np.abs(dy) * ex + (rows + 64) * U * np.abs(dy * xhat)).sum(axis=0)
    return eh, ew, (rows + 64) * U * np.abs(dy).sum(axis=0)


def probability_bound(z):
    """Relative error of a row's probabilities and of its gates (both share it, [rows, 1])."""
    spread = np.array([np.ptp(row[row > -np.inf]) if (row > -np.inf).any() else 0.0 for row in z])
    return (2 * (2 * (spread + 4) + DEPTH) * U)[:, None]


def logits(seed: int, rows: int, E: int, dtype: str, closed: float = 0.0, ties: bool = False) -> torch.Tensor:
    """Router logits; some experts closed to some rows, the first three rows' all, all but one and all but two."""
    z = normal(seed, (rows, E), 2.0, "fp32")
    if ties:
        z = torch.round(z)
    if closed:
        g = torch.Generator().manual_seed(seed + 1)
        z[torch.rand((rows, E), generator=g) < closed] = -float("inf")
        for t, left in enumerate((0, 1, 2)):
            if t < rows:
                z[t, left:] = -float("inf")
    return z.to(TD[dtype])
