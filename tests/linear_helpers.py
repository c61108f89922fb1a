"""Inputs and error bounds of the linear and gated product tests.

Bounds, derived from the arithmetic (u = 2^-24 fp32, r = eps/2 of the storage type: 2^-8 for
bf16, 2^-24 for fp32; every operand is exact in the storage type):
  * a product of depth K: |z - z*| <= G(K) (|x| |W|^T + |b|), G(K) = 2 (K + 4) u: the usual
    bound on K products summed in fp32 in any order, doubled;
  * an activation: fp32 evaluation within A = 32 u of (1 + |z|) (1 + |act|) terms, plus its
    slope (at most 1.13 for any of them) times the error of z.  The evaluations are a handful
    of operations, each off by a few u of its operands, of size at most 1 + |z| + |z|^3 inside
    tanh, where the slope of tanh damps them: |inner| sech^2(inner) < 1;
  * slopes likewise within A (1 + |z|);
  * one rounding of the result: r |y|, and the smallest subnormal's half step.
Backward, operands dz rounded once more: dx off by (r + G(N)) |dz| |W| and the evaluation
error of dz carried through, then rounded; likewise dW and db (which sums unrounded dz).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import linear as OL

TD = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
A = 32 * U
LIP = 1.13
TINY = 2.0 ** -126


def half_step(dtype: str) -> float:
    return torch.finfo(TD[dtype]).eps / 2


def growth(depth: int) -> float:
    return 2 * (depth + 4) * U


def normal(seed: int, shape, std: float, dtype: str) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(TD[dtype])


def strided(t: torch.Tensor, device, pad: int) -> torch.Tensor:
    """The matrix on the device with `pad` more elements between its rows (NaN there)."""
    if pad == 0 or t.dim() != 2:
        return t.to(device)
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=device)
    buf[:, : t.shape[1]] = t.to(device)
    return buf[:, : t.shape[1]]


def f64(t) -> np.ndarray:
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def product_error(x, w, b) -> np.ndarray:
    mag = np.abs(x) @ np.abs(w).T
    return growth(x.shape[1]) * (mag if b is None else mag + np.abs(b))


def act_error(z, dz, act: str) -> np.ndarray:
    """Error of act(z) evaluated in fp32 on a z that is off by dz."""
    if act == "none":
        return dz
    if act == "relu":
        return dz
    return LIP * dz + A * (1 + np.abs(z)) * (1 + np.abs(OL.act_value(z, act)))


def linear_bounds(x, w, b, res, act, dtype):
    """(bound of y, bound of z)"""
    r = half_step(dtype)
    y, z = OL.linear(x, w, b, res, act)
    ez = product_error(x, w, b)
    ey = act_error(z, ez, act)
    if res is not None:
        ey = ey + U * (np.abs(y) + ey)
    return r * (np.abs(y) + ey) + ey + TINY, r * (np.abs(z) + ez) + ez + TINY


def glu_bounds(x, wg, wu, bg, bu, act, dtype):
    """(bound of y, of g, of u)"""
    r = half_step(dtype)
    y, g, u = OL.glu(x, wg, wu, bg, bu, act)
    eg, eu = product_error(x, wg, bg), product_error(x, wu, bu)
    a = OL.act_value(g, act)
    ea = act_error(g, eg, act)
    ey = ea * (np.abs(u) + eu) + np.abs(a) * eu + 2 * U * np.abs(y)
    return (r * (np.abs(y) + ey) + ey + TINY, r * (np.abs(g) + eg) + eg + TINY, r * (np.abs(u) + eu) + eu + TINY)


def slope_error(dy, z, act: str) -> np.ndarray:
    """Error of dy act'(z) evaluated in fp32 on exact dy and z."""
    if act in ("none", "relu"):
        return np.zeros_like(dy)
    return A * (1 + np.abs(z)) * np.abs(dy)


def grad_bounds(dzs, edzs, x, ws, dtype):
    """Bounds of dx, [dw], [db] given the exact dz's, their evaluation errors and operands."""
    r = half_step(dtype)
    rows, n = dzs[0].shape
    eop = [r * (np.abs(d) + e) + e for d, e in zip(dzs, edzs)]  # what the rounded operand is off by
    dx = sum(d @ w for d, w in zip(dzs, ws))
    edx = sum((e + growth(len(dzs) * n) * (np.abs(d) + e)) @ np.abs(w) for d, e, w in zip(dzs, eop, ws))
    out = [r * (np.abs(dx) + edx) + edx + TINY]
    for d, e in zip(dzs, eop):
        dw = d.T @ x
        edw = (e + growth(rows) * (np.abs(d) + e)).T @ np.abs(x)
        out.append(r * (np.abs(dw) + edw) + edw + TINY)
    for d, e in zip(dzs, edzs):
        db = d.sum(axis=0)
        edb = (e + growth(rows) * (np.abs(d) + e)).sum(axis=0)
        out.append(r * (np.abs(db) + edb) + edb + TINY)
    return out


def assert_within(got, ref: np.ndarray, bound: np.ndarray, what: str):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    err = np.abs(g - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err - bound, -np.inf)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of bounds; worst at {i}: got {g[i]!r}, "
                             f"ref {ref[i]!r}, err {err[i]:.3e}, bound {bound[i]:.3e}")
