"""fp64 oracle of the linear and gated feed-forward products and their backward passes.

y = act(x W^T + b) + residual;  y = act(x Wg^T + bg) * (x Wu^T + bu).  NumPy only; written
from the formulas, independent of the product's code.  Forward calls also return the
pre-activations; backward calls take them as given (as a forward pass stored them).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _normal_cdf(z):
    return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) if z.size else z


def _normal_pdf(z):
    return np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _logistic(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def _tanh_inner(z):
    return math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)


def act_value(z: np.ndarray, act: str) -> np.ndarray:
    if act == "none":
        return z
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "silu":
        return z * _logistic(z)
    if act == "gelu":
        return z * _normal_cdf(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_tanh_inner(z)))
    raise ValueError(act)


def act_slope(z: np.ndarray, act: str) -> np.ndarray:
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = _logistic(z)
        return s + z * s * (1.0 - s)
    if act == "gelu":
        return _normal_cdf(z) + z * _normal_pdf(z)
    if act == "gelu_tanh":
        t = np.tanh(_tanh_inner(z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * z * z)
    raise ValueError(act)


def _product(x, w, b):
    z = x @ w.T
    return z if b is None else z + b


def linear(x, w, bias=None, residual=None, act="none"):
    """(y, z)"""
    z = _product(x, w, bias)
    y = act_value(z, act)
    return (y if residual is None else y + residual), z


def linear_backward(dy, x, w, z, act="none"):
    """(dx, dw, dbias, dz); z is not read for act "none"."""
    dz = dy if act == "none" else dy * act_slope(z, act)
    return dz @ w, dz.T @ x, dz.sum(axis=0), dz


def glu(x, w_gate, w_up, bias_gate=None, bias_up=None, act="silu"):
    """(y, g, u)"""
    g, u = _product(x, w_gate, bias_gate), _product(x, w_up, bias_up)
    return act_value(g, act) * u, g, u


def glu_backward(dy, x, w_gate, w_up, g, u, act="silu"):
    """(dx, dw_gate, dw_up, dbias_gate, dbias_up, dg, du)"""
    dg = dy * u * act_slope(g, act)
    du = dy * act_value(g, act)
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x, dg.sum(axis=0), du.sum(axis=0), dg, du
