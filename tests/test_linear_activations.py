"""Activations and slopes over a dense sweep of z, relative to the function everywhere.

The weights are an identity, so that z is x exactly (its sum has one product that is not zero)
and dx is dz.  u = 2^-24; a rounded operation is within u of its result, expf within 2 u.  A partial
result under 2^-126 may be 0: it is then off by less than 2^-126 times what it is multiplied by
afterwards (s by z, by z^2 in the gated pair; in gelu_tanh's slope f by 2 c z (1 + 3 k z^2)), and
no formula has more than four such results.  In fp32:
  * silu z / (1 + e): e 2 u, the sum, the quotient and the product 1 u each: 5 u.
  * gelu: t 3 u (product, sum, quotient), worth up to 3 times as much in t P(t) (its slope in
    ln t is at most 1 + P'(1) / P(1) = 2.97); the fit 0.5 u; Horner's sums, with products inside
    them (2 u of the partial results, at most 0.92 in all against P >= 0.107, of which the
    highest enter at t <= 1): 4 u; e 4 u with z^2's rounding made good; three products 3 u:
    20.5 u of the tail, and for z > 0 of at most half of y, with one subtraction: 24 u covers both.
  * gelu_tanh: v2 = 2 c (z + k z^3) is within 6 u of itself, hence e within 6 u v2 + 2 u, of
    which the logistic keeps the part 1 - s, with 2 u more, and the product 1 u: 6 + 7 |v2| (1 - s).
  * slopes: silu s (1 + z f), f = e s: s 4 u, f 7 u, z f 8 u, the sum and the product: 15 u of
    s (1 + |z| f).  gelu: 24 u of the tail's part, 6 u of z pdf and the sum: 24 u of
    Phi + |z| pdf.  gelu_tanh: s as above and f = e s^2, each of whose factors carries v2's
    error: 3 (7 |v2|) + 14, and 6 more for its factor: (7 + 7 |v2| (1 - s)) s + (21 + 21 |v2|) |rest|.
In bf16 the exponent is rounded as it stands: silu |z|, gelu z^2, gelu_tanh |v2| times 2 u more
at most of either of its roundings; all of it is small beside the half step 2^-8 of the result.
"""
import math

import numpy as np
import pytest
import torch

import linear_helpers as H
from weight_merge_amd import api as A

DEV = "cuda"
U = H.U
TINY = 2.0 ** -126
C, K = math.sqrt(2 / math.pi), 0.044715
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


@np.errstate(over="ignore")
def parts(z, act):
    """(s, rest): the share of z that the activation is, and the slope's other part, in 64 bits."""
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        return s, z * s / (1 + np.exp(z))
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)), z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    v2 = 2 * C * (z + K * z ** 3)
    s = 1 / (1 + np.exp(-v2))
    return s, 2 * C * z * s / (1 + np.exp(v2)) * (1 + 3 * K * z * z)


def value_units(z, act):
    """Error of the value in u of itself, in fp32."""
    if act == "silu":
        return np.full_like(z, 6.0)
    if act == "gelu":
        return np.full_like(z, 24.0)
    v2 = np.abs(2 * C * (z + K * z ** 3))
    return 6 + 7 * v2 * (1 - parts(z, act)[0])


def slope_bound(z, act):
    s, rest = parts(z, act)
    if act == "silu":
        return 15 * U * (s + np.abs(rest))
    if act == "gelu":
        return 24 * U * (s + np.abs(rest))
    v2 = np.abs(2 * C * (z + K * z ** 3))
    return U * ((7 + 7 * v2 * (1 - s)) * s + (21 + 21 * v2) * np.abs(rest))


def rough(z, act):
    """What bf16's evaluation may be off by more, relative to s and to the slope's other part."""
    v2 = np.abs(2 * C * (z + K * z ** 3))
    w = {"silu": np.abs(z), "gelu": z * z, "gelu_tanh": v2}[act]
    return 4 * U * (16 + w * (1 - parts(z, act)[0])), 4 * U * (16 + w)


def sweep(rows, cols, dtype, lo):
    n = rows * cols
    z = torch.cat([torch.linspace(-14, 14, n - n // 4, dtype=torch.float64),
                   torch.linspace(lo, -14, n // 8, dtype=torch.float64),
                   torch.linspace(14, 3e4, n // 4 - n // 8, dtype=torch.float64)])
    return z.to(H.TD[dtype]).reshape(rows, cols)


def check(got, ref, bound, factor, z, what):
    """factor: what a partial result under 2^-126 is multiplied by."""
    err = np.abs(H.f64(got) - ref)
    bad = ~(err <= bound + 4 * TINY * factor)
    i = np.unravel_index(np.argmax(np.where(bad, err / (bound + TINY), -1)), err.shape)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, z {z[i]!r} got {H.f64(got)[i]!r} ref {ref[i]!r} " \
                          f"err {err[i]:.3e} bound {bound[i]:.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh"))
@pytest.mark.parametrize("rows, cols", ((1, 8192), (24, 1024), (300, 136)))
def test_sweep(rows, cols, act, dtype):
    x = sweep(rows, cols, dtype, -85.0)
    z, eye = H.f64(x), torch.eye(cols, dtype=H.TD[dtype], device=DEV)
    s, rest = parts(z, act)
    y, r = z * s, H.half_step(dtype) if dtype == "bf16" else 0.0
    f = 1 + np.abs(z)
    fs = f + np.abs(2 * C * z * (1 + 3 * K * z * z)) if act == "gelu_tanh" else f
    more, more_rest = rough(z, act) if dtype == "bf16" else (0.0, 0.0)
    by = (value_units(z, act) * U + more) * np.abs(y)
    by = by + r * (np.abs(y) + by)
    check(A.ada_linear(x.to(DEV), eye, act=act), y, by, f, z, "linear")
    b2 = (value_units(z, act) * U + U + more) * np.abs(y * z)  # y z: one product more
    check(A.ada_glu(x.to(DEV), eye, eye, act=act), y * z, b2 + r * (np.abs(y * z) + b2), f * f, z, "glu")

    ones = torch.ones((rows, cols), dtype=H.TD[dtype], device=DEV)
    slope = s + rest
    bs = slope_bound(z, act) + more * s + more_rest * np.abs(rest)
    bs = bs + 2 * r * (np.abs(slope) + bs)  # dz and dx
    got = A.ada_linear_backward(ones, ones, eye, pre=x.to(DEV), act=act, want_dw=False)[0]
    check(got, slope, bs, fs, z, "slope")
    # d_gate = dy u slope and d_up = dy act, the other projection's weights being zeros
    zero = torch.zeros_like(eye)
    dx = A.ada_glu_backward(ones, ones, eye, zero, x.to(DEV), ones, act=act, want_dw=False)[0]
    check(dx, slope, bs + U * np.abs(slope), fs, z, "dg")
    dx = A.ada_glu_backward(ones, ones, zero, eye, x.to(DEV), ones, act=act, want_dw=False)[0]
    check(dx, y, by + 2 * r * np.abs(y) + U * np.abs(y), f, z, "du")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("act", ("none", "relu"))
def test_exact_activations(act, dtype):
    x = sweep(70, 136, dtype, -85.0).to(DEV)
    eye = torch.eye(136, dtype=H.TD[dtype], device=DEV)
    want = x if act == "none" else x.clamp(min=0)
    assert torch.equal(A.ada_linear(x, eye, act=act), want)
    ones = torch.ones_like(x)
    slope = ones if act == "none" else (x > 0).to(x.dtype)
    assert torch.equal(A.ada_linear_backward(ones, ones, eye, pre=x, act=act, want_dw=False)[0], slope)
