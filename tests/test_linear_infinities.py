"""Activations and slopes at infinities and NaN, forward and backward, in every kernel that
evaluates them.

At +inf the activations are +inf (the limit, and what their formulas give).  At -inf relu is
0, the identity -inf, and the others are the formula's -inf * 0 = NaN.  The slopes take their
limits: 1 at +inf, 0 at -inf.  NaN stays NaN, except that relu's slope is that of a comparison.
"""
import pytest
import torch

import linear_helpers as H
from weight_merge_amd import api as A

DEV = "cuda"
INF, NAN = float("inf"), float("nan")
Z = [INF, -INF, NAN, 2.0]
VALUES = {"none": [INF, -INF, NAN], "relu": [INF, 0.0, NAN], "silu": [INF, NAN, NAN], "gelu": [INF, NAN, NAN],
          "gelu_tanh": [INF, NAN, NAN]}
SLOPES = {"none": [1.0, 1.0, 1.0], "relu": [1.0, 0.0, 0.0], "silu": [1.0, 0.0, NAN], "gelu": [1.0, 0.0, NAN],
          "gelu_tanh": [1.0, 0.0, NAN]}


def same(got: torch.Tensor, want: list) -> bool:
    """Row i of got holds want[i] throughout."""
    ref = torch.tensor(want, dtype=got.dtype, device=got.device)[:, None].expand(-1, got.shape[1])
    return bool(((got[: len(want)] == ref) | (got[: len(want)].isnan() & ref.isnan())).all())


def rows_of(values, rows, cols, dtype):
    """Row i holds values[i], the rows behind them 2."""
    t = torch.full((rows, cols), 2.0, dtype=H.TD[dtype], device=DEV)
    t[: len(values)] = torch.tensor(values, dtype=H.TD[dtype], device=DEV)[: rows, None]
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("act", SLOPES)
@pytest.mark.parametrize("rows", (4, 40, 300))
def test_activations_at_infinities(rows, act, dtype):
    """z = x, the weight's first column being ones and its others zeros, and x zero but for its
    first column."""
    x = torch.zeros((rows, 16), dtype=H.TD[dtype], device=DEV)
    x[:, 0] = rows_of(Z, rows, 1, dtype)[:, 0]
    w = torch.zeros((72, 16), dtype=H.TD[dtype], device=DEV)
    w[:, 0] = 1
    assert same(A.ada_linear(x, w, act=act), VALUES[act])
    assert same(A.ada_glu(x, w, w, act=act), [a * z for a, z in zip(VALUES[act], Z)])


@pytest.mark.gpu
@pytest.mark.parametrize("act", SLOPES)
@pytest.mark.parametrize("row", range(3))
def test_one_row_at_infinities(row, act):
    """One row, whose kernel is another."""
    for dtype in ("fp32", "bf16"):
        x = torch.zeros((1, 16), dtype=H.TD[dtype], device=DEV)
        x[0, 0] = Z[row]
        w = torch.zeros((72, 16), dtype=H.TD[dtype], device=DEV)
        w[:, 0] = 1
        assert same(A.ada_linear(x, w, act=act), VALUES[act][row: row + 1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("act", SLOPES)
@pytest.mark.parametrize("rows", (4, 40, 300))
def test_slopes_at_infinities(rows, act, dtype):
    """dbias of single rows is their dz; dx with an identity for the weights is dz as well."""
    pre = rows_of(Z, rows, 72, dtype)
    eye = torch.eye(72, dtype=H.TD[dtype], device=DEV)
    x = torch.ones((rows, 72), dtype=H.TD[dtype], device=DEV)
    for i in range(3):
        dy = torch.ones((1, 72), dtype=H.TD[dtype], device=DEV)
        db = A.ada_linear_backward(dy, x[:1], eye, pre=pre[i: i + 1], act=act, want_dx=False, want_dw=False,
                                   want_dbias=True)[2]
        assert same(db[None], SLOPES[act][i: i + 1]), i
        one = torch.full_like(dy, 3.0)
        dbg, dbu = A.ada_glu_backward(dy, x[:1], eye, eye, pre[i: i + 1], one, act=act, want_dx=False, want_dw=False,
                                      want_dbias=True)[3:]
        assert same(dbg[None], [3 * SLOPES[act][i]]) and same(dbu[None], VALUES[act][i: i + 1]), i
    finite = [s for s in range(3) if SLOPES[act][s] == SLOPES[act][s]]
    pre[: 3] = rows_of([Z[s] for s in finite] + [2.0] * (3 - len(finite)), 3, 72, dtype)
    dx = A.ada_linear_backward(torch.ones((rows, 72), dtype=H.TD[dtype], device=DEV), x, eye, pre=pre, act=act)[0]
    assert same(dx, [SLOPES[act][s] for s in finite])
