"""Infinite weights and inputs: a sum that holds one infinity is that infinity, in every kernel
and wherever along the contraction it lies.  What pads a row or repeats an element of it may
not meet the infinity as a zero factor."""
import pytest
import torch

from weight_merge_amd import api as A
import linear_helpers as H

DEV = "cuda"
INF = float("inf")


def ones(rows, cols, dtype):
    return torch.ones((rows, cols), dtype=H.TD[dtype], device=DEV)


def places(k):
    return sorted({0, 3, 7, 8 % k, k // 2, k - 8, k - 1})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("d_in", (8, 520, 2048, 4104, 11008))
@pytest.mark.parametrize("rows", (1, 2, 33, 70))
def test_an_infinite_weight(rows, d_in, dtype):
    """Weight row i holds an infinity of alternating sign at place i; x is ones.  One row: depths
    on and off the multiples of its kernel's batch of loads."""
    at = places(d_in)
    x, w = ones(rows, d_in, dtype), ones(24, d_in, dtype)
    want = torch.full((24,), float(d_in), dtype=H.TD[dtype], device=DEV)
    for i, k in enumerate(at):
        w[i, k] = want[i] = INF if i % 2 else -INF
    assert torch.equal(A.ada_linear(x, w), want.expand(rows, -1))
    finite = ones(24, d_in, dtype) / d_in
    finite[:, 1:] = 0
    finite[:, 0] = 1  # the other projection is 1
    assert torch.equal(A.ada_glu(x, w, finite, act="none"), want.expand(rows, -1))
    assert torch.equal(A.ada_glu(x, finite, w, act="none"), want.expand(rows, -1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("d_in", (8, 520, 4104, 11008))
@pytest.mark.parametrize("rows", (1, 2, 33, 70))
def test_an_infinite_input(rows, d_in, dtype):
    """x's last row holds the infinity."""
    for k in places(d_in):
        x, w = ones(rows, d_in, dtype), ones(24, d_in, dtype)
        x[rows - 1, k] = -INF
        want = torch.full((rows, 24), float(d_in), dtype=H.TD[dtype], device=DEV)
        want[rows - 1] = -INF
        assert torch.equal(A.ada_linear(x, w), want), k
        want[: rows - 1] = float(d_in) ** 2
        want[rows - 1] = INF
        assert torch.equal(A.ada_glu(x, w, w, act="none"), want), k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("d_out, d_in", ((24, 520), (4104, 1032)))
@pytest.mark.parametrize("rows", (1, 2, 33, 70))
def test_infinities_in_the_gradients(rows, d_out, d_in, dtype):
    """An infinite weight in its column of dx, an infinite input in its column of dw; the
    contractions are d_out and rows long."""
    for n in sorted({0, 7, 8, d_out // 2, d_out - 1}):
        x, w, dy = ones(rows, d_in, dtype), ones(d_out, d_in, dtype), ones(rows, d_out, dtype)
        w[n, 5], x[rows - 1, 11] = -INF, INF
        dx, dw, _ = A.ada_linear_backward(dy, x, w)
        want_dx = torch.full_like(x, float(d_out))
        want_dx[:, 5] = -INF
        want_dw = torch.full_like(w, float(rows))
        want_dw[:, 11] = INF
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw), n
