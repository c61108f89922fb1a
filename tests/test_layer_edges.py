"""Norm, dropout and router calls at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

import layer_helpers as H
from oracle import layer as OL
from weight_merge_amd import api as A

DEV = "cuda"
EPS = 1e-5


def many_rows(rows, d, dtype):
    """A block of normal rows over and over, each row 1 to 1.9 times as large: rows a power of two apart differ."""
    block = H.normal(1, (4099, d), 1.0, dtype).to(DEV)
    x = torch.empty((rows, d), dtype=H.TD[dtype], device=DEV)
    for first in range(0, rows, len(block)):
        n = min(len(block), rows - first)
        size = 1 + 0.1 * ((first // len(block)) % 10)
        torch.mul(block[:n], size, out=x[first:first + n])
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ("rms", "layer"))
@pytest.mark.parametrize("d, dtype", ((1544, "fp32"), (2056, "bf16"), (4104, "bf16"), (8200, "bf16")))
def test_rows_that_a_workgroup_takes_second(d, dtype, kind):
    """Several waves share a row and a workgroup takes two: the same as calls in which none does, bit for bit, and
    the oracle's on the rows at the seam."""
    most = 1 << 20
    rows = most + 6000
    x = many_rows(rows, d, dtype)
    w = (1 + H.normal(2, (d,), 0.1, "fp32")).to(H.TD[dtype]).to(DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    A.ada_norm(x, w, kind=kind, eps=EPS, y=y, stats=(None, rstd))
    part_rstd = torch.empty(most, device=DEV)
    for first, n in ((0, most), (most, rows - most)):
        part = A.ada_norm(x[first:first + n], w, kind=kind, eps=EPS, stats=(None, part_rstd[:n]))
        assert torch.equal(rstd[first:first + n], part_rstd[:n]), first
        assert torch.equal(y[first:first + n], part), first
        del part
    for first in (0, most - 2, rows - 2):
        h = H.f64(x[first:first + 2])
        ref = OL.norm(h, H.f64(w), None, kind, EPS)[0]
        bound = H.norm_bounds(h, np.zeros_like(h), H.f64(w), None, kind, EPS, dtype)[0]
        H.assert_within(y[first:first + 2], ref, bound, f"rows {first}")
