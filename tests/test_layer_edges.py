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


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("E, k", ((5, 3), (12, 3), (30, 7), (64, 9)))
def test_a_pick_out_of_range_has_no_part_in_its_row_s_gradient(E, k, renorm):
    """Whatever its gate and its gate's gradient: neither at an expert nor in the sum over the row's picks."""
    rows = 40
    z = H.logits(1, rows, E, "fp32").to(DEV)
    out = A.ada_route(z, k, renorm=renorm)
    idx, gate = out.idx.clone(), out.gate.clone()
    idx[2, 1], idx[3, k - 1], idx[4, 1], idx[5, 0], idx[6, 1] = 1 << 30, E, -7, E + 1, -1
    gate[7, 2], idx[7, 2] = float("nan"), 2 ** 31 - 1
    g = H.normal(2, (rows, k), 1.0, "fp32").to(DEV)
    got = A.ada_route_backward(z, out._replace(idx=idx, gate=gate), dgate=g, renorm=renorm)
    n, ni, ng, nz = H.f64(g), idx.cpu().numpy(), H.f64(gate), H.f64(z)
    ref = OL.route_backward(nz, ni, ng, None, rows, n, None, renorm)
    inside = (ni >= 0) & (ni < E)
    p, rel = OL.softmax_rows(nz), H.probability_bound(nz)
    part = np.where(inside, np.abs(ng) * (np.abs(n) + np.sum(np.where(inside, np.abs(ng * n), 0.0), axis=1, keepdims=True))
                    if renorm else np.abs(n), 0.0)
    mag = np.zeros((rows, E))
    np.add.at(mag, (np.arange(rows)[:, None], np.where(inside, ni, 0)), part)
    if not renorm:
        mag = p * (mag + np.sum(p * mag, axis=1, keepdims=True))
    # as for picks in range: the probabilities enter twice, sums are over k + 8 + 3 terms
    H.assert_within(got, ref, H.rounded((2 * rel + (k + 16) * H.U) * mag, ref, "fp32"), "dlogits")
