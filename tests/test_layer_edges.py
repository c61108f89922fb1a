"""Norm, dropout and router calls at the edges of what their documentation allows."""
import types

import numpy as np
import pytest
import torch

import layer_helpers as H
from oracle import layer as OL
from weight_merge_amd import _lib
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


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: runs where no GPU is visible")


@no_gpu
@pytest.mark.parametrize("dt, rows, d", ((_lib.ADA_BF16, 5000, 64), (_lib.ADA_F32, 4096, 8192)))
def test_norm_backward_of_rows_alone_needs_no_workspace(dt, rows, d):
    """Only the sums over rows go through it."""
    lib = _lib.load()
    need = lib.ada_norm_backward_workspace(rows, d, dt)
    assert need > 0
    at = {n: (i + 1) << 36 for i, n in enumerate(("dy", "hidden", "dhidden", "weight", "mean", "rstd", "dx", "dresidual",
                                                  "dweight", "dbias"))}
    lds = dict.fromkeys(("ld_dy", "ld_hidden", "ld_dhidden", "ld_dx", "ld_dresidual"), d)

    def call(ws, nbytes, **kw):
        return lib.ada_norm_backward(_lib.AdaNormGradArgs(**{**at, **lds, "rows": rows, "d": d, **kw}), dt, ws, nbytes, None)

    # with no GPU a call that passes the checks ends at its first HIP call
    assert call(None, 0, dweight=None, dbias=None) == _lib.ADA_EHIP
    assert call(8, 0, dweight=None, dbias=None) == _lib.ADA_EALIGN
    for one in ("dweight", "dbias"):
        assert call(None, 0, **{one: None}) == _lib.ADA_EINVAL
        assert call(1 << 46, need - 1, **{one: None}) == _lib.ADA_ESHAPE
        assert call(1 << 46, need, **{one: None}) == _lib.ADA_EHIP


def test_norm_backward_allocates_no_workspace_for_rows_alone(monkeypatch):
    needs = []
    monkeypatch.setattr(A, "_current", lambda dev: None)
    monkeypatch.setattr(A, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(A, "_workspace", lambda need, ws, dev: needs.append(need) or (None, 0, None))
    monkeypatch.setattr(A, "_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(A._lib, "load", lambda: types.SimpleNamespace(ada_norm_backward=lambda *a: 0))
    x, stats = torch.zeros(2000, 24), (torch.zeros(2000), torch.zeros(2000))
    A.ada_norm_backward(x, x, stats, want_dweight=False)
    A.ada_norm_backward(x, x, stats)
    A.ada_norm_backward(x, x, stats, want_dweight=False, want_dbias=True)
    A.ada_norm_backward(x, x, stats, want_dweight=False, dbias=torch.zeros(24))
    assert needs == [0, 4096, 4096, 4096]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows, d", ((900, 264), (2047, 4096)))
def test_gradients_of_rows_alone_are_those_of_the_whole_call(rows, d, dtype):
    dy, h, dhidden = (H.normal(i, (rows, d), 1.0, dtype).to(DEV) for i in (1, 2, 3))
    stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in OL.norm(H.f64(h), None, None, "layer", EPS)[1:]]
    kw = dict(dhidden=dhidden, p=0.1, seed=3, want_dresidual=True)
    dx, dr, dw, _ = A.ada_norm_backward(dy, h, stats, **kw)
    got = A.ada_norm_backward(dy, h, stats, want_dweight=False, **kw)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dr) and got[2] is None


def test_a_balance_needs_somewhere_to_go():
    """A Routing of a call without balance is not written to by one that is asked for it."""
    z = torch.zeros(4, 6)
    bare = (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), None, None, None, None)
    full = (*bare[:2], torch.zeros(6, dtype=torch.int32), torch.zeros(6), torch.zeros(1), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="no tensors for the balance"):
        A.ada_route(z, 2, out=bare)
    with pytest.raises(ValueError, match="no tensors for the balance"):
        A.ada_route(z, 2, out=A.Routing(*bare), balance=True)
    for i in range(2, 6):
        with pytest.raises(ValueError, match="no tensors for the balance"):
            A.ada_route(z, 2, out=full[:i] + (None,) + full[i + 1:])
    for kw in (dict(out=full), dict(out=bare, balance=False), dict(out=full, balance=False)):
        with pytest.raises(ValueError, match="must be on the device"):  # the next thing that is wrong
            A.ada_route(z, 2, **kw)


def test_seeds_and_offsets_are_whole_numbers_of_any_kind():
    """Python's and NumPy's alike, modulo 2^64."""
    m = 2 ** 64
    for v in (0, 7, -1, 2 ** 31 - 1, -2 ** 31):
        for kind in (int, np.int64, np.int32) + ((np.uint64, np.uint32) if v >= 0 else ()):
            assert A._drop(0.1, kind(v), kind(v), -1) == (0.1, v % m, v % m, None)
    assert A._drop(0.1, np.uint64(m - 1), np.int64(-2 ** 63), -1) == (0.1, m - 1, 2 ** 63, None)
    state = torch.zeros(2, dtype=torch.int64)
    assert A._drop(0.1, state, np.int64(-3), -1) == (0.1, 0, m - 3, state.data_ptr())
    for bad in (1.0, "1", np.float64(2)):
        with pytest.raises(TypeError):
            A._drop(0.1, bad, 0, -1)
        with pytest.raises(TypeError):
            A._drop(0.1, 1, bad, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("d", (8, 264, 4104, 16392))
def test_rows_whose_sums_pass_the_type_s_range(d, dtype):
    """Finite rows: squares that overflow are a deviation without end, rstd 0; a sum that does leaves no mean. The rows
    beside them are as without them."""
    low = torch.finfo(H.TD[dtype]).min
    x = H.normal(1, (6, d), 1.0, dtype)
    sign = torch.where(torch.arange(d) % 2 == 0, 1.0, -1.0).to(H.TD[dtype])
    ref = {kind: A.ada_norm(x.to(DEV), kind=kind) for kind in ("layer", "rms")}
    x[1], x[3], x[5] = 2.0 ** 65 * sign, low, 2.0 ** 65
    x, w, b = x.to(DEV), H.normal(2, (d,), 1.0, dtype).to(DEV), H.normal(3, (d,), 1.0, dtype).to(DEV)
    for kind in ("layer", "rms"):
        rstd, mean = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
        y = A.ada_norm(x, kind=kind, eps=EPS, stats=(mean, rstd))
        assert torch.equal(y[::2], ref[kind][::2])
        affine = A.ada_norm(x, w, bias=b, kind=kind, eps=EPS)
        assert (y[1] == 0).all() and rstd[1] == 0 and torch.equal(affine[1], b)
        if kind == "rms":
            assert (y[3] == 0).all() and rstd[3] == 0 and torch.equal(affine[3], b)
            assert (y[5] == 0).all() and rstd[5] == 0
        else:
            assert y[3].isnan().all() and rstd[3].isnan()
            assert (y[5] == 0).all() and mean[5] == 2.0 ** 65  # a constant row: powers of two are exact


@pytest.mark.gpu
@pytest.mark.parametrize("rows, d, chains", ((1 << 18, 8200, 40), (1 << 18, 8192, 256), (1 << 20, 2056, 768), (1 << 22, 264, 4096)))
def test_sums_over_many_rows_keep_what_is_small(rows, d, chains):
    """dw and db in fp32 of ones in the first rows, one for each lane that sums a column, and 2^-25 in all others, each
    of which alone vanishes beside a one. A lane puts its sum aside every 256 rows: in the run that holds the one 255 of the
    small ones may be lost, 2^-17 in all, later runs are exact (multiples of 2^-25 below 2^-16). The lanes' sums meet in
    fewer than 64 roundings one after the other, 2^-18 of the total."""
    dy = torch.full((rows, d), 2.0 ** -25, device=DEV)
    dy[:chains] = 1.0
    h = torch.ones((rows, d), device=DEV)
    stats = (None, torch.ones(rows, device=DEV))
    _, _, dw, db = A.ada_norm_backward(dy, h, stats, kind="rms", want_dx=False, want_dbias=True)
    small = (rows - chains) * 2.0 ** -25
    true = chains + small
    bound = chains * 2.0 ** -17 + true * 2.0 ** -18
    assert small > 2 * bound
    for name, got in (("dw", dw), ("db", db)):
        H.assert_within(got, np.full(d, true), np.full(d, bound), name)


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("E, k", ((5, 3), (16, 4), (64, 9)))
def test_an_expert_that_a_row_names_twice_gets_both_parts(E, k, renorm):
    """In slots of one lane and of two; equal calls give equal bits."""
    rows = 300
    z = H.logits(3, rows, E, "fp32").to(DEV)
    out = A.ada_route(z, k, renorm=renorm)
    idx = out.idx.clone()
    idx[::2, 1], idx[1::2, k - 1] = idx[::2, 0], idx[1::2, 0]
    g = H.normal(4, (rows, k), 1.0, "fp32").to(DEV)
    got = [A.ada_route_backward(z, out._replace(idx=idx), dgate=g, renorm=renorm) for _ in range(4)]
    assert all(torch.equal(v, got[0]) for v in got)
    n, ni, ng, nz = H.f64(g), idx.cpu().numpy(), H.f64(out.gate), H.f64(z)
    ref = OL.route_backward(nz, ni, ng, None, rows, n, None, renorm)
    p, rel = OL.softmax_rows(nz), H.probability_bound(nz)
    part = np.abs(ng) * (np.abs(n) + np.sum(np.abs(ng * n), axis=1, keepdims=True)) if renorm else np.abs(n)
    mag = np.zeros((rows, E))
    np.add.at(mag, (np.arange(rows)[:, None], ni), part)
    if not renorm:
        mag = p * (mag + np.sum(p * mag, axis=1, keepdims=True))
    # as for picks named once: the probabilities enter twice, sums are over k + 8 + 3 terms
    H.assert_within(got[0], ref, H.rounded((2 * rel + (k + 16) * H.U) * mag, ref, "fp32"), "dlogits")
