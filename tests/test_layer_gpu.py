"""The norms, dropout and the batched router, and their backward passes, against the fp64 oracle,
element by element, within bounds derived from the arithmetic (layer_helpers)."""
import numpy as np
import pytest
import torch

import layer_helpers as H
from oracle import layer as OL
from weight_merge_amd import api as A

DEV = "cuda"
EPS = 1e-5
# past the rows at which the backward pass sums rows and columns in one pass
ONE_PASS = [(700, 24), (900, 136), (700, 264), (800, 520), (1300, 1032), (2100, 1536), (1200, 4096), (1700, 8192)]
BOTH = pytest.mark.parametrize("dtype", ("fp32", "bf16"))
# (rows, d): d from one block of eight to the widest, every way a row is shared among lanes, on and
# off its edges; rows one, few, off the row groups, more than there are workgroups
SHAPES = [(1, 8), (300, 8), (2, 16), (37, 24), (700, 40), (5, 64), (129, 136), (3, 256), (33, 264), (65, 512), (7, 520),
          (257, 520), (300, 1032), (1, 2048), (31, 2056), (1, 4096), (513, 4096), (3, 6152), (40, 8192), (5, 8200),
          (2, 16384), (3, 16392), (1, 28672), (270, 28672), (2, 32768)]


def row_scales(seed, d):
    """Channels of many sizes, as a residual stream has."""
    return torch.exp(H.normal(seed, (d,), 0.5, "fp32"))


def made(seed, rows, d, dtype, pad=0):
    t = {"x": H.normal(seed, (rows, d), 1.0, dtype), "dy": H.normal(seed + 1, (rows, d), 0.1, dtype),
         "res": (H.normal(seed + 2, (rows, d), 2.0, "fp32") * row_scales(seed + 3, d) + 0.3).to(H.TD[dtype]),
         "dhidden": H.normal(seed + 4, (rows, d), 0.1, dtype), "w": (1 + H.normal(seed + 5, (d,), 0.2, "fp32")).to(H.TD[dtype]),
         "b": H.normal(seed + 6, (d,), 0.2, dtype)}
    return {k: H.f64(v) for k, v in t.items()}, {k: H.strided(v, DEV, pad) for k, v in t.items()}


def empty(*shape, dtype="fp32", pad=0):
    return torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=H.TD[dtype], device=DEV)[..., : shape[-1]]


def gaps_untouched(*tensors):
    for t in tensors:
        assert t._base[:, t.shape[1]:].isnan().all(), "the gap between rows was written"


def check_norm(rows, d, dtype, kind, p=0.0, residual=True, affine=True, pad=0, seed=0):
    n, t = made(seed, rows, d, dtype, pad)
    w, b = (n["w"], n["b"]) if affine else (None, None)
    y, hidden = empty(rows, d, dtype=dtype, pad=pad), empty(rows, d, dtype=dtype, pad=pad)
    mean, rstd = empty(rows), empty(rows)
    got = A.ada_norm(t["x"], t["w"] if affine else None, bias=t["b"] if affine else None,
                     residual=t["res"] if residual else None, kind=kind, eps=EPS, p=p, seed=seed + 11, offset=5, y=y,
                     hidden=hidden, stats=(mean, rstd))
    assert got is y
    dropped = OL.dropout(n["x"], p, seed + 11, 5) if p else n["x"]
    h = dropped + n["res"] if residual else dropped
    eh = np.zeros_like(h)
    if p:
        eh = eh + H.U * np.abs(dropped)
    if residual:
        eh = eh + H.U * (np.abs(h) + eh)
    ref, rmean, rrstd = OL.norm(h, w, b, kind, EPS)
    by, bm, bs = H.norm_bounds(h, eh, w, b, kind, EPS, dtype)
    what = f"{rows}x{d} {dtype} {kind}"
    H.assert_within(hidden, h, H.rounded(eh, h, dtype), "hidden " + what)
    H.assert_within(rstd, rrstd, bs, "rstd " + what)
    if kind == "layer":
        H.assert_within(mean, rmean, bm, "mean " + what)
    else:
        assert mean.isnan().all()
    H.assert_within(y, ref, by, "y " + what)
    if pad:
        gaps_untouched(y, hidden)


def check_norm_backward(rows, d, dtype, kind, p=0.0, dhidden=True, weight=True, pad=0, seed=0):
    n, t = made(seed, rows, d, dtype, pad)
    _, mean, rstd = OL.norm(n["res"], None, None, kind, EPS)
    stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in (mean, rstd)]
    mean, rstd = (H.f64(v) for v in stats)
    dx, dr = empty(rows, d, dtype=dtype, pad=pad), empty(rows, d, dtype=dtype, pad=pad)
    dw, db = empty(d, dtype=dtype), empty(d, dtype=dtype)
    A.ada_norm_backward(t["dy"], t["res"], (stats[0] if kind == "layer" else None, stats[1]), t["w"] if weight else None,
                        dhidden=t["dhidden"] if dhidden else None, kind=kind, p=p, seed=seed + 11, offset=5, dx=dx,
                        dresidual=dr, dweight=dw, dbias=db)
    args = (n["dy"], n["res"], mean, rstd, n["w"] if weight else None, n["dhidden"] if dhidden else None, kind)
    rh, rw, rb = OL.norm_backward(*args)
    eh, ew, eb = H.norm_grad_bounds(*args)
    what = f"{rows}x{d} {dtype} {kind}"
    H.assert_within(dr, rh, H.rounded(eh, rh, dtype), "dresidual " + what)
    if p:
        kept, scale = OL.dropout_mask(rows, d, p, seed + 11, 5)
        rx = np.where(kept, rh * scale, 0.0)
        H.assert_within(dx, rx, np.where(kept, H.rounded(eh * scale + H.U * np.abs(rx), rx, dtype), 0.0), "dx " + what)
    else:
        assert torch.equal(dx, dr)
    H.assert_within(dw, rw, H.rounded(ew, rw, dtype), "dw " + what)
    H.assert_within(db, rb, H.rounded(eb, rb, dtype), "db " + what)
    if pad:
        gaps_untouched(dx, dr)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", SHAPES + [(2050, 264), (2051, 520), (2048, 1032), (2049, 1536)],
                         ids=lambda s: "x".join(map(str, s)))
def test_norm_shapes(shape, dtype):
    check_norm(*shape, dtype, "layer", seed=sum(shape))
    check_norm(*shape, dtype, "rms", p=0.2, seed=sum(shape) + 1)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", SHAPES + ONE_PASS, ids=lambda s: "x".join(map(str, s)))
def test_norm_backward_shapes(shape, dtype):
    check_norm_backward(*shape, dtype, "rms", seed=sum(shape))
    check_norm_backward(*shape, dtype, "layer", p=0.2, seed=sum(shape) + 1)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", [(17000, 248), (2051, 2056), (520, 8136), (257, 16392)],
                         ids=lambda s: "x".join(map(str, s)))
def test_matrices_past_the_caches(shape, dtype):
    """From 2^22 elements on, some accesses are of another kind."""
    rows, d = shape
    assert rows * d >= 2 ** 22
    check_norm(*shape, dtype, "layer", p=0.2, pad=8, seed=3)
    check_norm_backward(*shape, dtype, "layer", p=0.2, pad=8, seed=4)
    n, t = made(5, *shape, dtype, pad=8)
    y = empty(*shape, dtype=dtype, pad=8)
    A.ada_dropout(t["x"], 0.2, 6, 7, residual=t["res"], y=y)
    dropped = OL.dropout(n["x"], 0.2, 6, 7)
    H.assert_within(y, dropped + n["res"], H.dropout_bound(dropped + n["res"], dropped, n["res"], dtype), "dropout")
    gaps_untouched(y)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("kind", ("layer", "rms"))
@pytest.mark.parametrize("p", (0.0, 0.3))
def test_norm_operands_on_and_off(kind, p, dtype):
    for i, (residual, affine, pad) in enumerate([(False, True, 0), (True, False, 8), (False, False, 24), (True, True, 64)]):
        check_norm(70, 328, dtype, kind, p=p, residual=residual, affine=affine, pad=pad, seed=i)
        check_norm_backward(70, 328, dtype, kind, p=p, dhidden=residual, weight=affine, pad=pad, seed=i)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows", (300, 900))
def test_gradients_do_not_depend_on_which_are_asked_for(rows, dtype):
    n, t = made(5, rows, 264, dtype)
    stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in OL.norm(n["res"], None, None, "layer", EPS)[1:]]
    kw = dict(weight=t["w"], dhidden=t["dhidden"], p=0.1, seed=3)
    every = A.ada_norm_backward(t["dy"], t["res"], stats, want_dresidual=True, want_dbias=True, **kw)
    names = ("want_dx", "want_dresidual", "want_dweight", "want_dbias")
    for i, one in enumerate(names):
        got = A.ada_norm_backward(t["dy"], t["res"], stats, **{n: n == one for n in names}, **kw)
        assert torch.equal(got[i], every[i]) and all(got[j] is None for j in range(4) if j != i)


@pytest.mark.gpu
@BOTH
def test_norm_in_place(dtype):
    for rows, d in ((65, 520), (3, 4096), (2, 20480)):
        n, t = made(7, rows, d, dtype)
        kw = dict(bias=t["b"], p=0.1, seed=9)
        hidden = empty(rows, d, dtype=dtype)
        ref = A.ada_norm(t["x"], t["w"], residual=t["res"], hidden=hidden, **kw)
        for y, h in (("x", "res"), ("res", "x")):
            c = {k: v.clone() for k, v in t.items()}
            A.ada_norm(c["x"], t["w"], residual=c["res"], y=c[y], hidden=c[h], **kw)
            assert torch.equal(c[y], ref) and torch.equal(c[h], hidden)
        stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in OL.norm(n["res"], None, None, "layer", EPS)[1:]]
        kw = dict(weight=t["w"], p=0.1, seed=9, want_dresidual=True)
        ref = A.ada_norm_backward(t["dy"], t["res"], stats, dhidden=t["dhidden"], **kw)
        for x, r in (("dy", "dhidden"), ("dhidden", "dy")):
            c = {k: v.clone() for k, v in t.items()}
            got = A.ada_norm_backward(c["dy"], t["res"], stats, dhidden=c["dhidden"], dx=c[x], dresidual=c[r], **kw)
            assert all(torch.equal(a, b) for a, b in zip(got[:3], ref[:3]))


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", [(512, 8192), (900, 264), (200, 16392)], ids=lambda s: "x".join(map(str, s)))
def test_gradients_in_the_place_of_dy(shape, dtype):
    """dw and db read dy too, whichever workgroup is the first to write there."""
    n, t = made(12, *shape, dtype)
    stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in OL.norm(n["res"], None, None, "layer", EPS)[1:]]
    kw = dict(weight=t["w"], dhidden=t["dhidden"], want_dbias=True)
    ref = A.ada_norm_backward(t["dy"], t["res"], stats, **kw)
    for rep in range(10):
        for where in ("dx", "dresidual"):
            dy = t["dy"].clone()
            got = A.ada_norm_backward(dy, t["res"], stats, **{where: dy}, want_dx=where == "dx", **kw)
            assert torch.equal(got[0 if where == "dx" else 1], ref[0])
            assert torch.equal(got[2], ref[2]) and torch.equal(got[3], ref[3])


@pytest.mark.gpu
@pytest.mark.parametrize("shift", (300.0, 5e4))
def test_rows_far_from_zero(shift):
    """fp32 rows whose mean is many standard deviations from zero: the bound on y, which holds the
    rounding of one sum of the row times 1 / std, would allow a thousandth; the second pass takes that
    sum's error out, so what stays is a few roundings of (h - mean)."""
    rows, d = 9, 4104
    h = (H.normal(1, (rows, d), 1.0, "fp32") + shift).to(DEV)
    n = H.f64(h)
    ref, mean, rstd = OL.norm(n, None, None, "layer", EPS)
    m = empty(rows)
    y = A.ada_norm(h, eps=EPS, stats=(m, None))
    # h - m is exact up to its own rounding (both are multiples of h's last place and the difference
    # is small); the rest of the mean is off by DEPTH u of its few last places of m
    left = H.DEPTH * H.U * (H.DEPTH * H.U * shift) + 2 * H.U * np.abs(n - mean[:, None])
    H.assert_within(y, ref, 2 * left + (H.DEPTH + 8) * H.U * np.abs(ref) + H.TINY, "y")
    H.assert_within(m, mean, (2 * H.U * shift) * np.ones(rows), "mean")


@pytest.mark.gpu
@BOTH
def test_constant_rows_and_zero_eps(dtype):
    x = torch.full((3, 264), 1.5, dtype=H.TD[dtype], device=DEV)
    rstd = empty(3)
    y = A.ada_norm(x, eps=0.25, stats=(None, rstd))
    assert (y == 0).all() and (rstd == 2).all()
    y = A.ada_norm(x, kind="rms", eps=0.0)
    assert (y == 1).all()
    assert A.ada_norm(x, eps=0.0).isnan().all()  # 0 / 0, as in the formula


@pytest.mark.gpu
@BOTH
def test_nan_and_infinity_stay_in_their_rows(dtype):
    n, t = made(2, 6, 328, dtype)
    bad = t["x"].clone()
    bad[1, 5], bad[3, 300], bad[5, 0] = float("nan"), float("inf"), -float("inf")
    stats, ref_stats = (empty(6), empty(6)), (empty(6), empty(6))
    y = A.ada_norm(bad, t["w"], bias=t["b"], stats=stats)
    ref = A.ada_norm(t["x"], t["w"], bias=t["b"], stats=ref_stats)
    for r in range(6):
        if r % 2:
            assert y[r].isnan().all() and stats[1][r].isnan()
        else:
            assert torch.equal(y[r], ref[r]) and stats[0][r] == ref_stats[0][r]
    dy = t["dy"].clone()
    dy[1, 5] = float("nan")
    dx, _, dw, db = A.ada_norm_backward(dy, t["x"], ref_stats, t["w"], want_dbias=True)
    rx, _, rw, rb = A.ada_norm_backward(t["dy"], t["x"], ref_stats, t["w"], want_dbias=True)
    assert dx[1].isnan().all() and torch.equal(dx[[0, 2, 3, 4, 5]], rx[[0, 2, 3, 4, 5]])
    keep = torch.arange(328, device=DEV) != 5
    assert dw[5].isnan() and db[5].isnan() and torch.equal(dw[keep], rw[keep]) and torch.equal(db[keep], rb[keep])


# ---- dropout ---------------------------------------------------------------------------
@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", [(1, 8), (1, 4096), (700, 8), (3, 1032), (129, 264), (513, 2056), (2, 65544)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("pad", (0, 8))
def test_dropout_shapes(shape, pad, dtype):
    rows, d = shape
    n, t = made(rows + d, rows, d, dtype, pad)
    for p, seed, offset in ((0.1, 1, 0), (0.5, 2 ** 40 + 3, 2 ** 33 + 1), (0.0, 5, 6), (1.0, 5, 6), (0.9, -1, 2 ** 64 - 1)):
        y, y2, dx = (empty(rows, d, dtype=dtype, pad=pad) for _ in range(3))
        assert A.ada_dropout(t["x"], p, seed, offset, y=y) is y
        dropped = OL.dropout(n["x"], p, seed, offset)
        H.assert_within(y, dropped, H.dropout_bound(dropped, dropped, None, dtype), f"y p={p}")
        assert torch.equal(y == 0, torch.from_numpy(dropped == 0).to(DEV))
        A.ada_dropout(t["x"], p, seed, offset, residual=t["res"], y=y2)
        H.assert_within(y2, dropped + n["res"], H.dropout_bound(dropped + n["res"], dropped, n["res"], dtype), "sum")
        A.ada_dropout_backward(t["dy"], p, seed, offset, dx=dx)
        grad = OL.dropout(n["dy"], p, seed, offset)
        H.assert_within(dx, grad, H.dropout_bound(grad, grad, None, dtype), "dx")
        if pad:
            gaps_untouched(y, y2, dx)


@pytest.mark.gpu
@BOTH
def test_what_is_dropped_is_zero_whatever_it_was(dtype):
    rows, d, p = 40, 264, 0.4
    n, t = made(3, rows, d, dtype)
    kept = torch.from_numpy(OL.dropout_mask(rows, d, p, 7, 1)[0]).to(DEV)
    x = t["x"].clone()
    holes = torch.where(torch.arange(rows, device=DEV)[:, None] % 2 == 0, float("nan"), float("inf")).to(x.dtype)
    x = torch.where(kept, x, holes)
    assert torch.equal(A.ada_dropout(x, p, 7, 1), A.ada_dropout(t["x"], p, 7, 1))
    assert torch.equal(A.ada_dropout_backward(x, p, 7, 1), A.ada_dropout_backward(t["x"], p, 7, 1))
    for kind in ("layer", "rms"):
        kw = dict(weight=t["w"], residual=t["res"], kind=kind, p=p, seed=7, offset=1)
        assert torch.equal(A.ada_norm(x, **kw), A.ada_norm(t["x"], **kw))
    # the other way round: a kept infinity stays
    assert torch.equal(A.ada_dropout(torch.where(kept, float("inf"), x).to(x.dtype), p, 7, 1).isinf(), kept)


@pytest.mark.gpu
@BOTH
def test_dropout_in_place_and_the_norm_s_dropout(dtype):
    n, t = made(4, 33, 520, dtype)
    state = torch.tensor([-12345, 2 ** 62], dtype=torch.int64, device=DEV)
    ref = A.ada_dropout(t["x"], 0.25, -12345, 2 ** 62 + 9, residual=t["res"])
    for y in ("x", "res"):
        c = {k: v.clone() for k, v in t.items()}
        A.ada_dropout(c["x"], 0.25, state, 9, residual=c["res"], y=c[y])
        assert torch.equal(c[y], ref)
    c = t["dy"].clone()
    A.ada_dropout_backward(c, 0.25, state, 9, dx=c)
    assert torch.equal(c, A.ada_dropout_backward(t["dy"], 0.25, -12345, 2 ** 62 + 9))
    hidden = empty(33, 520, dtype=dtype)
    A.ada_norm(t["x"], residual=t["res"], p=0.25, seed=state, offset=9, hidden=hidden)
    assert torch.equal(hidden, ref)


@pytest.mark.gpu
def test_dropout_past_32_bits_of_elements():
    """More than 2^32 elements in place, and rows further apart than that."""
    rows, d = 2 ** 19 + 5, 8200
    x = torch.ones((rows, d), dtype=torch.bfloat16, device=DEV)
    A.ada_dropout(x, 0.5, 3, 4, y=x)
    for first in (0, 2 ** 18 - 1, rows - 3):
        kept, scale = OL.dropout_mask(3, d, 0.5, 3, 4, first_row=first)
        assert np.array_equal(H.f64(x[first:first + 3]), kept * scale), first
    del x
    buf = torch.empty(2 * (2 ** 32 + 8) + 1024, dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((3, 264), (2 ** 32 + 8, 1))
    near = H.normal(1, (3, 264), 1.0, "bf16").to(DEV)
    far.copy_(near)
    w = torch.ones(264, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(A.ada_norm(far, w, p=0.3, seed=1), A.ada_norm(near, w, p=0.3, seed=1))
    assert torch.equal(A.ada_dropout(far, 0.3, 1, y=far), A.ada_dropout(near, 0.3, 1))


@pytest.mark.gpu
def test_more_rows_than_workgroups():
    """Workgroups of the norm that take a second row, with the dropout's place of it."""
    rows, d = 2 ** 20 + 3, 2056
    x = torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
    x.view(-1)[: 1 << 24].normal_()
    x.view(-1)[1 << 24:].copy_(x.view(-1)[: 1 << 24].repeat(rows * d // (1 << 24) + 1)[: rows * d - (1 << 24)])
    w = (1 + H.normal(1, (d,), 0.1, "fp32")).to(H.TD["bf16"]).to(DEV)
    for first in (0, 2 ** 20 - 2, rows - 2):
        at = x[first:first + 2]
        kept = torch.from_numpy(OL.dropout_mask(2, d, 0.5, 3, 4, first_row=first)[0]).to(DEV)
        part = torch.where(kept, at * 2, 0.0)
        expect = (part.clone(), A.ada_norm(part, w))
        if first == 0:
            hidden = torch.empty_like(x)
            y = A.ada_norm(x, w, p=0.5, seed=3, offset=4, hidden=hidden)
        assert torch.equal(hidden[first:first + 2], expect[0]) and torch.equal(y[first:first + 2], expect[1])


# ---- the router ------------------------------------------------------------------------
# (rows, experts, k): one lane to eight lanes a row, experts on and off multiples of eight, every
# number of picks, rows that fill no, one and several workgroups
ROUTES = [(1, 1, 1), (5, 2, 2), (48, 8, 2), (1, 8, 8), (1025, 8, 2), (100, 13, 4), (513, 16, 4), (700, 24, 5), (33, 32, 32),
          (300, 40, 3), (257, 64, 8), (40, 64, 64), (1500, 63, 6), (2600, 16, 4)]


def route_inputs(seed, rows, E, dtype, closed=0.0, ties=False, valid=False, pad=0):
    z = H.logits(seed, rows, E, dtype, closed, ties)
    flags = None
    if valid:
        flags = torch.arange(rows) % 5 != 3
    dev = H.strided(z, DEV, pad)
    return H.f64(z), dev, flags


def check_route(rows, E, k, dtype, renorm=True, closed=0.0, ties=False, valid=False, pad=0, seed=0):
    z, dz, flags = route_inputs(seed, rows, E, dtype, closed, ties, valid, pad)
    dev_flags = None if flags is None else flags.to(DEV)
    got = A.ada_route(dz, k, renorm=renorm, valid=dev_flags)
    ref = OL.route(z, k, renorm, None if flags is None else flags.numpy())
    assert np.array_equal(got.idx.cpu().numpy(), ref[0])
    assert np.array_equal(got.counts.cpu().numpy(), ref[2]) and int(got.used) == ref[5]
    rel = H.probability_bound(z)
    H.assert_within(got.gate, ref[1], rel * ref[1] + H.TINY, "gate")
    eprob = (rel * OL.softmax_rows(z)).sum(axis=0) / max(ref[5], 1) + (rows + H.DEPTH) * H.U * ref[3]
    H.assert_within(got.prob, ref[3], eprob + H.TINY, "prob")
    eloss = E * np.sum(ref[2] / (k * max(ref[5], 1)) * eprob) + 4 * H.U * ref[4]
    H.assert_within(got.loss, np.array([ref[4]]), np.array([eloss + H.TINY]), "loss")
    bare = A.ada_route(dz, k, renorm=renorm, valid=dev_flags, balance=False)
    assert torch.equal(bare.idx, got.idx) and torch.equal(bare.gate, got.gate) and bare.counts is None
    check_route_backward(z, dz, got, renorm, dtype, pad, seed)


def check_route_backward(z, dz, out, renorm, dtype, pad, seed):
    rows, E = z.shape
    k = out.idx.shape[1]
    g = H.normal(seed + 7, (rows, k), 0.3, "fp32").to(DEV)
    one = torch.full((1,), 0.37, dtype=torch.float32, device=DEV)
    idx, gate, counts = out.idx.cpu().numpy(), H.f64(out.gate), out.counts.cpu().numpy()
    n = max(int(out.used), 1)
    p = OL.softmax_rows(z)
    rel = H.probability_bound(z)
    for dgate, dloss in ((g, one), (g, None), (None, one)):
        got = empty(rows, E, dtype=dtype, pad=pad)
        assert A.ada_route_backward(dz, out, dgate=dgate, dloss=dloss, renorm=renorm, dlogits=got) is got
        dg = None if dgate is None else H.f64(dgate)
        ref = OL.route_backward(z, idx, gate, counts, int(out.used), dg, None if dloss is None else float(dloss), renorm)
        # magnitudes of everything that is added up
        dp = np.zeros((rows, E)) if dloss is None else np.tile(float(dloss) * E * counts / (k * n * n), (rows, 1))
        mag = np.zeros((rows, E))
        if dgate is not None:
            at = np.where(idx >= 0, idx, 0)
            part = np.abs(gate) * (np.abs(dg) + np.sum(np.abs(gate * dg), axis=1, keepdims=True)) if renorm else np.abs(dg)
            np.add.at(mag if renorm else dp, (np.arange(rows)[:, None], at), np.where(idx >= 0, part, 0.0))
        mag += p * (np.abs(dp) + np.sum(p * np.abs(dp), axis=1, keepdims=True))
        # the probabilities enter twice, sums are over k + 8 + 3 terms
        err = (2 * rel + (k + 16) * H.U) * mag
        H.assert_within(got, ref, H.rounded(err, ref, dtype), f"dlogits {renorm} {dgate is None} {dloss is None}")
        assert (got.float()[idx[:, 0] < 0] == 0).all()
        if pad:
            gaps_untouched(got)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("shape", ROUTES, ids=lambda s: "x".join(map(str, s)))
def test_route_shapes(shape, dtype):
    check_route(*shape, dtype, seed=sum(shape))
    check_route(*shape, dtype, renorm=False, closed=0.3, ties=True, valid=True, pad=3, seed=sum(shape) + 1)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("E", (8, 12, 64))
def test_route_ties_closed_experts_and_padding(E, renorm, dtype):
    for i, (closed, ties, valid, pad) in enumerate([(0.0, True, False, 0), (0.5, False, False, 8), (0.9, True, True, 5),
                                                    (0.0, False, True, 16)]):
        check_route(90, E, 4, dtype, renorm=renorm, closed=closed, ties=ties, valid=valid, pad=pad, seed=i)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, E, k", (("fp32", 64, 3), ("bf16", 7, 2)))
def test_route_of_many_rows(dtype, E, k):
    """More rows than the workgroups take in one step."""
    rows = {64: 36000, 7: 280000}[E]
    z = H.logits(5, rows, E, dtype, ties=dtype == "bf16").to(DEV)
    valid = torch.arange(rows, device=DEV) % 7 != 2
    got = A.ada_route(z, k, valid=valid)
    order = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :k]
    idx = torch.where(valid[:, None], order, -1)
    assert torch.equal(got.idx.long(), idx) and int(got.used) == int(valid.sum())
    counts = torch.bincount(idx[valid].flatten(), minlength=E)
    assert torch.equal(got.counts.long(), counts)
    p = torch.softmax(z.double(), 1)
    rel = torch.from_numpy(H.probability_bound(H.f64(z))).to(DEV)
    mean = p[valid].mean(0)
    # sums of at most 16 steps of 64 rows on a lane and of 256 workgroups
    eprob = (rel * p)[valid].mean(0) + (16 + H.DEPTH + 256) * H.U * mean
    H.assert_within(got.prob, H.f64(mean), H.f64(eprob), "prob")
    share = counts.double() / (k * valid.sum())
    loss = E * (share * mean).sum()
    H.assert_within(got.loss, H.f64(loss[None]), H.f64((E * (share * eprob).sum() + 4 * H.U * loss)[None]), "loss")
    picked = torch.gather(p, 1, order)
    ref = torch.where(valid[:, None], picked / picked.sum(1, keepdim=True), 0.0)
    H.assert_within(got.gate, H.f64(ref), H.f64(rel * ref + H.TINY), "gate")


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("E", (8, 16, 21))
def test_route_of_logits_that_begin_anywhere(E, dtype):
    """Columns of a wider product from an odd one on, and rows from an odd one on: no vector is aligned."""
    z = H.logits(6, 70, E, dtype, closed=0.2)
    ref = A.ada_route(z.to(DEV), 3)
    g = H.normal(7, (70, 3), 0.3, "fp32").to(DEV)
    dref = A.ada_route_backward(z.to(DEV), ref, dgate=g, dloss=ref.loss)
    wide = torch.full((71, E + 16), float("nan"), dtype=H.TD[dtype], device=DEV)
    for first, at in ((1, 0), (3, 1), (0, 1)):
        view, dview = wide[at:at + 70, first:first + E], wide.clone()[at:at + 70, first:first + E]
        view.copy_(z)
        got = A.ada_route(view, 3)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        A.ada_route_backward(view, got, dgate=g, dloss=got.loss, dlogits=dview)
        assert torch.equal(dview, dref)
    flat = torch.empty(70 * E + 1, dtype=H.TD[dtype], device=DEV)[1:].view(70, E)
    flat.copy_(z)
    assert all(torch.equal(a, b) for a, b in zip(A.ada_route(flat, 3), ref))


@pytest.mark.gpu
def test_route_of_nothing():
    z = torch.zeros((4, 8), device=DEV)
    none = torch.zeros(4, dtype=torch.bool, device=DEV)
    closed = torch.full((4, 8), -float("inf"), device=DEV)
    for got in (A.ada_route(z, 2, valid=none), A.ada_route(closed, 2), A.ada_route(z[:0], 2)):
        assert (got.idx == -1).all() and (got.gate == 0).all() and (got.counts == 0).all() and (got.prob == 0).all()
        assert int(got.used) == 0 and float(got.loss) == 0
    for logits, got in ((z, A.ada_route(z, 2, valid=none)), (closed, A.ada_route(closed, 2))):
        one = torch.ones(1, device=DEV)
        assert (A.ada_route_backward(logits, got, dgate=torch.ones((4, 2), device=DEV), dloss=one) == 0).all()
    assert A.ada_route_backward(z[:0], A.ada_route(z[:0], 2), dloss=torch.ones(1, device=DEV)).shape == (0, 8)


@pytest.mark.gpu
def test_rows_that_lie_on_each_other_are_refused():
    """Rows broadcast from one, or closer than their length: no row stride the calls take."""
    for z in (torch.zeros((1, 16), device=DEV).expand(5, 16), torch.zeros(100, device=DEV).as_strided((5, 16), (8, 1))):
        out = A.ada_route(torch.zeros((5, 16), device=DEV), 2)
        stats = (torch.zeros(5, device=DEV), torch.ones(5, device=DEV))
        for call in (lambda: A.ada_route(z, 2), lambda: A.ada_route_backward(z, out, dloss=out.loss), lambda: A.ada_norm(z),
                     lambda: A.ada_norm(torch.zeros((5, 16), device=DEV), residual=z), lambda: A.ada_dropout(z, 0.1, 1),
                     lambda: A.ada_dropout_backward(z, 0.1, 1), lambda: A.ada_norm_backward(z, z, stats),
                     lambda: A.ada_dropout(torch.zeros((5, 16), device=DEV), 0.1, 1, y=z),
                     lambda: A.ada_route_backward(out.gate.new_zeros((5, 16)), out, dloss=out.loss, dlogits=z)):
            with pytest.raises(A.AdaError):
                call()


@pytest.mark.gpu
def test_no_balance_into_the_buffers_of_one_that_had_it():
    z = H.logits(1, 9, 12, "fp32").to(DEV)
    out = A.ada_route(z, 3)
    bare = A.ada_route(z, 2, balance=False, out=(torch.empty_like(out.idx[:, :2]).contiguous(),
                                                 torch.empty_like(out.gate[:, :2]).contiguous(), *out[2:]))
    assert bare[2:] == (None,) * 4 and torch.equal(bare.idx, out.idx[:, :2])


@pytest.mark.gpu
def test_route_of_the_largest_and_lowest_logits():
    """The type's lowest value is an open expert of no probability, not a closed one; equal
    zeros of either sign tie; NaN and +inf are picked and stay in their row, out of range never."""
    low = torch.finfo(torch.float32).min
    z = torch.tensor([[low, low, 0.0, -0.0], [low, low, low, low], [-0.0, 0.0, -0.0, 0.0], [3e38, low, -3e38, 0.0]], device=DEV)
    got = A.ada_route(z, 3)
    assert got.idx.tolist() == [[2, 3, 0], [0, 1, 2], [0, 1, 2], [0, 3, 2]]
    assert torch.equal(got.gate, torch.tensor([[0.5, 0.5, 0], [1 / 3] * 3, [1 / 3] * 3, [1, 0, 0]], device=DEV))
    assert int(got.used) == 4 and got.counts.tolist() == [4, 2, 4, 2]
    nan, inf = float("nan"), float("inf")
    z = torch.tensor([[1.0, nan, -inf, 2.0], [1.0, 3.0, 2.0, inf], [1.0, 2.0, 3.0, 0.0]], device=DEV)
    got = A.ada_route(z, 2)
    assert got.idx.tolist() == [[1, 3], [3, 1], [2, 1]]
    assert got.gate[0].isnan().all() and got.gate[1, 0].isnan() and not got.gate[2].isnan().any()
    assert got.loss.isnan().all() and int(got.used) == 3
    only = A.ada_route(z, 2, valid=torch.tensor([0, 0, 1], dtype=torch.uint8, device=DEV))
    assert not only.loss.isnan().any() and not only.prob.isnan().any() and only.idx[:2].eq(-1).all()
    dz = A.ada_route_backward(z, only, dgate=torch.ones((3, 2), device=DEV), dloss=torch.ones(1, device=DEV))
    assert (dz[:2] == 0).all() and not dz.isnan().any()


@pytest.mark.gpu
def test_route_passes_over_indices_out_of_range():
    z = H.logits(1, 6, 12, "fp32").to(DEV)
    out = A.ada_route(z, 3)
    bad = out.idx.clone()
    bad[2, 1], bad[3, 2], bad[4, 1] = 1 << 30, 12, -7
    g = H.normal(2, (6, 3), 1.0, "fp32").to(DEV)
    got = A.ada_route_backward(z, out._replace(idx=bad), dgate=g, renorm=False)
    rows = [0, 1, 5]
    assert torch.equal(got[rows], A.ada_route_backward(z, out, dgate=g, renorm=False)[rows])
    ref = OL.route_backward(H.f64(z), bad.cpu().numpy(), H.f64(out.gate), None, 6, H.f64(g), None, False)
    p = OL.softmax_rows(H.f64(z))
    err = (2 * H.probability_bound(H.f64(z)) + 32 * H.U) * p * 8 * np.abs(H.f64(g)).max()
    H.assert_within(got, ref, 2 * err + H.TINY, "dlogits")


@pytest.mark.gpu
def test_route_agrees_with_pregate():
    for E, k, renorm in ((4, 2, True), (16, 4, True), (64, 5, False)):
        h, R = H.normal(E, (256,), 1.0, "bf16").to(DEV), H.normal(E + 1, (E, 256), 0.1, "bf16").to(DEV)
        idx, gate = A.ada_pregate(h, R, k, renorm=renorm)
        z = (R.double() @ h.double()).float()[None]
        got = A.ada_route(z, k, renorm=renorm, balance=False)
        assert torch.equal(got.idx[0], idx)
        # the logits of the two differ by the fp32 sums over 256 products
        assert torch.allclose(got.gate[0], gate, rtol=4 * 260 * H.U * 40, atol=1e-6)


# ---- empty matrices, streams, graphs ---------------------------------------------------
@pytest.mark.gpu
@BOTH
def test_no_rows(dtype):
    x = torch.empty((0, 264), dtype=H.TD[dtype], device=DEV)
    w = torch.ones(264, dtype=H.TD[dtype], device=DEV)
    assert A.ada_norm(x, w).shape == (0, 264) and A.ada_dropout(x, 0.1, 1).shape == (0, 264)
    none = torch.empty(0, device=DEV)
    dx, _, dw, db = A.ada_norm_backward(x, x, (none, none), w, want_dbias=True)
    assert dx.shape == (0, 264) and (dw == 0).all() and (db == 0).all()


def training_step(t, state, offset=0):
    """Every call once, as a captured step makes them."""
    rows, d = t["x"].shape
    hidden = torch.empty_like(t["x"])
    stats = (torch.empty(rows, device=DEV), torch.empty(rows, device=DEV))
    y = A.ada_norm(t["x"], t["w"], bias=t["b"], residual=t["res"], p=0.2, seed=state, offset=offset, hidden=hidden, stats=stats)
    z = A.ada_dropout(y, 0.1, state, offset + 1, residual=hidden)
    out = A.ada_route(z[:, :16].float().contiguous(), 4)
    dz = A.ada_route_backward(z[:, :16].float().contiguous(), out, dgate=out.gate, dloss=out.loss)
    dy = A.ada_dropout_backward(t["dy"], 0.1, state, offset + 1)
    grads = A.ada_norm_backward(dy, hidden, stats, t["w"], dhidden=t["dhidden"], p=0.2, seed=state, offset=offset,
                                want_dresidual=True, want_dbias=True)
    return [y, hidden, *stats, z, *out, dz, dy, *grads]


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows", (5, 1500))
def test_captured_and_replayed_with_a_state_that_moves(rows, dtype):
    """Two graphs with workspaces of their own pool; the generator's state changes between replays,
    and other eager calls run on the same tensors in between."""
    _, t = made(8, rows, 264, dtype)
    state = torch.tensor([77, 0], dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        training_step(t, state)
    torch.cuda.synchronize()
    graphs = []
    for offset in (0, 100):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            graphs.append((g, offset, training_step(t, state, offset)))
    seen = []
    for rep in range(4):
        state.copy_(torch.tensor([77 + rep // 2, 1000 * rep], device=DEV))
        t["x"].copy_(H.normal(50 + rep, (rows, 264), 1.0, dtype))
        torch.cuda.synchronize()
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, offset, got in graphs:
            with torch.cuda.stream(side):
                ref = training_step(t, state, offset)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref)), (rep, offset)
        seen.append(graphs[0][2][1].clone())
    assert not torch.equal(seen[0] == t["res"], seen[1] == t["res"])  # other elements are dropped


@pytest.mark.gpu
@BOTH
def test_inputs_dropped_behind_the_call(dtype):
    """The call's stream has work before it; meanwhile the inputs are dropped and others of their
    sizes are made on the current stream."""
    n, _ = made(9, 40, 520, dtype)
    stats = OL.norm(n["res"], None, None, "layer", EPS)[1:]

    def inputs():
        _, t = made(9, 40, 520, dtype)
        t["mean"], t["rstd"] = (torch.tensor(v, dtype=torch.float32, device=DEV) for v in stats)
        t["state"] = torch.tensor([5, 6], dtype=torch.int64, device=DEV)
        t["z"] = H.logits(3, 40, 16, "fp32").to(DEV)
        t["valid"] = torch.arange(40, device=DEV) % 3 != 1
        return t

    def route_both(t, s):
        out = A.ada_route(t["z"], 4, valid=t["valid"], stream=s)
        with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
            dgate = out.gate * 2
        return [*out, A.ada_route_backward(t["z"], out, dgate=dgate, dloss=out.loss, stream=s)]

    runs = [lambda t, s: [A.ada_norm(t["x"], t["w"], bias=t["b"], residual=t["res"], p=0.1, seed=t["state"], stream=s)],
            lambda t, s: list(A.ada_norm_backward(t["dy"], t["res"], (t["mean"], t["rstd"]), t["w"], dhidden=t["dhidden"],
                                                  want_dbias=True, stream=s))[::2],
            lambda t, s: [A.ada_dropout(t["x"], 0.1, t["state"], residual=t["res"], stream=s)],
            lambda t, s: [A.ada_dropout_backward(t["dy"], 0.1, t["state"], stream=s)], route_both]
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device=DEV)
    for run in runs:
        ref = run(inputs(), None)
        t = inputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.add_(1)  # some milliseconds
        got = run(t, side)
        shapes = [(v.shape, v.dtype) for v in t.values()]
        del t
        others = [torch.full(s, 1, dtype=dt, device=DEV) for s, dt in shapes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        del others


@pytest.mark.gpu
@BOTH
def test_calls_on_two_streams_at_once(dtype):
    _, t = made(13, 1500, 1032, dtype)
    state = torch.tensor([3, 4], dtype=torch.int64, device=DEV)
    refs = [training_step(t, state, offset) for offset in (0, 50)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        got = []
        for side, offset in zip(sides, (0, 50)):
            with torch.cuda.stream(side):
                got.append(training_step(t, state, offset))
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_another_device_is_refused(monkeypatch):
    x = torch.zeros((4, 64), device=DEV)
    z = torch.zeros((4, 8), device=DEV)
    out = A.ada_route(z, 2)
    monkeypatch.setattr(A, "_device_now", lambda: 1)
    stats = (x[:, 0].contiguous(), x[:, 0].contiguous())
    for call in (lambda: A.ada_norm(x), lambda: A.ada_norm_backward(x, x, stats), lambda: A.ada_dropout(x, 0.1, 1),
                 lambda: A.ada_dropout_backward(x, 0.1, 1), lambda: A.ada_route(z, 2),
                 lambda: A.ada_route_backward(z, out, dloss=out.loss)):
        with pytest.raises(ValueError, match="is current"):
            call()


@pytest.mark.gpu
def test_equal_calls_give_equal_bits_and_exact_workspaces_do():
    n, t = made(10, 3000, 1032, "bf16")
    stats = [torch.tensor(v, dtype=torch.float32, device=DEV) for v in OL.norm(n["res"], None, None, "layer", EPS)[1:]]
    need = A.norm_backward_workspace_bytes(3000, 1032, torch.bfloat16)
    z = H.logits(4, 3000, 16, "fp32").to(DEV)
    rneed = A.route_workspace_bytes(3000, 16)
    first = None
    for rep in range(3):
        ws = torch.full((need + 64,), 0xA5 + rep, dtype=torch.uint8, device=DEV)
        rws = torch.full((rneed + 64,), 0xA5 + rep, dtype=torch.uint8, device=DEV)
        got = [*A.ada_norm_backward(t["dy"], t["res"], stats, t["w"], want_dbias=True, workspace=ws[:need])[::2],
               *A.ada_route(z, 4, workspace=rws[:rneed])]
        assert (ws[need:] == 0xA5 + rep).all() and (rws[rneed:] == 0xA5 + rep).all()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
