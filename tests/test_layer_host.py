"""Refusals of the norm, dropout and router calls (argument checks run on the host before any
HIP call), and the oracle against published numbers and differences.  No GPU needed."""
import math

import numpy as np
import pytest
import torch

from oracle import layer as OL
from weight_merge_amd import _lib
from weight_merge_amd import api as A
from weight_merge_amd._lib import (ADA_BF16, ADA_EALIGN, ADA_EDTYPE, ADA_EHIP, ADA_EINVAL, ADA_ESHAPE, ADA_F32,
                                   ADA_NORM_RMS, AdaDropoutArgs, AdaDropoutGradArgs, AdaNormArgs,
                                   AdaNormGradArgs, AdaRouteArgs, AdaRouteGradArgs)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: runs where no GPU is visible")

MB = 1 << 20
ROWS, D, E, K = 40, 64, 12, 3
# fake, aligned, far-apart addresses: every call below fails before it could touch them
SETS = {
    "dropout": (AdaDropoutArgs, dict(x=MB, residual=2 * MB, y=3 * MB, ld_x=D, ld_res=D, ld_y=D, rows=ROWS, d=D)),
    "dropout_backward": (AdaDropoutGradArgs, dict(dy=MB, dx=2 * MB, ld_dy=D, ld_dx=D, rows=ROWS, d=D)),
    "norm": (AdaNormArgs, dict(x=MB, residual=2 * MB, weight=3 * MB, bias=4 * MB, y=5 * MB, hidden=6 * MB, mean=7 * MB,
                               rstd=8 * MB, ld_x=D, ld_res=D, ld_y=D, ld_hidden=D, rows=ROWS, d=D, eps=1e-5)),
    "norm_backward": (AdaNormGradArgs, dict(dy=MB, hidden=2 * MB, dhidden=3 * MB, weight=4 * MB, mean=5 * MB,
                                            rstd=6 * MB, dx=7 * MB, dresidual=8 * MB, dweight=9 * MB, dbias=10 * MB,
                                            ld_dy=D, ld_hidden=D, ld_dhidden=D, ld_dx=D, ld_dresidual=D, rows=ROWS,
                                            d=D)),
    "route": (AdaRouteArgs, dict(logits=MB, valid=2 * MB, idx=3 * MB, gate=4 * MB, counts=5 * MB, prob=6 * MB,
                                 loss=7 * MB, used=8 * MB, ld_logits=E, rows=ROWS, E=E, k=K, renorm=1)),
    "route_backward": (AdaRouteGradArgs, dict(logits=MB, idx=2 * MB, gate=3 * MB, counts=4 * MB, used=5 * MB,
                                              dgate=6 * MB, dloss=7 * MB, dlogits=8 * MB, ld_logits=E, ld_dlogits=E,
                                              rows=ROWS, E=E, k=K, renorm=1)),
}
REQUIRED = {"dropout": ("x", "y"), "dropout_backward": ("dy", "dx"), "norm": ("x", "y"),
            "norm_backward": ("dy", "hidden", "mean", "rstd"), "route": ("logits", "idx", "gate"),
            "route_backward": ("logits", "idx", "gate", "counts", "used", "dlogits")}
OUTPUTS = {"dropout": ("y",), "dropout_backward": ("dx",), "norm": ("y", "hidden", "mean", "rstd"),
           "norm_backward": ("dx", "dresidual", "dweight", "dbias"),
           "route": ("idx", "gate", "counts", "prob", "loss", "used"), "route_backward": ("dlogits",)}
# outputs that may be an input itself
SAME = {"dropout": {("y", "x"), ("y", "residual")}, "dropout_backward": {("dx", "dy")},
        "norm": {("y", "x"), ("y", "residual"), ("hidden", "x"), ("hidden", "residual")},
        "norm_backward": {("dx", "dy"), ("dx", "dhidden"), ("dresidual", "dy"), ("dresidual", "dhidden")},
        "route": set(), "route_backward": set()}
MATRICES = {"dropout": ("x", "residual", "y"), "dropout_backward": ("dy", "dx"), "norm": ("x", "residual", "y", "hidden"),
            "norm_backward": ("dy", "hidden", "dhidden", "dx", "dresidual"), "route": (), "route_backward": ()}
LAYER = [n for n in SETS if not n.startswith("route")]
ROUTE = [n for n in SETS if n.startswith("route")]


def call(name, dt=ADA_BF16, ws=64 * MB, ws_bytes=1 << 30, p=0.1, state=None, **kw):
    cls, good = SETS[name]
    drop = dict(p=p, seed=1, offset=2, state=state) if name in LAYER else {}
    args = cls(**dict(good, **drop, **kw))
    space = (ws, ws_bytes) if name in ("norm_backward", "route") else ()
    return getattr(_lib.load(), f"ada_{name}")(args, dt, *space, None)


def pointers(name):
    return [f for f, t in SETS[name][0]._fields_ if t is _lib.c_void_p and f != "state"]


def strides(name):
    return [f for f in SETS[name][1] if f.startswith("ld_")]


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_good_calls_pass_the_checks(name):
    """They end at the first HIP call, there being no GPU."""
    assert call(name) == ADA_EHIP
    assert call(name, dt=ADA_F32) == ADA_EHIP
    for out, source in SAME[name]:
        assert call(name, **{out: SETS[name][1][source]}) == ADA_EHIP, (out, source)


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_refusals(name):
    space = (None, 0) if name in ("norm_backward", "route") else ()
    assert getattr(_lib.load(), f"ada_{name}")(None, ADA_BF16, *space, None) == ADA_EINVAL
    for p in REQUIRED[name]:
        assert call(name, **{p: None}) == ADA_EINVAL, p
    for dt in (-1, 2):
        assert call(name, dt=dt) == ADA_EDTYPE
    assert call(name, rows=-1) == ADA_ESHAPE
    assert call(name, rows=(1 << 22) + 1) == ADA_ESHAPE
    good = SETS[name][1]
    for ld in strides(name):
        assert call(name, **{ld: good[ld] - 8}) == ADA_ESHAPE, ld
        assert call(name, **{ld: (1 << 36) + 8}) == ADA_ESHAPE, ld
    for p in pointers(name):
        assert call(name, **{p: good[p] + 2}) in ((ADA_EALIGN,) if p not in ("logits", "valid", "dlogits") else (ADA_EHIP,)), p
        if p in ("logits", "dlogits"):
            assert call(name, dt=ADA_F32, **{p: good[p] + 2}) == ADA_EALIGN


@no_gpu
@pytest.mark.parametrize("name", LAYER)
def test_refusals_of_sizes_and_dropout(name):
    for d in (0, -8, 4, 60, (1 << 22) + 8):
        assert call(name, d=d) == ADA_ESHAPE
    if name.startswith("norm"):
        big = {ld: 32768 + 8 for ld in strides(name)}
        assert call(name, d=32768 + 8, **big) == ADA_ESHAPE
    good = SETS[name][1]
    for ld in strides(name):
        assert call(name, **{ld: good[ld] + 4}) == ADA_EALIGN, ld   # 8 bytes off in bf16
        assert call(name, dt=ADA_F32, **{ld: good[ld] + 2}) == ADA_EALIGN, ld
    for m in MATRICES[name]:
        assert call(name, **{m: good[m] + 8}) == ADA_EALIGN, m
    for p in (-0.1, 1.0000001, float("nan"), float("inf")):
        assert call(name, p=p) == ADA_EINVAL
    assert call(name, state=60 * MB + 4) == ADA_EALIGN
    for o in OUTPUTS[name]:
        assert call(name, state=good[o]) == ADA_EINVAL, o


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_overlaps_are_refused(name):
    good = SETS[name][1]
    for o in OUTPUTS[name]:
        for p in pointers(name):
            if p == o or (o, p) in SAME[name]:
                continue
            assert call(name, **{o: good[p]}) == ADA_EINVAL, (o, p)
    for o, p in SAME[name]:  # the same matrix, but not one that is shifted or has other rows
        assert call(name, **{o: good[p] + 16}) == ADA_EINVAL
        ld = next(l for l in strides(name) if l == "ld_" + ("res" if o == "residual" else o))
        assert call(name, **{o: good[p], ld: D + 8}) == ADA_EINVAL
    if name == "norm":  # neighbours are no overlap
        assert call(name, mean=good["rstd"] - 4 * ROWS) == ADA_EHIP
        assert call(name, mean=good["rstd"] - 4 * ROWS + 4) == ADA_EINVAL


@no_gpu
def test_outputs_that_may_not_be_one():
    good = SETS["norm"][1]
    assert call("norm", y=good["x"], hidden=good["x"]) == ADA_EINVAL
    assert call("norm", y=good["x"], hidden=good["residual"]) == ADA_EHIP
    good = SETS["norm_backward"][1]
    assert call("norm_backward", dx=good["dy"], dresidual=good["dy"]) == ADA_EINVAL
    assert call("norm_backward", dx=good["dy"], dresidual=good["dhidden"]) == ADA_EHIP


@no_gpu
def test_norm_refusals():
    for name in ("norm", "norm_backward"):
        assert call(name, kind=2) == ADA_EINVAL and call(name, kind=-1) == ADA_EINVAL
    assert call("norm", eps=-1e-9) == ADA_EINVAL
    assert call("norm", eps=float("nan")) == ADA_EINVAL
    # what a root-mean-square norm does not touch is not looked at
    assert call("norm", kind=ADA_NORM_RMS, mean=3) == ADA_EHIP
    assert call("norm_backward", kind=ADA_NORM_RMS, mean=None) == ADA_EHIP
    assert call("norm_backward", **{o: None for o in OUTPUTS["norm_backward"]}) == ADA_EINVAL
    for o in OUTPUTS["norm_backward"]:  # any one of them will do
        assert call("norm_backward", **{q: None for q in OUTPUTS["norm_backward"] if q != o}) == ADA_EHIP


@no_gpu
@pytest.mark.parametrize("name", ROUTE)
def test_route_refusals(name):
    for e in (0, -1, 65):
        assert call(name, E=e, ld_logits=128) == ADA_ESHAPE
    for k in (0, -1, E + 1):
        assert call(name, k=k) == ADA_ESHAPE
    for r in (-1, 2):
        assert call(name, renorm=r) == ADA_EINVAL
    if name == "route":
        for o in ("counts", "prob", "loss", "used"):
            assert call(name, **{o: None}) == ADA_EINVAL, o
        assert call(name, counts=None, prob=None, loss=None, used=None, ws=None, ws_bytes=0) == ADA_EHIP
    else:
        assert call(name, dgate=None, dloss=None) == ADA_EINVAL
        assert call(name, dgate=None, gate=None) == ADA_EHIP
        assert call(name, renorm=0, gate=None) == ADA_EHIP
        assert call(name, dloss=None, counts=None, used=None) == ADA_EHIP


@no_gpu
def test_workspace_refusals():
    lib = _lib.load()
    f = lib.ada_norm_backward_workspace
    assert f(-1, D, ADA_BF16) == ADA_ESHAPE and f(ROWS, 12, ADA_BF16) == ADA_ESHAPE and f(ROWS, D, 7) == ADA_EDTYPE
    assert f(0, D, ADA_F32) == 0
    for rows, d in ((1, 8), (ROWS, D), (5000, 8192), (1 << 20, 32768)):
        for dt in (ADA_F32, ADA_BF16):
            assert 0 <= f(rows, d, dt) <= 2 * 4 * d * 256  # a bounded number of partial sums
    assert f(ROWS, D, ADA_BF16) == 0  # few rows need none
    assert call("norm_backward", ws=None, ws_bytes=0) == ADA_EHIP
    assert call("norm_backward", ws=64 * MB + 8) == ADA_EALIGN
    rows = 5000
    far = {p: (i + 1) << 34 for i, p in enumerate(pointers("norm_backward"))}
    need = f(rows, D, ADA_BF16)
    assert need > 0
    assert call("norm_backward", rows=rows, ws=None, **far) == ADA_EINVAL
    assert call("norm_backward", rows=rows, ws=1 << 40, ws_bytes=need - 1, **far) == ADA_ESHAPE
    assert call("norm_backward", rows=rows, ws=1 << 40, ws_bytes=need, **far) == ADA_EHIP
    for p in far:
        assert call("norm_backward", rows=rows, **dict(far, ws=far[p])) == ADA_EINVAL, p
    g = lib.ada_route_workspace
    assert g(-1, E) == ADA_ESHAPE and g(ROWS, 0) == ADA_ESHAPE and g(ROWS, 65) == ADA_ESHAPE
    assert g(0, 64) == 0 and g(1, 1) == 0
    rows = 1 << 20
    far = {p: (i + 1) << 34 for i, p in enumerate(pointers("route"))}
    need = g(rows, E)
    assert need > 0
    assert call("route", rows=rows, ws=None, **far) == ADA_EINVAL
    assert call("route", rows=rows, ws=1 << 40, ws_bytes=need - 1, **far) == ADA_ESHAPE
    assert call("route", rows=rows, ws=1 << 40, ws_bytes=need, **far) == ADA_EHIP
    assert call("route", rows=rows, ws=far["idx"], **far) == ADA_EINVAL


@no_gpu
@pytest.mark.parametrize("name", [n for n in SETS if n not in ("norm_backward", "route")])
def test_no_rows_is_no_work(name):
    assert call(name, **dict({p: None for p in pointers(name)}, rows=0)) == 0


@no_gpu
def test_interleaved_columns_pass_the_checks():
    """x, residual, hidden and y as column ranges of the same rows."""
    ld = 4 * D
    at = dict(x=MB, residual=MB + D * 2, hidden=MB + 2 * D * 2, y=MB + 3 * D * 2)
    lds = {n: ld for n in strides("norm")}
    assert call("norm", **at, **lds) == ADA_EHIP
    assert call("norm", **dict(at, y=at["y"] - 16), **lds) == ADA_EINVAL


def test_python_refusals():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    for f in (lambda **kw: A.ada_norm(x, w, **kw), lambda **kw: A.ada_dropout(x, 0.1, 0, **kw)):
        with pytest.raises(ValueError, match="device"):
            f()
        with pytest.raises(ValueError, match=r"residual must be \[4, 16\]"):
            f(residual=torch.zeros(4, 8))
        with pytest.raises(TypeError, match="residual must be torch.float32"):
            f(residual=torch.zeros(4, 16, dtype=torch.bfloat16))
        with pytest.raises(ValueError, match="unit column stride"):
            f(residual=torch.zeros(16, 4).t())
    with pytest.raises(ValueError, match="unknown norm"):
        A.ada_norm(x, w, kind="batch")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        A.ada_norm(x.half(), w)
    with pytest.raises(TypeError, match="mean must be torch.float32"):
        A.ada_norm(x, stats=(torch.zeros(4, dtype=torch.float64), torch.zeros(4)))
    with pytest.raises(ValueError, match=r"must be \[rows, d\]"):
        A.ada_norm(torch.zeros(16), w)
    with pytest.raises(TypeError, match="seed on the device"):
        A.ada_dropout(x, 0.1, torch.zeros(2))
    with pytest.raises(TypeError, match="seed on the device"):
        A.ada_dropout(x, 0.1, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="needs a seed"):
        A.ada_norm(x, w, p=0.1)
    with pytest.raises(ValueError, match="needs a seed"):
        A.ada_dropout(x, float("nan"), None)
    with pytest.raises(ValueError, match="stats must hold"):
        A.ada_norm_backward(x, x, (None, torch.zeros(4)), w)
    z, out = torch.zeros(4, 6), (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), None, None, None, None)
    with pytest.raises(TypeError, match="bool or uint8"):
        A.ada_route(z, 2, valid=torch.zeros(4), out=out)
    with pytest.raises(ValueError, match=r"valid must be \[4\]"):
        A.ada_route(z, 2, valid=torch.zeros(5, dtype=torch.bool), out=out)
    with pytest.raises(ValueError, match=r"idx must be \[4, 3\]"):
        A.ada_route(z, 3, out=out)
    with pytest.raises(ValueError, match="dgate or dloss"):
        A.ada_route_backward(z, out)
    with pytest.raises(ValueError, match="without balance"):
        A.ada_route_backward(z, out, dloss=torch.zeros(1))
    with pytest.raises(ValueError, match="gate must be contiguous"):
        A.ada_route_backward(z, (out[0], torch.zeros(2, 4).t(), None, None, None, None), dgate=torch.zeros(4, 2))


# ---- the oracle ------------------------------------------------------------------------
def test_generator_gives_the_published_numbers():
    """Known answers of Philox4x32-10, printed with the generator's publication."""
    def words(counter, key):
        return OL.philox4x32(np.array([counter], np.uint32), key)[0].tolist()

    ones = 0xFFFFFFFF
    assert words((0,) * 4, (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words((ones,) * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("p", (0.0, 2.0 ** -17, 0.1, 0.5, 0.999, 1.0))
def test_kept_share_and_scale(p):
    kept, scale = OL.dropout_mask(400, 2048, p, 5, 9)
    share = 1 - np.rint(65536 * p) / 65536
    # six standard deviations of a binomial share
    assert abs(kept.mean() - share) <= 6 * math.sqrt(share * (1 - share) / kept.size)
    assert scale == (1 / share if share else 0)


def test_masks_differ_between_rows_seeds_and_offsets():
    a = OL.dropout_numbers(8, 64, 1, 1)
    assert np.array_equal(OL.dropout_numbers(3, 64, 1, 1, first_row=5), a[5:])
    for other in (OL.dropout_numbers(8, 64, 2, 1), OL.dropout_numbers(8, 64, 1, 2),
                  OL.dropout_numbers(8, 64, 1 + 2 ** 32, 1), OL.dropout_numbers(8, 64, 1, 1 + 2 ** 32)):
        assert (other == a).mean() < 0.05


@pytest.mark.parametrize("kind", ("layer", "rms"))
def test_norm_gradient_against_differences(kind):
    g = np.random.default_rng(3)
    h, w, b, dy = g.normal(size=(3, 8)), 1 + 0.2 * g.normal(size=8), g.normal(size=8), g.normal(size=(3, 8))
    dhidden = g.normal(size=(3, 8))

    def value(h, w, b):
        return np.sum(OL.norm(h, w, b, kind, 1e-3)[0] * dy) + np.sum(h * dhidden)

    _, mean, rstd = OL.norm(h, w, b, kind, 1e-3)
    dh, dw, db = OL.norm_backward(dy, h, mean, rstd, w, dhidden, kind)
    step = 1e-5
    for at, grad in ((h, dh), (w, dw), (b, db)):
        for i in np.ndindex(at.shape):
            keep = at[i]
            at[i] = keep + step
            up = value(h, w, b)
            at[i] = keep - step
            down = value(h, w, b)
            at[i] = keep
            assert abs((up - down) / (2 * step) - grad[i]) <= 1e-6 * (1 + abs(grad[i]))


@pytest.mark.parametrize("renorm", (True, False))
def test_route_gradient_against_differences(renorm):
    g = np.random.default_rng(4)
    z = g.normal(size=(6, 5))
    z[1, 2] = z[2] = -np.inf
    valid = np.array([1, 1, 1, 0, 1, 1], bool)
    dgate, dloss = g.normal(size=(6, 3)), 0.7
    idx, gate, counts, prob, loss, used = OL.route(z, 3, renorm, valid)
    assert used == 4 and (idx[2] == -1).all() and (idx[3] == -1).all() and counts.sum() == 12
    dz = OL.route_backward(z, idx, gate, counts, used, dgate, dloss, renorm)

    def value():  # away from ties the picks, and so the counts, do not move
        i, gt, _, pr, _, _ = OL.route(z, 3, renorm, valid)
        assert np.array_equal(i, idx)
        return np.sum(gt * dgate) + dloss * 5 * np.sum(counts / (3 * used) * pr)

    step = 1e-6
    for i in np.ndindex(z.shape):
        if z[i] == -np.inf:
            assert dz[i] == 0
            continue
        keep = z[i]
        z[i] = keep + step
        up = value()
        z[i] = keep - step
        down = value()
        z[i] = keep
        assert abs((up - down) / (2 * step) - dz[i]) <= 1e-7 * (1 + abs(dz[i]))


def test_even_load_has_loss_one():
    z = np.full((8, 4), 0.0)
    z[np.arange(8), np.arange(8) % 4] = 1.0
    assert abs(OL.route(z, 1, True)[4] - 1.0) < 1e-12
