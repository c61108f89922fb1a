"""Refusals of the linear and gated product calls (argument checks run on the host before
any HIP call), and the oracle's gradients against differences.  No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import linear as OL
from weight_merge_amd import _lib
from weight_merge_amd import api as A
from weight_merge_amd._lib import (ADA_ACT_GELU, ADA_ACT_NONE, ADA_ACT_SILU, ADA_BF16, ADA_EALIGN, ADA_EDTYPE,
                                   ADA_EINVAL, ADA_ESHAPE, ADA_F32, AdaGluArgs, AdaGluGradArgs, AdaLinearArgs,
                                   AdaLinearGradArgs)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: runs where no GPU is visible")

MB = 1 << 20
ROWS, N, K = 40, 64, 128
# fake, aligned, far-apart addresses: every call below fails before it could touch them
SETS = {
    "linear": (AdaLinearArgs, dict(x=MB, w=2 * MB, bias=3 * MB, residual=4 * MB, y=5 * MB, pre=6 * MB, ld_x=K, ld_w=K,
                                   ld_res=N, ld_y=N, ld_pre=N)),
    "linear_backward": (AdaLinearGradArgs, dict(dy=MB, x=2 * MB, w=3 * MB, pre=4 * MB, dx=5 * MB, dw=6 * MB,
                                                dbias=7 * MB, ld_dy=N, ld_x=K, ld_w=K, ld_pre=N, ld_dx=K, ld_dw=K)),
    "glu": (AdaGluArgs, dict(x=MB, w_gate=2 * MB, w_up=3 * MB, bias_gate=4 * MB, bias_up=5 * MB, y=6 * MB,
                             gate_pre=7 * MB, up_pre=8 * MB, ld_x=K, ld_w_gate=K, ld_w_up=K, ld_y=N, ld_gate_pre=N,
                             ld_up_pre=N)),
    "glu_backward": (AdaGluGradArgs, dict(dy=MB, x=2 * MB, w_gate=3 * MB, w_up=4 * MB, gate_pre=5 * MB, up_pre=6 * MB,
                                          dx=7 * MB, dw_gate=8 * MB, dw_up=9 * MB, dbias_gate=10 * MB,
                                          dbias_up=11 * MB, ld_dy=N, ld_x=K, ld_w_gate=K, ld_w_up=K, ld_gate_pre=N,
                                          ld_up_pre=N, ld_dx=K, ld_dw_gate=K, ld_dw_up=K)),
}
REQUIRED = {"linear": ("x", "w", "y"), "linear_backward": ("dy", "x", "w", "pre"), "glu": ("x", "w_gate", "w_up", "y"),
            "glu_backward": ("dy", "x", "w_gate", "w_up", "gate_pre", "up_pre")}
OUTPUTS = {"linear": ("y", "pre"), "linear_backward": ("dx", "dw", "dbias"), "glu": ("y", "gate_pre", "up_pre"),
           "glu_backward": ("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")}


def need(name, act=ADA_ACT_SILU, rows=ROWS, n=N, k=K, dt=ADA_BF16):
    f = getattr(_lib.load(), f"ada_{name}_workspace")
    return f(rows, n, k, act, dt) if name.endswith("backward") else f(rows, n, k, dt)


def call(name, act=ADA_ACT_SILU, dt=ADA_BF16, ws=64 * MB, ws_bytes=None, rows=ROWS, n=N, k=K, **kw):
    cls, good = SETS[name]
    args = cls(**dict(good, rows=rows, d_out=n, d_in=k, **kw))
    return getattr(_lib.load(), f"ada_{name}")(args, act, dt, ws, 1 << 30 if ws_bytes is None else ws_bytes, None)


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_refusals(name):
    assert getattr(_lib.load(), f"ada_{name}")(None, 0, ADA_BF16, None, 0, None) == ADA_EINVAL
    for p in REQUIRED[name]:
        assert call(name, **{p: None}) == ADA_EINVAL, p
    for act in (-1, 5):
        assert call(name, act=act) == ADA_EINVAL
    for dt in (-1, 2):
        assert call(name, dt=dt) == ADA_EDTYPE
    assert call(name, rows=-1) == ADA_ESHAPE
    assert call(name, rows=(1 << 22) + 1) == ADA_ESHAPE
    for d in (0, -8, 4, 60, (1 << 22) + 8):
        assert call(name, n=d) == ADA_ESHAPE
        assert call(name, k=d) == ADA_ESHAPE
    for p, v in SETS[name][1].items():
        if p.startswith("ld_"):
            assert call(name, **{p: v - 8}) == ADA_ESHAPE, p     # shorter than the row
            assert call(name, **{p: v + 4}) == ADA_EALIGN, p     # 8 bytes off in bf16
            assert call(name, dt=ADA_F32, **{p: v + 2}) == ADA_EALIGN, p
            assert call(name, **{p: (1 << 36) + 8}) == ADA_ESHAPE, p
        else:
            assert call(name, **{p: v + 4}) == ADA_EALIGN, p
    assert call(name, ws=64 * MB + 8) == ADA_EALIGN


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_overlaps_are_refused(name):
    good = SETS[name][1]
    ptrs = [p for p in good if not p.startswith("ld_")]
    for o in OUTPUTS[name]:
        for p in ptrs:
            if p == o or (name, p, o) == ("linear", "residual", "y"):
                continue
            assert call(name, **{o: good[p]}) == ADA_EINVAL, (o, p)
    if name == "linear":  # the residual in place is fine (refused for another reason here); shifted it is not
        assert call(name, y=4 * MB, act=9) == ADA_EINVAL
        assert call(name, y=4 * MB + 16) == ADA_EINVAL
        assert call(name, y=4 * MB, ld_y=N + 8) == ADA_EINVAL
        assert call(name, pre=4 * MB) == ADA_EINVAL


@no_gpu
@pytest.mark.parametrize("name", [n for n in SETS if n.endswith("backward")])
def test_backward_asks_for_something(name):
    assert call(name, **{o: None for o in OUTPUTS[name]}) == ADA_EINVAL


@no_gpu
@pytest.mark.parametrize("name", SETS)
def test_workspace_refusals(name):
    f = getattr(_lib.load(), f"ada_{name}_workspace")
    tail = (ADA_ACT_SILU, ADA_BF16) if name.endswith("backward") else (ADA_BF16,)
    assert f(-1, N, K, *tail) == ADA_ESHAPE
    assert f(ROWS, 12, K, *tail) == ADA_ESHAPE
    assert f(ROWS, N, 0, *tail) == ADA_ESHAPE
    assert f(ROWS, N, K, *tail[:-1], 7) == ADA_EDTYPE
    if name.endswith("backward"):
        assert f(ROWS, N, K, 8, ADA_BF16) == ADA_EINVAL
    for rows, n, k in ((ROWS, N, K), (200, 4096, 4096), (1, 64, 1 << 16)):
        for dt in (ADA_F32, ADA_BF16):
            b = need(name, rows=rows, n=n, k=k, dt=dt)
            assert b >= 0
            if b:
                big = dict(rows=rows, n=n, k=k, dt=dt)
                # far-apart operands for the larger sizes
                for i, p in enumerate(q for q in SETS[name][1] if not q.startswith("ld_")):
                    big[p] = (i + 1) << 34
                for p in SETS[name][1]:
                    if p.startswith("ld_"):
                        big[p] = max(n, k)
                assert call(name, ws=None, **big) == ADA_EINVAL
                assert call(name, ws=1 << 40, ws_bytes=b - 1, **big) == ADA_ESHAPE
                assert call(name, ws=big[next(iter(SETS[name][1]))], ws_bytes=b, **big) == ADA_EINVAL


@no_gpu
def test_interleaved_column_ranges_pass_the_checks():
    """Column ranges of one buffer's rows do not overlap: the call gets past its checks (and
    then fails at the first HIP call, there being no GPU)."""
    e = 2
    ld = K + 3 * N
    base = MB
    st = call("glu", x=base, ld_x=ld, y=base + K * e, ld_y=ld, gate_pre=base + (K + N) * e, ld_gate_pre=ld,
              up_pre=base + (K + 2 * N) * e, ld_up_pre=ld)
    assert st == _lib.ADA_EHIP
    assert call("glu", x=base, ld_x=ld, y=base + K * e - 16, ld_y=ld) == ADA_EINVAL
    assert call("glu", x=base, ld_x=ld, y=base + K * e, ld_y=ld, gate_pre=base + (K + N) * e - 16,
                ld_gate_pre=ld) == ADA_EINVAL
    # the same the other way round, whole rows down
    assert call("glu", y=base, ld_y=ld, x=base + (5 * ld + N) * e, ld_x=ld) == _lib.ADA_EHIP
    assert call("glu", y=base, ld_y=ld, x=base + (5 * ld + N) * e - 16, ld_x=ld) == ADA_EINVAL


@no_gpu
def test_residual_in_place_passes_the_checks():
    assert call("linear", y=4 * MB) == _lib.ADA_EHIP


@no_gpu
def test_no_rows_needs_no_matrices():
    z = dict(rows=0, ws=None, ws_bytes=0)
    assert call("linear", x=None, y=None, residual=None, pre=None, **z) == 0
    assert call("glu", x=None, y=None, gate_pre=None, up_pre=None, **z) == 0


def cpu(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def test_python_refusals():
    x, w = cpu(4, 64), cpu(32, 64)
    with pytest.raises(ValueError, match="unknown activation"):
        A.ada_linear(x, w, act="swish")
    with pytest.raises(TypeError, match="unsupported dtype"):
        A.ada_linear(x.half(), w.half())
    with pytest.raises(ValueError, match=r"x must be \[rows, d_in\]"):
        A.ada_linear(x[0], w)
    with pytest.raises(ValueError, match=r"x must be \[4, 72\]"):
        A.ada_linear(x, cpu(32, 72))
    with pytest.raises(TypeError, match="w must be torch.bfloat16"):
        A.ada_linear(x, w.float())
    with pytest.raises(ValueError, match=r"bias must be \[32\]"):
        A.ada_linear(x, w, bias=cpu(64))
    with pytest.raises(ValueError, match=r"residual must be \[4, 32\]"):
        A.ada_linear(x, w, residual=cpu(4, 64))
    with pytest.raises(ValueError, match="unit column stride"):
        A.ada_linear(cpu(64, 4).t(), w)
    with pytest.raises(ValueError, match="contiguous"):
        A.ada_linear(x, w, bias=cpu(64)[::2])
    with pytest.raises(ValueError, match="on the device"):
        A.ada_linear(x, w)
    with pytest.raises(ValueError, match="on the device"):
        A.ada_glu(x, w, w)
    with pytest.raises(ValueError, match="w_up must be"):
        A.ada_glu(x, w, cpu(40, 64))
    with pytest.raises(ValueError, match="gate_pre must be"):
        A.ada_glu(x, w, w, pre=(cpu(4, 64), cpu(4, 32)))
    with pytest.raises(ValueError, match="pre is needed"):
        A.ada_linear_backward(cpu(4, 32), x, w, act="gelu")
    with pytest.raises(ValueError, match="dy must be"):
        A.ada_linear_backward(cpu(4, 64), x, w)
    with pytest.raises(ValueError, match="dw must be"):
        A.ada_linear_backward(cpu(4, 32), x, w, dw=cpu(64, 32))
    with pytest.raises(ValueError, match="are needed"):
        A.ada_glu_backward(cpu(4, 32), x, w, w, None, None)
    with pytest.raises(ValueError, match="dbias_up must be"):
        A.ada_glu_backward(cpu(4, 32), x, w, w, cpu(4, 32), cpu(4, 32), dbias_up=cpu(64))


def test_workspace_queries_from_python():
    for f, extra in ((A.linear_workspace_bytes, ()), (A.glu_workspace_bytes, ()),
                     (A.linear_backward_workspace_bytes, ("silu",)), (A.glu_backward_workspace_bytes, ("silu",))):
        assert f(1, 64, 64, *extra, torch.bfloat16) >= 0
        with pytest.raises(A.AdaError):
            f(1, 60, 64, *extra, torch.bfloat16)


@pytest.mark.parametrize("act", ("none", "relu", "silu", "gelu", "gelu_tanh"))
def test_oracle_gradients_against_differences(act):
    """Central differences in 64 bits: off by e^2 / 6 of the third derivative (below 10 for
    these functions and inputs) and 1e-16 / e of the loss, e = 1e-5: 1e-8 covers both with a
    loss of at most ~100.  relu's kink: no input lies within e of it."""
    rng = np.random.default_rng(3)
    rows, n, k = 5, 8, 6
    x, w, w2 = rng.normal(size=(rows, k)), rng.normal(size=(n, k)), rng.normal(size=(n, k))
    b, b2, dy = rng.normal(size=n), rng.normal(size=n), rng.normal(size=(rows, n))
    z = OL.linear(x, w, b)[1]
    assert np.abs(z).min() > 1e-3 and np.abs(OL.glu(x, w, w2, b, b2)[1]).min() > 1e-3

    def check(loss, leaf, grad):
        for _ in range(6):
            v = rng.normal(size=leaf.shape)
            v /= np.linalg.norm(v)
            e = 1e-5
            assert abs((loss(leaf + e * v) - loss(leaf - e * v)) / (2 * e) - (grad * v).sum()) < 1e-8

    dx, dw, db, _ = OL.linear_backward(dy, x, w, z, act)
    check(lambda t: (dy * OL.linear(t, w, b, None, act)[0]).sum(), x, dx)
    check(lambda t: (dy * OL.linear(x, t, b, None, act)[0]).sum(), w, dw)
    check(lambda t: (dy * OL.linear(x, w, t, None, act)[0]).sum(), b, db)
    _, g, u = OL.glu(x, w, w2, b, b2, act)
    dx, dwg, dwu, dbg, dbu, _, _ = OL.glu_backward(dy, x, w, w2, g, u, act)
    check(lambda t: (dy * OL.glu(t, w, w2, b, b2, act)[0]).sum(), x, dx)
    check(lambda t: (dy * OL.glu(x, t, w2, b, b2, act)[0]).sum(), w, dwg)
    check(lambda t: (dy * OL.glu(x, w, t, b, b2, act)[0]).sum(), w2, dwu)
    check(lambda t: (dy * OL.glu(x, w, w2, t, b2, act)[0]).sum(), b, dbg)
    check(lambda t: (dy * OL.glu(x, w, w2, b, t, act)[0]).sum(), b2, dbu)


def test_none_backward_ignores_pre():
    """Without an activation z is not read: a pre of another shape is not looked at."""
    with pytest.raises(ValueError, match="on the device"):
        A.ada_linear_backward(cpu(4, 32), cpu(4, 64), cpu(32, 64), pre=cpu(1, 1), act="none")
    assert ADA_ACT_NONE == 0 and ADA_ACT_GELU == 3 and ctypes.sizeof(AdaLinearArgs) == 104


EXTREMES = [(1 << 22, 8, 8), (8, 1 << 22, 8), (8, 8, 1 << 22), (1, 1 << 22, 1 << 13), (1 << 22, 1 << 13, 1 << 13),
            (1 << 13, 1 << 22, 1 << 13), (1 << 13, 1 << 13, 1 << 22), (1 << 17, 1 << 18, 1 << 17), ((1 << 22) - 1, 8184, 8184),
            (33, (1 << 22) - 8, 8), (48, 8192, 1 << 22), (32, 1 << 22, 8192), (64, 1 << 22, 8192), (1 << 22, 8, 8192)]


@pytest.mark.parametrize("rows, n, k", EXTREMES)
def test_workspaces_at_the_largest_sizes(rows, n, k):
    """The plan of the largest rows, dimensions and matrices that are admitted: found, and no larger
    than dz, its column sums and the parts of splits into 128 at most."""
    lib = _lib.load()
    for dt, e in ((ADA_F32, 4), (ADA_BF16, 2)):
        for gated in (1, 2):
            names = ("linear", "glu")[gated - 1]
            forward = getattr(lib, f"ada_{names}_workspace")(rows, n, k, dt)
            assert 0 <= forward <= 16 * 4 * rows * n * gated
            for act in (ADA_ACT_NONE, ADA_ACT_GELU):
                b = getattr(lib, f"ada_{names}_backward_workspace")(rows, n, k, act, dt)
                dz = rows * n * gated * e if gated == 2 or act != ADA_ACT_NONE else 0
                assert dz <= b <= dz + (rows // 64 + 1) * n * gated * 4 + 128 * 4 * (rows + gated * n) * k + 1024


@pytest.mark.parametrize("rows, n, k", [((1 << 22) + 1, 8, 8), (1, (1 << 22) + 8, 8), (1, 8, (1 << 22) + 8),
                                        (1 << 22, 8200, 8), (1 << 22, 8, 8200), (1, 1 << 22, 8200)])
def test_larger_sizes_are_refused(rows, n, k):
    lib = _lib.load()
    for dt in (ADA_F32, ADA_BF16):
        assert lib.ada_linear_workspace(rows, n, k, dt) == ADA_ESHAPE
        assert lib.ada_glu_workspace(rows, n, k, dt) == ADA_ESHAPE
        assert lib.ada_linear_backward_workspace(rows, n, k, ADA_ACT_NONE, dt) == ADA_ESHAPE
        assert lib.ada_glu_backward_workspace(rows, n, k, ADA_ACT_SILU, dt) == ADA_ESHAPE
