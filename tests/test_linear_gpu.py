"""The linear and gated feed-forward products and their backward passes against the fp64
oracle, element by element, within bounds derived from the arithmetic (linear_helpers)."""
import numpy as np
import pytest
import torch

import linear_helpers as H
from oracle import linear as OL
from weight_merge_amd import api as A

DEV = "cuda"
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
# (rows, d_out, d_in): one row; row counts around every tile edge; d_out and d_in from the
# smallest to past a tile, on and off the step depth (64 bf16 or 32 fp32 elements of k)
SHAPES = [(1, 8, 8), (1, 264, 520), (2, 72, 136), (3, 1032, 64), (7, 136, 1032), (15, 24, 2056), (16, 512, 256),
          (17, 264, 264), (31, 8, 4096), (33, 520, 72), (48, 1288, 328), (63, 64, 64), (65, 136, 1000),
          (100, 2056, 8), (127, 256, 512), (129, 392, 264), (255, 128, 520), (257, 264, 136), (300, 1032, 520),
          (513, 520, 1032), (700, 8, 72)]
FEW = [(1, 264, 520), (5, 136, 72), (33, 520, 264), (129, 264, 1032), (300, 72, 136)]


def inputs(seed, rows, d_out, d_in, dtype, parts=1, bias=True, pad=0):
    t = {"x": H.normal(seed, (rows, d_in), 1.0, dtype)}
    for h in range(parts):
        t[f"w{h}"] = H.normal(seed + 10 + h, (d_out, d_in), d_in ** -0.5, dtype)
        t[f"b{h}"] = H.normal(seed + 20 + h, (d_out,), 0.5, dtype) if bias else None
    t["res"] = H.normal(seed + 30, (rows, d_out), 1.0, dtype)
    t["dy"] = H.normal(seed + 31, (rows, d_out), 0.3, dtype)
    dev = {k: None if v is None else H.strided(v, DEV, pad) for k, v in t.items()}
    return {k: H.f64(v) for k, v in t.items()}, dev


def empty(rows, cols, dtype, pad=0):
    return torch.full((rows, cols + pad), float("nan"), dtype=H.TD[dtype], device=DEV)[:, :cols]


def check_linear(rows, d_out, d_in, dtype, act, bias=True, res=True, pre=True, pad=0, seed=0):
    n, d = inputs(seed, rows, d_out, d_in, dtype, bias=bias, pad=pad)
    y, p = empty(rows, d_out, dtype, pad), empty(rows, d_out, dtype, pad) if pre else None
    got = A.ada_linear(d["x"], d["w0"], bias=d["b0"], residual=d["res"] if res else None, act=act, y=y, pre=p)
    assert got is y
    r = n["res"] if res else None
    yref, zref = OL.linear(n["x"], n["w0"], n["b0"], r, act)
    by, bz = H.linear_bounds(n["x"], n["w0"], n["b0"], r, act, dtype)
    H.assert_within(y, yref, by, f"y {rows}x{d_out}x{d_in} {dtype} {act}")
    if pre:
        H.assert_within(p, zref, bz, "pre")
    if pad:
        assert y._base[:, d_out:].isnan().all(), "the gap between rows was written"


def check_glu(rows, d_out, d_in, dtype, act, bias=True, pre=True, pad=0, seed=0):
    n, d = inputs(seed, rows, d_out, d_in, dtype, parts=2, bias=bias, pad=pad)
    y = empty(rows, d_out, dtype, pad)
    g, u = empty(rows, d_out, dtype, pad), empty(rows, d_out, dtype)
    A.ada_glu(d["x"], d["w0"], d["w1"], bias_gate=d["b0"], bias_up=d["b1"], act=act, y=y, pre=(g, u) if pre else None)
    ref = OL.glu(n["x"], n["w0"], n["w1"], n["b0"], n["b1"], act)
    bounds = H.glu_bounds(n["x"], n["w0"], n["w1"], n["b0"], n["b1"], act, dtype)
    for t, r, b, what in list(zip((y, g, u), ref, bounds, ("y", "g", "u")))[: 3 if pre else 1]:
        H.assert_within(t, r, b, f"{what} {rows}x{d_out}x{d_in} {dtype} {act}")
    if pad:
        assert y._base[:, d_out:].isnan().all(), "the gap between rows was written"


def saved(seed, rows, d_out, dtype, pad):
    """A saved pre-activation: any stored values do (the backward pass takes them as given)."""
    t = H.normal(seed, (rows, d_out), 1.5, dtype)
    return H.f64(t), H.strided(t, DEV, pad)


def check_linear_backward(rows, d_out, d_in, dtype, act, pad=0, seed=0):
    n, d = inputs(seed, rows, d_out, d_in, dtype, pad=pad)
    zn, zd = saved(seed + 40, rows, d_out, dtype, pad)
    dx, dw = empty(rows, d_in, dtype, pad), empty(d_out, d_in, dtype, pad)
    db = torch.full((d_out,), float("nan"), dtype=H.TD[dtype], device=DEV)
    A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=zd, act=act, dx=dx, dw=dw, dbias=db)
    rx, rw, rb, rz = OL.linear_backward(n["dy"], n["x"], n["w0"], zn, act)
    bounds = H.grad_bounds([rz], [H.slope_error(n["dy"], zn, act)], n["x"], [n["w0"]], dtype)
    for t, r, b, what in zip((dx, dw, db), (rx, rw, rb), bounds, ("dx", "dw", "db")):
        H.assert_within(t, r, b, f"{what} {rows}x{d_out}x{d_in} {dtype} {act}")
    if pad:
        assert dx._base[:, d_in:].isnan().all() and dw._base[:, d_in:].isnan().all()


def check_glu_backward(rows, d_out, d_in, dtype, act, pad=0, seed=0):
    n, d = inputs(seed, rows, d_out, d_in, dtype, parts=2, pad=pad)
    gn, gd = saved(seed + 40, rows, d_out, dtype, pad)
    un, ud = saved(seed + 41, rows, d_out, dtype, 0)
    outs = [empty(rows, d_in, dtype, pad), empty(d_out, d_in, dtype, pad), empty(d_out, d_in, dtype)]
    outs += [torch.full((d_out,), float("nan"), dtype=H.TD[dtype], device=DEV) for _ in range(2)]
    A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], gd, ud, act=act, dx=outs[0], dw_gate=outs[1],
                       dw_up=outs[2], dbias_gate=outs[3], dbias_up=outs[4])
    *ref, dg, du = OL.glu_backward(n["dy"], n["x"], n["w0"], n["w1"], gn, un, act)
    ea = np.zeros_like(gn) if act in ("none", "relu") else H.act_error(gn, np.zeros_like(gn), act)
    edg = (H.slope_error(n["dy"], gn, act) + 3 * H.U * np.abs(n["dy"])) * np.abs(un) + 3 * H.U * np.abs(dg)
    edu = np.abs(n["dy"]) * ea + 2 * H.U * np.abs(du)
    bounds = H.grad_bounds([dg, du], [edg, edu], n["x"], [n["w0"], n["w1"]], dtype)
    for t, r, b, what in zip(outs, ref, bounds, ("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")):
        H.assert_within(t, r, b, f"{what} {rows}x{d_out}x{d_in} {dtype} {act}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_linear_shapes(shape, dtype):
    check_linear(*shape, dtype, "gelu", seed=sum(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_glu_shapes(shape, dtype):
    check_glu(*shape, dtype, "silu", seed=sum(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_linear_backward_shapes(shape, dtype):
    check_linear_backward(*shape, dtype, "silu", seed=sum(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_glu_backward_shapes(shape, dtype):
    check_glu_backward(*shape, dtype, "gelu_tanh", seed=sum(shape))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", FEW, ids=lambda s: "x".join(map(str, s)))
def test_activations_and_operands(shape, act, dtype):
    """Every activation with strided rows, and each optional operand left out."""
    pad = 8 if dtype == "bf16" else 4
    check_linear(*shape, dtype, act, pad=pad, seed=1)
    check_linear(*shape, dtype, act, bias=False, res=True, pre=False, seed=2)
    check_linear(*shape, dtype, act, bias=True, res=False, pre=False, seed=3)
    check_glu(*shape, dtype, act, pad=pad, seed=4)
    check_glu(*shape, dtype, act, bias=False, pre=False, seed=5)
    check_linear_backward(*shape, dtype, act, pad=pad, seed=6)
    check_glu_backward(*shape, dtype, act, pad=pad, seed=7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_no_rows(dtype):
    """No rows: the forward calls write nothing; gradients summed over rows are zeros."""
    n, d = inputs(3, 0, 72, 136, dtype, parts=2)
    assert A.ada_linear(d["x"], d["w0"], act="silu").shape == (0, 72)
    assert A.ada_glu(d["x"], d["w0"], d["w1"]).shape == (0, 72)
    none = torch.empty((0, 72), dtype=H.TD[dtype], device=DEV)
    dx, dw, db = A.ada_linear_backward(none, d["x"], d["w0"], pre=none, act="silu", want_dbias=True)
    assert dx.shape == (0, 136) and not dw.any() and not db.any()
    got = A.ada_glu_backward(none, d["x"], d["w0"], d["w1"], none, none, want_dbias=True)
    assert got[0].shape == (0, 136) and not any(t.any() for t in got[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 20, 150))
def test_wanted_gradients_alone(rows, dtype):
    """Each gradient asked for by itself equals the one of the full call; the others are None."""
    n, d = inputs(5, rows, 136, 264, dtype, parts=2)
    _, z = saved(6, rows, 136, dtype, 0)
    _, u = saved(7, rows, 136, dtype, 0)
    for act in ("none", "gelu"):
        full = A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act=act, want_dbias=True)
        for i in range(3):
            want = dict(zip(("want_dx", "want_dw", "want_dbias"), (i == 0, i == 1, i == 2)))
            got = A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act=act, **want)
            assert [t is None for t in got] == [j != i for j in range(3)]
            assert torch.equal(got[i], full[i]), (act, i)
    full = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, u, want_dbias=True)
    for i, want in enumerate(("want_dx", "want_dw", "want_dbias")):
        got = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, u,
                                 **{w: w == want for w in ("want_dx", "want_dw", "want_dbias")})
        for j, (a, b) in enumerate(zip(got, full)):
            assert a is None if (j + 1) // 2 != i else torch.equal(a, b)
    one = torch.empty_like(d["w1"])
    got = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, u, dw_up=one, want_dx=False, want_dw=False)
    assert got[0] is None and got[1] is None and torch.equal(one, full[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 9, 40, 200))
def test_rows_alone_change_nothing_else(rows, dtype):
    """NaN and infinities in one row of x stay in that row of y; NaN in a weight row stays in
    its column."""
    n, d = inputs(8, rows, 136, 264, dtype, parts=2)
    clean, cglu = A.ada_linear(d["x"], d["w0"], act="silu"), A.ada_glu(d["x"], d["w0"], d["w1"])
    x = d["x"].clone()
    x[rows - 1, 5] = float("nan")
    x[rows - 1, 200] = float("inf")
    w = d["w0"].clone()
    w[77, 3] = float("nan")
    for got, ref in ((A.ada_linear(x, w, act="silu"), clean), (A.ada_glu(x, w, d["w1"]), cglu)):
        assert got[rows - 1].isnan().all() and got[:, 77].isnan().all()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[rows - 1] = False
        keep[:, 77] = False
        assert torch.equal(got[keep], ref[keep])
    relu = A.ada_linear(x, w, act="relu")
    assert relu[rows - 1].isnan().all() and relu[:, 77].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 12, 77, 300))
def test_residual_in_place(rows, dtype):
    n, d = inputs(9, rows, 264, 136, dtype)
    ref = A.ada_linear(d["x"], d["w0"], residual=d["res"], act="gelu")
    y = d["res"].clone()
    assert A.ada_linear(d["x"], d["w0"], residual=y, act="gelu", y=y) is y
    assert torch.equal(y, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 24, 130))
def test_column_ranges_of_one_buffer(rows, dtype):
    """x, y and both saved matrices as column ranges of one buffer."""
    n, d = inputs(10, rows, 72, 136, dtype, parts=2)
    buf = torch.full((rows, 136 + 3 * 72), float("nan"), dtype=H.TD[dtype], device=DEV)
    buf[:, :136] = d["x"]
    y, g, u = (buf[:, 136 + 72 * i: 136 + 72 * (i + 1)] for i in range(3))
    A.ada_glu(buf[:, :136], d["w0"], d["w1"], y=y, pre=(g, u))
    g2, u2 = empty(rows, 72, dtype), empty(rows, 72, dtype)
    y2 = A.ada_glu(d["x"], d["w0"], d["w1"], pre=(g2, u2))
    assert torch.equal(buf[:, :136], d["x"]) and torch.equal(y, y2) and torch.equal(g, g2) and torch.equal(u, u2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 18, 140))
def test_feed_forward_block_and_its_gradient(rows, dtype):
    """The block as it is used: h = glu(x), y = linear(h) + x, and back.  Its gradients are
    held against the oracle's on the stored intermediates, and against differences of the
    oracle's forward pass in 64 bits."""
    d_ff, d = 264, 136
    n, t = inputs(11, rows, d_ff, d, dtype, parts=2)
    wd = H.normal(60, (d, d_ff), d_ff ** -0.5, dtype)
    bd = H.normal(61, (d,), 0.5, dtype)
    dy = H.normal(62, (rows, d), 0.3, dtype)
    g, u = empty(rows, d_ff, dtype), empty(rows, d_ff, dtype)
    h = A.ada_glu(t["x"], t["w0"], t["w1"], bias_gate=t["b0"], bias_up=t["b1"], pre=(g, u))
    y = A.ada_linear(h, wd.to(DEV), bias=bd.to(DEV), residual=t["x"])
    hn, gn, un = H.f64(h), H.f64(g), H.f64(u)
    by, _ = H.linear_bounds(hn, H.f64(wd), H.f64(bd), n["x"], "none", dtype)
    H.assert_within(y, OL.linear(hn, H.f64(wd), H.f64(bd), n["x"])[0], by, "y")
    dh, dwd, dbd = A.ada_linear_backward(dy.to(DEV), h, wd.to(DEV), want_dbias=True)
    dx, dwg, dwu, dbg, dbu = A.ada_glu_backward(dh, t["x"], t["w0"], t["w1"], g, u, want_dbias=True)
    dhn = H.f64(dh)
    *ref, dg, du = OL.glu_backward(dhn, n["x"], n["w0"], n["w1"], gn, un)
    ea = H.act_error(gn, np.zeros_like(gn), "silu")
    edg = (H.slope_error(dhn, gn, "silu") + 3 * H.U * np.abs(dhn)) * np.abs(un) + 3 * H.U * np.abs(dg)
    bounds = H.grad_bounds([dg, du], [edg, np.abs(dhn) * ea + 2 * H.U * np.abs(du)], n["x"], [n["w0"], n["w1"]], dtype)
    for a, r, b, what in zip((dx, dwg, dwu, dbg, dbu), ref, bounds, ("dx", "dwg", "dwu", "dbg", "dbu")):
        H.assert_within(a, r, b, what)
    H.assert_within(dwd, H.f64(dy).T @ hn, H.grad_bounds([H.f64(dy)], [np.zeros((rows, d))], hn, [H.f64(wd)], dtype)[1],
                    "dwd")

    # differences: L = sum(dy * y); a step along a random direction of every leaf
    def loss(x, wg, wu, bg, bu, w, b):
        hh = OL.glu(x, wg, wu, bg, bu)[0]
        return float((H.f64(dy) * OL.linear(hh, w, b, x)[0]).sum())

    leaves = [n["x"], n["w0"], n["w1"], n["b0"], n["b1"], H.f64(wd), H.f64(bd)]
    grads = [H.f64(dx) + H.f64(dy), H.f64(dwg), H.f64(dwu), H.f64(dbg), H.f64(dbu), H.f64(dwd), H.f64(dbd)]
    rng = np.random.default_rng(5)
    for i, (leaf, grad) in enumerate(zip(leaves, grads)):
        v = rng.choice((-1.0, 1.0), size=leaf.shape) * (np.abs(leaf) + 0.01)
        e = 1e-5
        up, down = list(leaves), list(leaves)
        up[i], down[i] = leaf + e * v, leaf - e * v
        diff = (loss(*up) - loss(*down)) / (2 * e)
        # each gradient element is off by a few roundings of the storage type (of h, dh, g, u,
        # dg, du and itself: at most 8) of terms of its own size, with signs at random along v:
        # 8 r sqrt(sum g^2 v^2) bounds ten standard deviations or more of what they add up to
        # for elements of random sign; the difference itself is exact to ~1e-9
        bound = 8 * H.half_step(dtype) * np.sqrt(((grad * v) ** 2).sum()) * 4 + 1e-7 * np.abs(grad * v).sum()
        assert abs(diff - float((grad * v).sum())) <= bound, (i, diff, float((grad * v).sum()), bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_same_call_same_bits(dtype):
    """Two calls on the same inputs give the same bits, at sizes of every kernel variant."""
    for rows, d_out, d_in in ((1, 264, 2056), (20, 264, 2056), (90, 264, 2056), (400, 1032, 520)):
        n, d = inputs(12, rows, d_out, d_in, dtype, parts=2)
        _, z = saved(13, rows, d_out, dtype, 0)
        for f in (lambda: [A.ada_linear(d["x"], d["w0"], act="gelu")], lambda: [A.ada_glu(d["x"], d["w0"], d["w1"])],
                  lambda: A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act="silu", want_dbias=True),
                  lambda: A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, z, want_dbias=True)):
            first, second = f(), f()
            assert all(torch.equal(a, b) for a, b in zip(first, second)), (rows, d_out, d_in)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 20, 260))
def test_captured_and_replayed(rows, dtype):
    """A block forward and backward captured into a graph gives the eager bits on every
    replay, with eager calls (on workspaces of their own) and new inputs in between."""
    n, d = inputs(14, rows, 264, 520, dtype, parts=2)
    x = d["x"].clone()
    g, u = empty(rows, 264, dtype), empty(rows, 264, dtype)
    ws = torch.empty(max(1, A.glu_workspace_bytes(rows, 264, 520, x.dtype),
                         A.glu_backward_workspace_bytes(rows, 264, 520, "silu", x.dtype)), dtype=torch.uint8, device=DEV)
    y = empty(rows, 264, dtype)
    outs = [torch.empty_like(x), torch.empty_like(d["w0"]), torch.empty_like(d["w1"]),
            torch.empty_like(d["b0"]), torch.empty_like(d["b1"])]

    def step(x, y, g, u, outs, ws):
        A.ada_glu(x, d["w0"], d["w1"], bias_gate=d["b0"], bias_up=d["b1"], y=y, pre=(g, u), workspace=ws)
        A.ada_glu_backward(y, x, d["w0"], d["w1"], g, u, dx=outs[0], dw_gate=outs[1], dw_up=outs[2],
                           dbias_gate=outs[3], dbias_up=outs[4], workspace=ws)

    step(x, y, g, u, outs, ws)  # warm-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, y, g, u, outs, ws)
    for rep in range(4):
        x.copy_(H.normal(200 + rep, (rows, 520), 1.0, dtype))
        graph.replay()
        e = [torch.empty_like(t) for t in outs]
        ey, eg, eu = (empty(rows, 264, dtype) for _ in range(3))
        step(x, ey, eg, eu, e, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([y, g, u] + outs, [ey, eg, eu] + e)), rep


@pytest.mark.gpu
def test_streams():
    """On a stream other than the current one, given as a stream or as its handle: results and
    workspaces belong to that stream."""
    n, d = inputs(15, 90, 264, 2056, "bf16", parts=2)
    _, z = saved(16, 90, 264, "bf16", 0)
    ref = A.ada_glu(d["x"], d["w0"], d["w1"])
    gref = A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = A.ada_glu(d["x"], d["w0"], d["w1"], stream=s)
        ggot = A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act="silu", stream=s)
        side.synchronize()
        assert torch.equal(got, ref) and torch.equal(ggot[0], gref[0]) and torch.equal(ggot[1], gref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_large_values(dtype):
    """Pre-activations far out on both sides: no overflow in between, the limits of each
    activation and slope."""
    z = torch.tensor([-3e4, -200.0, -90.0, -20.0, -6.0, 0.0, 6.0, 20.0, 90.0, 200.0, 3e4], dtype=H.TD[dtype])
    rows = z.numel()
    x = torch.zeros((rows, 8), dtype=H.TD[dtype])
    x[:, 0] = z
    w = torch.zeros((8, 8), dtype=H.TD[dtype])
    w[:, 0] = 1
    dy = torch.ones((rows, 8), dtype=H.TD[dtype])
    pre = z[:, None].expand(rows, 8).contiguous()
    for act in ACTS:
        y = A.ada_linear(x.to(DEV), w.to(DEV), act=act)
        by, _ = H.linear_bounds(H.f64(x), H.f64(w), None, None, act, dtype)
        H.assert_within(y, OL.linear(H.f64(x), H.f64(w), None, None, act)[0], by, act)
        _, _, db = A.ada_linear_backward(dy.to(DEV), x.to(DEV), w.to(DEV), pre=pre.to(DEV), act=act, want_dx=False,
                                         want_dw=False, want_dbias=True)
        rz = OL.linear_backward(H.f64(dy), H.f64(x), H.f64(w), H.f64(pre), act)[3]
        b = H.grad_bounds([rz], [H.slope_error(H.f64(dy), H.f64(pre), act)], H.f64(x), [H.f64(w)], dtype)[2]
        H.assert_within(db, rz.sum(axis=0), b, act)


# sizes of the largest tile (at least 192 tiles of 256 x 256), ragged in every dimension
LARGE = [(3850, 3304, 200), (2047, 6664, 1096)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large_shapes(shape, dtype):
    rows, d_out, d_in = shape
    check_linear(rows, d_out, d_in, dtype, "silu", pad=8, seed=21)
    check_glu(rows, d_out // 2 // 8 * 8, d_in, dtype, "silu", seed=22)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", [(3850, 200, 3304), (200, 3848, 3304)], ids=lambda s: "x".join(map(str, s)))
def test_large_gradients(shape, dtype):
    """Many tiles of dx (depth d_out) in one shape, of dW (depth rows) in the other."""
    check_linear_backward(*shape, dtype, "silu", seed=23)
    check_glu_backward(*shape, dtype, "silu", seed=24)


# every tile at both of its kinds of rounds, every few-rows block, split contractions, ragged ends
# (of some products each: test_linear_plan.py has every form of every product, and counts them)
VARIANTS = [(17, 1000, 4096), (33, 1000, 4096), (48, 8200, 264), (49, 8200, 264), (64, 4096, 1000),
            (250, 1000, 4104), (509, 4104, 520), (1000, 1032, 2056), (1021, 4104, 264), (2047, 4096, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", VARIANTS, ids=lambda s: "x".join(map(str, s)))
def test_variants(shape, dtype):
    check_linear(*shape, dtype, "relu", pad=8, seed=31)
    check_glu(*shape, dtype, "silu", seed=32)
    check_linear_backward(*shape, dtype, "relu", pad=8, seed=33)
    check_glu_backward(*shape, dtype, "silu", pad=8, seed=34)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("d_out", (8, 56, 64, 72, 128, 200))
def test_seam_between_the_weights(d_out, dtype):
    """dx reads w_gate, then w_up, across its contraction: the seam inside a step, at its end and
    behind the first step, with different row strides."""
    check_glu_backward(70, d_out, 136, dtype, "silu", pad=8, seed=41)
    check_glu_backward(300, d_out, 264, dtype, "silu", pad=16, seed=42)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", (1, 2, 17, 40))
def test_rows_far_apart(rows):
    """Rows of x, y and the residual as the last tokens of long sequences: row strides whose
    offsets pass 32 bits."""
    ld = (1 << 28) // 3 // 8 * 8
    n, d = inputs(51, rows, 136, 264, "bf16")
    base = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)
    x = base.as_strided((rows, 264), (ld, 1))
    y = base.as_strided((rows, 136), (ld, 1), 1024)
    res = base.as_strided((rows, 136), (ld, 1), 2048)
    x.copy_(d["x"])
    res.copy_(d["res"])
    A.ada_linear(x, d["w0"], bias=d["b0"], residual=res, act="gelu", y=y)
    by, _ = H.linear_bounds(n["x"], n["w0"], n["b0"], n["res"], "gelu", "bf16")
    H.assert_within(y, OL.linear(n["x"], n["w0"], n["b0"], n["res"], "gelu")[0], by, "y")
    dx = base.as_strided((rows, 264), (ld, 1), 4096)
    dw = A.ada_linear_backward(d["dy"], x, d["w0"], dx=dx)[1]
    bounds = H.grad_bounds([n["dy"]], [np.zeros_like(n["dy"])], n["x"], [n["w0"]], "bf16")
    rx, rw, _, _ = OL.linear_backward(n["dy"], n["x"], n["w0"], None)
    H.assert_within(dx, rx, bounds[0], "dx")
    H.assert_within(dw, rw, bounds[1], "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_weights_far_apart(dtype):
    """Weight rows with a stride past 32-bit byte offsets, read along and across the contraction."""
    ld = (1 << 29) // 5 // 8 * 8
    rows, d_out, d_in = 20, 24, 72
    n, d = inputs(52, rows, d_out, d_in, dtype)
    w = torch.empty(d_out * ld, dtype=H.TD[dtype], device=DEV).as_strided((d_out, d_in), (ld, 1))
    w.copy_(d["w0"])
    by, _ = H.linear_bounds(n["x"], n["w0"], n["b0"], None, "none", dtype)
    ref = OL.linear(n["x"], n["w0"], n["b0"])[0]
    H.assert_within(A.ada_linear(d["x"], w, bias=d["b0"]), ref, by, "y")
    H.assert_within(A.ada_linear(d["x"][:1], w, bias=d["b0"]), ref[:1], by[:1], "y of one row")
    dx = A.ada_linear_backward(d["dy"], d["x"], w, want_dw=False)[0]
    H.assert_within(dx, n["dy"] @ n["w0"], H.grad_bounds([n["dy"]], [np.zeros_like(n["dy"])], n["x"], [n["w0"]], dtype)[0],
                    "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_two_streams_at_once(dtype):
    """Calls that overlap in time, each with a workspace of its own, do not touch each other."""
    n, d = inputs(53, 300, 1032, 2056, dtype, parts=2)
    _, z = saved(54, 300, 1032, dtype, 0)
    ref = A.ada_glu(d["x"], d["w0"], d["w1"])
    gref = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, z, want_dbias=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for rep in range(4):
        for s in streams:
            out.append((A.ada_glu(d["x"], d["w0"], d["w1"], stream=s),
                        A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, z, want_dbias=True, stream=s)))
    torch.cuda.synchronize()
    for y, g in out:
        assert torch.equal(y, ref) and all(torch.equal(a, b) for a, b in zip(g, gref))


@pytest.mark.gpu
def test_workspace_exactly_as_large_as_asked():
    """The workspace's bytes behind what the call asks for stay as they were, and its contents
    before the call do not matter."""
    rows, d_out, d_in = 250, 1000, 4104
    n, d = inputs(55, rows, d_out, d_in, "bf16", parts=2)
    _, z = saved(56, rows, d_out, "bf16", 0)
    calls = [(A.linear_workspace_bytes(rows, d_out, d_in, torch.bfloat16),
              lambda ws: [A.ada_linear(d["x"], d["w0"], workspace=ws)]),
             (A.glu_workspace_bytes(rows, d_out, d_in, torch.bfloat16),
              lambda ws: [A.ada_glu(d["x"], d["w0"], d["w1"], workspace=ws)]),
             (A.linear_backward_workspace_bytes(rows, d_out, d_in, "silu", torch.bfloat16),
              lambda ws: A.ada_linear_backward(d["dy"], d["x"], d["w0"], pre=z, act="silu", want_dbias=True,
                                               workspace=ws)),
             (A.glu_backward_workspace_bytes(rows, d_out, d_in, "silu", torch.bfloat16),
              lambda ws: A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w1"], z, z, want_dbias=True, workspace=ws))]
    for need, call in calls:
        ref = call(None)
        buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN in either type
        got = call(buf[:need]) if need else call(None)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert (buf[need:] == 0xFF).all()


def test_public_names():
    import weight_merge_amd

    for name in ("ada_linear", "ada_linear_backward", "ada_glu", "ada_glu_backward"):
        assert getattr(weight_merge_amd, name) is getattr(A, name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", [(2, 72, 8968), (12, 264, 28552), (16, 24, 16392), (30, 136, 17000), (48, 520, 9000),
                                   (5, 6000, 264), (20, 4200, 2056), (40, 4200, 520)], ids=lambda s: "x".join(map(str, s)))
def test_few_rows_variants(shape, dtype):
    """Few rows with the contraction split over workgroups (few columns, long rows), and with two
    waves a workgroup (many columns, short rows)."""
    check_linear(*shape, dtype, "gelu", pad=8, seed=61)
    check_glu(*shape, dtype, "silu", pad=8, seed=62)


@pytest.mark.gpu
def test_default_stream_by_handle():
    """The default stream given as a Stream, and as its handle 0."""
    n, d = inputs(71, 20, 72, 136, "bf16", parts=2)
    ref = A.ada_glu(d["x"], d["w0"], d["w1"])
    for s in (torch.cuda.default_stream(), 0):
        got = A.ada_glu(d["x"], d["w0"], d["w1"], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_few_far_apart_rows_of_a_long_contraction(dtype):
    """Rows too far apart for the few-rows kernel and a contraction that it would split."""
    rows, d_out, d_in, ld = 3, 40, 17000, (1 << 29) // 5 // 8 * 8
    n, d = inputs(72, rows, d_out, d_in, dtype)
    x = torch.empty(rows * ld, dtype=H.TD[dtype], device=DEV).as_strided((rows, d_in), (ld, 1))
    x.copy_(d["x"])
    by, _ = H.linear_bounds(n["x"], n["w0"], n["b0"], n["res"], "gelu", dtype)
    H.assert_within(A.ada_linear(x, d["w0"], bias=d["b0"], residual=d["res"], act="gelu"),
                    OL.linear(n["x"], n["w0"], n["b0"], n["res"], "gelu")[0], by, "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_one_matrix_for_both_projections(dtype):
    """The same weight, bias and saved matrix given twice: inputs may be one tensor."""
    n, d = inputs(73, 33, 136, 264, dtype)
    y = A.ada_glu(d["x"], d["w0"], d["w0"], bias_gate=d["b0"], bias_up=d["b0"], act="none")
    by = H.glu_bounds(n["x"], n["w0"], n["w0"], n["b0"], n["b0"], "none", dtype)[0]
    H.assert_within(y, OL.glu(n["x"], n["w0"], n["w0"], n["b0"], n["b0"], "none")[0], by, "y")
    same = A.ada_glu(d["x"], d["w0"], d["w0"].clone(), bias_gate=d["b0"], bias_up=d["b0"].clone(), act="none")
    assert torch.equal(y, same)
    _, z = saved(74, 33, 136, dtype, 0)
    a = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w0"], z, z, act="relu", want_dbias=True)
    b = A.ada_glu_backward(d["dy"], d["x"], d["w0"], d["w0"].clone(), z, z.clone(), act="relu", want_dbias=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


# weights large enough for the few-rows gradients: a row or two, around 16 and 32 rows and past
# them; d_out and d_in off the waves' 64 rows, 256 columns and contraction steps; long and short
# contractions (in many parts, in one)
FEW_GRADS = [(1, 1288, 2056), (2, 33000, 72), (7, 2056, 1288), (15, 4104, 520), (16, 72, 33000), (17, 520, 8200),
             (31, 18056, 264), (32, 1288, 4104)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("shape", FEW_GRADS, ids=lambda s: "x".join(map(str, s)))
def test_few_rows_gradients(shape, dtype):
    check_linear_backward(*shape, dtype, "silu", pad=8, seed=51)
    check_glu_backward(*shape, dtype, "relu", pad=16, seed=52)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(33, 4104, 4120), (49, 1288, 13064), (64, 16904, 1000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_two_blocks_of_rows_gradients(shape):
    check_linear_backward(*shape, "bf16", "none", seed=53)
    rows, d_out, d_in = shape
    check_glu_backward(rows, d_out // 16 * 8, d_in, "bf16", "silu", pad=8, seed=54)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (5, 17, 50))
def test_few_rows_gradients_alone_captured_and_with_infinities(rows, dtype):
    d_out, d_in = 4104, 4120
    n, d = inputs(55, rows, d_out, d_in, dtype, parts=2)
    z, u = H.normal(56, (rows, d_out), 1.0, dtype).to(DEV), H.normal(57, (rows, d_out), 1.0, dtype).to(DEV)
    args = (d["dy"], d["x"], d["w0"], d["w1"], z, u)
    full = A.ada_glu_backward(*args, want_dbias=True)
    dx = torch.empty_like(full[0])
    A.ada_glu_backward(*args, dx=dx, want_dw=False)
    assert torch.equal(dx, full[0])
    for h, name in ((1, "dw_gate"), (2, "dw_up")):
        one = torch.full_like(full[h], float("nan"))
        A.ada_glu_backward(*args, **{name: one}, want_dx=False, want_dw=False)
        assert torch.equal(one, full[h]), name

    outs = [torch.empty_like(t) for t in full]
    ws = torch.empty(A.glu_backward_workspace_bytes(rows, d_out, d_in, "silu", H.TD[dtype]), dtype=torch.uint8, device=DEV)

    def call():
        A.ada_glu_backward(*args, dx=outs[0], dw_gate=outs[1], dw_up=outs[2], dbias_gate=outs[3], dbias_up=outs[4],
                           workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, full))
        A.ada_glu_backward(*args)

    # an infinity reaches its own column of a gradient and no other element
    dz, x, w = d["dy"], d["x"].clone(), d["w0"].clone()
    dx, dw, _ = A.ada_linear_backward(dz, x, w)
    x[0, 5], w[0, 7], w[d_out - 1, 9] = float("inf"), float("-inf"), float("inf")
    ix, iw, _ = A.ada_linear_backward(dz, x, w)
    fx, fw = ix.isfinite(), iw.isfinite()
    assert not fx[:, [7, 9]].any() and not fw[:, 5].any()
    fx[:, [7, 9]], fw[:, 5] = True, True
    assert fx.all() and fw.all()
    keep_x, keep_w = torch.ones(d_in, dtype=torch.bool, device=DEV), torch.ones(d_in, dtype=torch.bool, device=DEV)
    keep_x[[7, 9]] = False
    keep_w[5] = False
    assert torch.equal(ix[:, keep_x], dx[:, keep_x]) and torch.equal(iw[:, keep_w], dw[:, keep_w])


@pytest.mark.gpu
def test_few_rows_gradients_of_far_apart_rows():
    rows, d_out, d_in, ld = 19, 4104, 520, 600_000  # 4.9 GB from the first row to the last
    n, d = inputs(58, rows, d_out, d_in, "bf16")
    w = torch.empty((d_out, ld), dtype=torch.bfloat16, device=DEV)[:, :d_in]
    dw = torch.empty((d_out, ld), dtype=torch.bfloat16, device=DEV)[:, :d_in]
    w.copy_(d["w0"])
    dx, _, _ = A.ada_linear_backward(d["dy"], d["x"], w, dw=dw)
    rx, rw, _, _ = OL.linear_backward(n["dy"], n["x"], n["w0"], None)
    bounds = H.grad_bounds([n["dy"]], [np.zeros_like(n["dy"])], n["x"], [n["w0"]], "bf16")
    H.assert_within(dx, rx, bounds[0], "dx")
    H.assert_within(dw, rw, bounds[1], "dw")
