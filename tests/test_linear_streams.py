"""Calls of the linear and gated products on a stream of their own: the tensors they were given
may be dropped while the work is still to come."""
import contextlib
import types

import pytest
import torch

import linear_helpers as H
from weight_merge_amd import api as A

ROWS, N, K = 6, 24, 40


class Marked(torch.Tensor):
    """A host tensor that passes for a device one and remembers the streams it was marked for."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        self.__dict__.setdefault("marks", []).append(stream)


class OwnStream:
    pass


class ForeignStream(OwnStream):
    def __init__(self, handle=0):
        self.handle = handle


def marked(*shape):
    return torch.zeros(shape).as_subclass(Marked)


def calls():
    """Every tensor argument of every call."""
    x, w, w2, y, b, b2 = marked(ROWS, K), marked(N, K), marked(N, K), marked(ROWS, N), marked(N), marked(N)
    pre, pre2, res, dy = marked(ROWS, N), marked(ROWS, N), marked(ROWS, N), marked(ROWS, N)
    dx, dw, dw2, db, db2, ws = marked(ROWS, K), marked(N, K), marked(N, K), marked(N), marked(N), marked(64)
    return [
        (A.ada_linear, dict(x=x, w=w, bias=b, residual=res, act="gelu", y=y, pre=pre, workspace=ws)),
        (A.ada_linear_backward, dict(dy=dy, x=x, w=w, pre=pre, act="silu", dx=dx, dw=dw, dbias=db, workspace=ws)),
        (A.ada_glu, dict(x=x, w_gate=w, w_up=w2, bias_gate=b, bias_up=b2, y=y, pre=(pre, pre2), workspace=ws)),
        (A.ada_glu_backward, dict(dy=dy, x=x, w_gate=w, w_up=w2, gate_pre=pre, up_pre=pre2, dx=dx, dw_gate=dw,
                                  dw_up=dw2, dbias_gate=db, dbias_up=db2, workspace=ws)),
    ]


def tensors(args):
    for v in args.values():
        yield from (t for t in (v if isinstance(v, tuple) else (v,)) if isinstance(t, torch.Tensor))


@pytest.mark.parametrize("which", range(4))
def test_every_tensor_is_marked_for_the_stream(which, monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", OwnStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ForeignStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(A, "_current", lambda dev: None)
    monkeypatch.setattr(A, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(A, "_workspace_bytes", lambda *a: 0)
    launched = []
    lib = types.SimpleNamespace(**{n: lambda *a: launched.append(a) or 0 for n in (
        "ada_linear", "ada_linear_backward", "ada_glu", "ada_glu_backward")})
    monkeypatch.setattr(A._lib, "load", lambda: lib)
    call, args = calls()[which]
    call(**args)
    assert len(launched) == 1 and not any("marks" in t.__dict__ for t in tensors(args))
    side = OwnStream()
    call(**args, stream=side)
    assert len(launched) == 2 and all(t.__dict__["marks"] == [side] for t in tensors(args))
    for foreign in (ForeignStream(), 0):  # may be destroyed before the allocator asks it: not marked
        call(**args, stream=foreign)
    assert len(launched) == 4 and all(t.__dict__["marks"] == [side] for t in tensors(args))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_inputs_dropped_behind_the_call(dtype):
    """The call's stream has work before it; meanwhile the inputs are dropped and others of their
    sizes are made and overwritten on the current stream."""
    rows, n, k = 40, 264, 520
    t = dict(x=H.normal(1, (rows, k), 1.0, dtype), w=H.normal(2, (n, k), 0.05, dtype), u=H.normal(3, (n, k), 0.05, dtype),
             dy=H.normal(4, (rows, n), 0.3, dtype), g=H.normal(5, (rows, n), 1.0, dtype), b=H.normal(6, (n,), 0.3, dtype))

    def made():
        return types.SimpleNamespace(**{name: v.to("cuda") for name, v in t.items()})

    runs = [lambda d, s: [A.ada_linear(d.x, d.w, bias=d.b, residual=d.dy, act="gelu", stream=s)],
            lambda d, s: [A.ada_glu(d.x, d.w, d.u, bias_gate=d.b, stream=s)],
            lambda d, s: list(A.ada_linear_backward(d.dy, d.x, d.w, pre=d.g, act="silu", want_dbias=True, stream=s)),
            lambda d, s: list(A.ada_glu_backward(d.dy, d.x, d.w, d.u, d.g, d.dy, want_dbias=True, stream=s))]
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device="cuda")
    for run in runs:
        ref = run(made(), None)
        d = made()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.add_(1)  # some milliseconds
        got = run(d, side)
        shapes = [(v.shape, v.dtype) for v in vars(d).values()]
        del d
        others = [torch.full(s, float("nan"), dtype=dt, device="cuda") for s, dt in shapes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        del others


@pytest.mark.gpu
@pytest.mark.parametrize("rows", (20, 250))
def test_captured_with_the_stream_given(rows):
    """A capture whose calls name its stream, with tensors made and dropped inside it."""
    n, k = 1000, 4104
    x, w, u = (H.normal(i, s, 0.05, "bf16").to("cuda") for i, s in enumerate(((rows, k), (n, k), (n, k))))
    side = torch.cuda.Stream()

    def step(s):
        h = A.ada_glu(x, w, u, stream=s)  # its workspace, and h below, go back to the pool here
        y = A.ada_linear(h * 2, w[:, :n].contiguous(), residual=h, act="gelu", stream=s)
        return [y, *A.ada_linear_backward(y, x, w, stream=s)[:2]]

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(side)
    for rep in range(4):
        x.copy_(H.normal(10 + rep, (rows, k), 0.05, "bf16"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ref = step(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), rep
