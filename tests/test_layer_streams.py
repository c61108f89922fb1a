"""Norm, dropout and router calls on a stream of their own: every tensor is marked as used there."""
import contextlib
import types

import pytest
import torch

from weight_merge_amd import api as A

ROWS, D, E, K = 6, 40, 8, 2


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


def marked(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Marked)


def matrix():
    return marked(ROWS, D)


def calls():
    """Every tensor argument of every call."""
    def routing():
        return (marked(ROWS, K, dtype=torch.int32), marked(ROWS, K), marked(E, dtype=torch.int32), marked(E), marked(1),
                marked(1, dtype=torch.int32))

    def state():
        return marked(2, dtype=torch.int64)

    return [
        (A.ada_norm, dict(x=matrix(), weight=marked(D), bias=marked(D), residual=matrix(), p=0.1, seed=state(), y=matrix(),
                          hidden=matrix(), stats=(marked(ROWS), marked(ROWS)))),
        (A.ada_norm_backward, dict(dy=matrix(), hidden=matrix(), stats=(marked(ROWS), marked(ROWS)), weight=marked(D),
                                   dhidden=matrix(), p=0.1, seed=state(), dx=matrix(), dresidual=matrix(),
                                   dweight=marked(D), dbias=marked(D), workspace=marked(64))),
        (A.ada_dropout, dict(x=matrix(), p=0.1, seed=state(), residual=matrix(), y=matrix())),
        (A.ada_dropout_backward, dict(dy=matrix(), p=0.1, seed=state(), dx=matrix())),
        (A.ada_route, dict(logits=marked(ROWS, E), k=K, valid=marked(ROWS, dtype=torch.bool), out=routing(),
                           workspace=marked(64))),
        (A.ada_route_backward, dict(logits=marked(ROWS, E), out=routing(), dgate=marked(ROWS, K), dloss=marked(1),
                                    dlogits=marked(ROWS, E))),
    ]


def tensors(args):
    for v in args.values():
        yield from (t for t in (v if isinstance(v, tuple) else (v,)) if isinstance(t, torch.Tensor))


@pytest.mark.parametrize("which", range(6))
def test_every_tensor_is_marked_for_the_stream(which, monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", OwnStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", ForeignStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(A, "_current", lambda dev: None)
    monkeypatch.setattr(A, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(A, "_workspace_bytes", lambda *a: 0)
    launched = []
    call, args = calls()[which]
    lib = types.SimpleNamespace(**{call.__name__: lambda *a: launched.append(a) or 0})
    monkeypatch.setattr(A._lib, "load", lambda: lib)
    call(**args)
    assert len(launched) == 1 and not any("marks" in t.__dict__ for t in tensors(args))
    side = OwnStream()
    call(**args, stream=side)
    assert len(launched) == 2 and all(t.__dict__["marks"] == [side] for t in tensors(args))
    for foreign in (ForeignStream(), 0):  # may be destroyed before the allocator asks it: not marked
        call(**args, stream=foreign)
    assert len(launched) == 4 and all(t.__dict__["marks"] == [side] for t in tensors(args))
