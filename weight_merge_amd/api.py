"""Python binding of libadafuse: argument marshalling only.

Every computation runs in the HIP kernels behind the C ABI; this module turns torch
tensors (device memory) and the current torch stream into the pointers and sizes the
C calls take, and turns negative status codes into exceptions.  Output tensors a
caller does not pass are allocated here with torch, outside the C calls.
"""
from __future__ import annotations

import ctypes
import functools
from operator import index
from typing import NamedTuple

import torch

from . import _lib
from ._lib import (ADA_BF16, ADA_F32, AdaDropoutArgs, AdaDropoutGradArgs, AdaGemvProj, AdaGluArgs,
                   AdaGluGradArgs, AdaLinearArgs, AdaLinearGradArgs, AdaLoraProj, AdaNormArgs, AdaNormGradArgs, AdaProj,
                   AdaRouteArgs, AdaRouteGradArgs)

_DT = {torch.float32: ADA_F32, torch.bfloat16: ADA_BF16}


class AdaError(RuntimeError):
    def __init__(self, status: int, call: str):
        msg = _lib.load().ada_status_string(status).decode()
        super().__init__(f"{call} failed with status {status}: {msg}")
        self.status = status


def _check(status: int, call: str):
    if status != 0:
        raise AdaError(status, call)


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16") from None


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _contig(t: torch.Tensor, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t: torch.Tensor, shape, dtype, name: str):
    """A caller-provided output: the C call writes numel(shape) contiguous elements."""
    _contig(t, name)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def ada_pregate(h: torch.Tensor, router: torch.Tensor, k: int, renorm: bool = True,
                idx_out: torch.Tensor | None = None, gate_out: torch.Tensor | None = None,
                stream=None):
    """Router GEMV + top-k + gates (one kernel).  Returns (idx int32[k], gate fp32[k])
    on the device."""
    _contig(h, "h")
    _contig(router, "router")
    E, d = router.shape
    if h.shape != (d,) or h.dtype != router.dtype:
        raise ValueError("h must be [d] with the router's dtype")
    if idx_out is None:
        idx_out = torch.empty(k, dtype=torch.int32, device=h.device)
    if gate_out is None:
        gate_out = torch.empty(k, dtype=torch.float32, device=h.device)
    _out(idx_out, (k,), torch.int32, "idx_out")
    _out(gate_out, (k,), torch.float32, "gate_out")
    st = _lib.load().ada_pregate(_dev(h, "h"), _dev(router, "router"), d, E, k, _dtype(h), int(bool(renorm)),
                                 _dev(idx_out, "idx_out"), _dev(gate_out, "gate_out"), _stream(stream))
    _check(st, "ada_pregate")
    return idx_out, gate_out


class AdaModel:
    """A registered stack of adapted projections (owns the device work table).

    projs: iterable of (w, w_out, a, b) with w [d_out, d_in] (row stride w.stride(0)),
    w_out None (merge in place) or a tensor like w, a [E, r, d_in], b [E, d_out, r].
    The tensors must outlive the model; the model keeps references to them.  The
    work table is uploaded on `stream` (default: torch's current stream), which
    orders it before the merges enqueued there.
    """

    def __init__(self, projs, E: int, r: int, stream=None):
        projs = list(projs)
        if not projs:
            raise ValueError("no projections")
        dt = projs[0][0].dtype
        arr = (AdaProj * len(projs))()
        keep = []
        for i, (w, w_out, a, b) in enumerate(projs):
            d_out, d_in = w.shape
            if w.stride(1) != 1 or (w_out is not None and (w_out.shape != w.shape or w_out.stride() != w.stride())):
                raise ValueError("w must have unit column stride; w_out must match w's layout")
            _contig(a, "a")
            _contig(b, "b")
            if a.shape != (E, r, d_in) or b.shape != (E, d_out, r):
                raise ValueError(f"adapter bank shapes {tuple(a.shape)}, {tuple(b.shape)} do not match "
                                 f"E={E}, r={r}, W {tuple(w.shape)}")
            for t in (w, a, b) + ((w_out,) if w_out is not None else ()):
                if t.dtype != dt:
                    raise TypeError("all tensors of a model share one dtype")
            arr[i] = AdaProj(_dev(w, "w"), _dev(w_out, "w_out") if w_out is not None else None,
                             _dev(a, "a"), _dev(b, "b"), d_out, d_in, w.stride(0))
            keep.append((w, w_out, a, b))
        handle = ctypes.c_void_p()
        st = _lib.load().ada_model_create(arr, len(projs), E, r, _DT[dt], _stream(stream), ctypes.byref(handle))
        _check(st, "ada_model_create")
        self._h = handle
        self._keep = keep
        self.E, self.r, self.dtype = E, r, dt
        self.n_proj = len(projs)

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("model destroyed")
        return self._h

    @property
    def tiles(self) -> int:
        return int(_lib.load().ada_model_tiles(self.handle))

    @property
    def device_bytes(self) -> int:
        """Device memory the model owns (its work tables)."""
        return int(_lib.load().ada_model_device_bytes(self.handle))

    def destroy(self):
        if getattr(self, "_h", None) is not None:
            _lib.load().ada_model_destroy(self._h)
            self._h = None
            self._keep = []

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _sel(idx: torch.Tensor, gate: torch.Tensor):
    if idx.dtype != torch.int32 or gate.dtype != torch.float32:
        raise TypeError("idx must be int32 and gate float32")
    if idx.dim() != 1 or gate.dim() != 1 or idx.numel() != gate.numel():
        raise ValueError("idx and gate must be one-dimensional and of the same length")
    _contig(idx, "idx")
    _contig(gate, "gate")
    return _dev(idx, "idx"), _dev(gate, "gate"), idx.numel()


def ada_merge(model: AdaModel, idx: torch.Tensor, gate: torch.Tensor, scale: float, stream=None):
    """Fuse the selected adapters into every registered projection (one launch)."""
    pi, pg, k = _sel(idx, gate)
    _check(_lib.load().ada_merge(model.handle, pi, pg, k, float(scale), _stream(stream)), "ada_merge")


def ada_unmerge(model: AdaModel, idx: torch.Tensor, gate: torch.Tensor, scale: float, stream=None):
    """De-fuse the selection from the merged buffer (one launch)."""
    pi, pg, k = _sel(idx, gate)
    _check(_lib.load().ada_unmerge(model.handle, pi, pg, k, float(scale), _stream(stream)), "ada_unmerge")


def ada_switch(model: AdaModel, prev, cur, scale: float, stream=None):
    """Undo selection `prev` and apply `cur` in one pass; prev, cur = (idx, gate)."""
    pi, pg, pk = _sel(*prev)
    ci, cg, ck = _sel(*cur)
    _check(_lib.load().ada_switch(model.handle, pi, pg, pk, ci, cg, ck, float(scale), _stream(stream)),
           "ada_switch")


def ada_decode_gemv(w: torch.Tensor, x: torch.Tensor, y: torch.Tensor | None = None, stream=None):
    """y = W x on the device (fp32 accumulation, one rounding)."""
    d_out, d_in = w.shape
    if w.stride(1) != 1:
        raise ValueError("w must have unit column stride")
    _contig(x, "x")
    if x.shape != (d_in,) or x.dtype != w.dtype:
        raise ValueError("x must be [d_in] with w's dtype")
    if y is None:
        y = torch.empty(d_out, dtype=w.dtype, device=w.device)
    _out(y, (d_out,), w.dtype, "y")
    st = _lib.load().ada_decode_gemv(_dev(w, "w"), d_out, d_in, w.stride(0), _dev(x, "x"), _dev(y, "y"),
                                     _dtype(w), _stream(stream))
    _check(st, "ada_decode_gemv")
    return y


def ada_decode_gemv_layer(projs, stream=None):
    """Independent GEMVs y_p = W_p x_p in one launch; projs: list of (w, x, y) with w
    [d_out, d_in], x [d_in], y [d_out] (written), all of one dtype."""
    projs = list(projs)
    arr = (AdaGemvProj * len(projs))()
    dt = projs[0][0].dtype
    for i, (w, x, y) in enumerate(projs):
        d_out, d_in = w.shape
        if w.stride(1) != 1:
            raise ValueError("w must have unit column stride")
        _contig(x, "x")
        _contig(y, "y")
        if x.shape != (d_in,) or y.shape != (d_out,):
            raise ValueError("x must be [d_in] and y [d_out]")
        if w.dtype != dt or x.dtype != dt or y.dtype != dt:
            raise TypeError("all tensors share one dtype")
        arr[i] = AdaGemvProj(_dev(w, "w"), _dev(x, "x"), _dev(y, "y"), d_out, d_in, w.stride(0))
    st = _lib.load().ada_decode_gemv_layer(arr, len(projs), _DT[dt], _stream(stream))
    _check(st, "ada_decode_gemv_layer")


def ada_lora_apply(w, a, b, idx, gate, scale: float, x, y=None, workspace=None, stream=None):
    """Unmerged routed projection y = W x + s sum_j g_j B_j (A_j x) (three launches)."""
    d_out, d_in = w.shape
    E, r, _ = a.shape
    pi, pg, k = _sel(idx, gate)
    if w.stride(1) != 1:
        raise ValueError("w must have unit column stride")
    for t, n in ((a, "a"), (b, "b"), (x, "x")):
        _contig(t, n)
    if a.shape != (E, r, d_in) or b.shape != (E, d_out, r) or x.shape != (d_in,):
        raise ValueError("projection shapes do not match")
    if a.dtype != w.dtype or b.dtype != w.dtype or x.dtype != w.dtype:
        raise TypeError("all tensors share one dtype")
    if y is None:
        y = torch.empty(d_out, dtype=w.dtype, device=w.device)
    _out(y, (d_out,), w.dtype, "y")
    need = (d_out + k * r) * 4
    if workspace is None:
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=w.device)
    _contig(workspace, "workspace")
    st = _lib.load().ada_lora_apply(_dev(w, "w"), d_out, d_in, w.stride(0), _dev(a, "a"), _dev(b, "b"),
                                    E, r, pi, pg, k, float(scale), _dev(x, "x"), _dev(y, "y"),
                                    _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                    _dtype(w), _stream(stream))
    _check(st, "ada_lora_apply")
    return y


def lora_layer_workspace_elems(d_outs, k: int, r: int) -> int:
    """fp32 elements of workspace ada_lora_layer needs for these projections."""
    n = 0
    for d in d_outs:
        n = (n + d + k * r + 3) // 4 * 4
    return n


def _lora_layer_projs(projs):
    w0, a0 = projs[0][0], projs[0][1]
    E, r, _ = a0.shape
    arr = (AdaLoraProj * len(projs))()
    for i, (w, a, b, x, y) in enumerate(projs):
        d_out, d_in = w.shape
        if w.stride(1) != 1:
            raise ValueError("w must have unit column stride")
        for t, n in ((a, "a"), (b, "b"), (x, "x"), (y, "y")):
            _contig(t, n)
        if a.shape != (E, r, d_in) or b.shape != (E, d_out, r) or x.shape != (d_in,) or y.shape != (d_out,):
            raise ValueError("projection shapes do not match")
        if any(t.dtype != w0.dtype for t in (w, a, b, x, y)):
            raise TypeError("all tensors share one dtype")
        arr[i] = AdaLoraProj(_dev(w, "w"), _dev(a, "a"), _dev(b, "b"), _dev(x, "x"), _dev(y, "y"), d_out, d_in,
                             w.stride(0))
    return arr, w0, E, r


def ada_lora_layer(projs, idx, gate, scale: float, workspace=None, stream=None):
    """One layer of the unmerged routed path (two launches for all projections).

    projs: list of (w, a, b, x, y) with w [d_out, d_in], a [E, r, d_in], b [E, d_out, r],
    x [d_in], y [d_out] (written)."""
    projs = list(projs)
    arr, w0, E, r = _lora_layer_projs(projs)
    pi, pg, k = _sel(idx, gate)
    need = lora_layer_workspace_elems([p[0].shape[0] for p in projs], k, r)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.float32, device=w0.device)
    _contig(workspace, "workspace")
    st = _lib.load().ada_lora_layer(arr, len(projs), E, r, pi, pg, k, float(scale), _dev(workspace, "workspace"),
                                    workspace.numel() * workspace.element_size(), _dtype(w0), _stream(stream))
    _check(st, "ada_lora_layer")


def ada_lora_layer_static(projs, idx, gate, scale: float, stream=None):
    """ada_lora_layer with its intermediates in the library's static device array (4 MiB
    per GPU): the C call allocates nothing.  Calls overlapping in time on one GPU race."""
    projs = list(projs)
    arr, w0, E, r = _lora_layer_projs(projs)
    pi, pg, k = _sel(idx, gate)
    st = _lib.load().ada_lora_layer_static(arr, len(projs), E, r, pi, pg, k, float(scale), _dtype(w0),
                                           _stream(stream))
    _check(st, "ada_lora_layer_static")


def lora_batch_workspace_elems(d_outs, nb: int, k: int, r: int) -> int:
    """fp32 elements of workspace ada_lora_batch needs for these projections."""
    n = 0
    for d in d_outs:
        n = (n + nb * (d + k * r) + 3) // 4 * 4
    return n


def ada_lora_batch(projs, idx, gate, scale: float, workspace=None, stream=None):
    """One layer of the unmerged routed path for a batch of requests with a selection
    each (two launches for all projections and requests).

    projs: list of (w, a, b, x, y) with w [d_out, d_in], a [E, r, d_in], b [E, d_out, r],
    x [nb, d_in], y [nb, d_out] (written); idx int32 [nb, k], gate fp32 [nb, k]."""
    projs = list(projs)
    w0, a0 = projs[0][0], projs[0][1]
    E, r, _ = a0.shape
    if idx.dim() != 2 or idx.shape != gate.shape:
        raise ValueError("idx and gate must be [nb, k] and of equal shape")
    if idx.dtype != torch.int32 or gate.dtype != torch.float32:
        raise TypeError("idx must be int32 and gate float32")
    _contig(idx, "idx")
    _contig(gate, "gate")
    nb, k = idx.shape
    arr = (AdaLoraProj * len(projs))()
    for i, (w, a, b, x, y) in enumerate(projs):
        d_out, d_in = w.shape
        if w.stride(1) != 1:
            raise ValueError("w must have unit column stride")
        for t, n in ((a, "a"), (b, "b"), (x, "x"), (y, "y")):
            _contig(t, n)
        if a.shape != (E, r, d_in) or b.shape != (E, d_out, r) or x.shape != (nb, d_in) or y.shape != (nb, d_out):
            raise ValueError("projection shapes do not match")
        if any(t.dtype != w0.dtype for t in (w, a, b, x, y)):
            raise TypeError("all tensors share one dtype")
        arr[i] = AdaLoraProj(_dev(w, "w"), _dev(a, "a"), _dev(b, "b"), _dev(x, "x"), _dev(y, "y"), d_out, d_in,
                             w.stride(0))
    need = lora_batch_workspace_elems([p[0].shape[0] for p in projs], nb, k, r)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.float32, device=w0.device)
    _contig(workspace, "workspace")
    st = _lib.load().ada_lora_batch(arr, len(projs), nb, E, r, _dev(idx, "idx"), _dev(gate, "gate"), k,
                                    float(scale), _dev(workspace, "workspace"),
                                    workspace.numel() * workspace.element_size(), _dtype(w0), _stream(stream))
    _check(st, "ada_lora_batch")


# ---- linear and gated feed-forward products ----------------------------------------
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _act(act: str) -> int:
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"unknown activation {act!r}; expected one of {', '.join(_ACTS)}") from None


def _refuse(t, shape, dt, dev: int, name: str):
    """The error for a tensor that is not of this shape, dtype and device with unit column stride."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt} like the other tensors, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not with the other tensors")
    raise ValueError(f"{name} must have unit column stride" if len(shape) == 2 else f"{name} must be contiguous")


def _mat(t, rows: int, cols: int, dt, dev: int, name: str):
    """Pointer and row stride of a [rows, cols] matrix."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols) or t.dtype is not dt or t.get_device() != dev:
        _refuse(t, (rows, cols), dt, dev, name)
    ld, one = t.stride()
    if one != 1:
        _refuse(t, (rows, cols), dt, dev, name)
    return t.data_ptr(), ld if rows > 1 else cols


def _vec(t, n: int, dt, dev: int, name: str):
    """Pointer of an [n] vector."""
    if t is None:
        return None
    if t.shape != (n,) or t.dtype is not dt or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, (n,), dt, dev, name)
    return t.data_ptr()


def _sizes(x: torch.Tensor, w: torch.Tensor):
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [rows, d_in] and the weights [d_out, d_in]")
    return x.shape[0], w.shape[0], w.shape[1]


# index of the current device (the public call looks whether the runtime is up each time; a device
# tensor is there already)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _current(dev: int):
    if dev < 0:
        raise ValueError("tensors must be on the device")
    if dev != _device_now():
        raise ValueError(f"tensors are on cuda:{dev}, but cuda:{torch.cuda.current_device()} is current")


def _on(stream, call, *args):
    """The call with its stream as the current one, so that what it allocates is made ready, and
    taken back, in that stream's order.  The tensors passed to it are marked as used there: the
    allocator then gives out their memory, if the caller drops them, only behind this work.
    (A foreign stream may be gone when the allocator asks it, so for those the caller keeps them.)"""
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        out = call(*args)
    if not isinstance(s, torch.cuda.ExternalStream):
        for a in args:
            for t in a if isinstance(a, (tuple, list)) else (a,):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(s)
    return out


def _raw_stream(dev: int) -> int:
    """Handle of the current stream (the public call builds a Stream object each time)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream().cuda_stream


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(call: str, *sizes) -> int:
    n = int(getattr(_lib.load(), call)(*sizes))
    _check(min(n, 0), call)
    return n


def _workspace(need: int, workspace, dev: int):
    """(pointer, bytes, tensor) of the caller's workspace, or of one allocated here."""
    if workspace is not None:
        _contig(workspace, "workspace")
        if workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, not with the other tensors")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if need == 0:
        return None, 0, None
    workspace = torch.empty(need, dtype=torch.uint8, device=f"cuda:{dev}")
    return workspace.data_ptr(), need, workspace


def linear_workspace_bytes(rows: int, d_out: int, d_in: int, dtype: torch.dtype) -> int:
    """Bytes of workspace ada_linear needs at these sizes."""
    return _workspace_bytes("ada_linear_workspace", rows, d_out, d_in, _DT[dtype])


def glu_workspace_bytes(rows: int, d_out: int, d_in: int, dtype: torch.dtype) -> int:
    """Bytes of workspace ada_glu needs at these sizes."""
    return _workspace_bytes("ada_glu_workspace", rows, d_out, d_in, _DT[dtype])


def linear_backward_workspace_bytes(rows: int, d_out: int, d_in: int, act: str, dtype: torch.dtype) -> int:
    """Bytes of workspace ada_linear_backward needs at these sizes."""
    return _workspace_bytes("ada_linear_backward_workspace", rows, d_out, d_in, _act(act), _DT[dtype])


def glu_backward_workspace_bytes(rows: int, d_out: int, d_in: int, act: str, dtype: torch.dtype) -> int:
    """Bytes of workspace ada_glu_backward needs at these sizes."""
    return _workspace_bytes("ada_glu_backward_workspace", rows, d_out, d_in, _act(act), _DT[dtype])


def ada_linear(x: torch.Tensor, w: torch.Tensor, bias=None, residual=None, act: str = "none", y=None, pre=None,
               workspace=None, stream=None):
    """y = act(x w^T + bias) + residual for x [rows, d_in], w [d_out, d_in] (rows of any
    matrix may be strided); `pre`, if given, receives x w^T + bias for the backward pass.

    act: "none", "relu", "silu", "gelu" (error function) or "gelu_tanh".  y may be the
    residual itself.  A workspace and a y not passed are allocated on the call's stream.

    `stream` (here and in the calls like this one): a torch.cuda.Stream, or the handle of one,
    else the current stream.  Work queued elsewhere before the call is not waited for.  Tensors
    passed with a torch.cuda.Stream may be dropped at once; with a handle or an ExternalStream
    keep those that belong to another stream until the work is done."""
    if stream is not None:
        return _on(stream, ada_linear, x, w, bias, residual, act, y, pre, workspace)
    rows, d_out, d_in = _sizes(x, w)
    code, dc, dt, dev = _act(act), _dtype(x), x.dtype, x.get_device()
    px, ldx = _mat(x, rows, d_in, dt, dev, "x")
    pw, ldw = _mat(w, d_out, d_in, dt, dev, "w")
    pb = _vec(bias, d_out, dt, dev, "bias")
    pr, ldr = _mat(residual, rows, d_out, dt, dev, "residual")
    pp, ldp = _mat(pre, rows, d_out, dt, dev, "pre")
    if y is not None:
        py, ldy = _mat(y, rows, d_out, dt, dev, "y")
    _current(dev)
    if y is None:
        y = torch.empty((rows, d_out), dtype=dt, device=x.device)
        py, ldy = y.data_ptr(), d_out
    ws, nbytes, _keep = _workspace(_workspace_bytes("ada_linear_workspace", rows, d_out, d_in, dc), workspace, dev)
    args = AdaLinearArgs(px, pw, pb, pr, py, pp, ldx, ldw, ldr, ldy, ldp, rows, d_out, d_in)
    _check(_lib.load().ada_linear(args, code, dc, ws, nbytes, _raw_stream(dev)), "ada_linear")
    return y


def ada_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, pre=None, act: str = "none", dx=None,
                        dw=None, dbias=None, want_dx: bool = True, want_dw: bool = True, want_dbias: bool = False,
                        workspace=None, stream=None):
    """(dx, dw, dbias) of ada_linear: dz = dy act'(pre), dx = dz w, dw = dz^T x, dbias the
    sum of dz over rows; None for what is neither passed nor wanted.  `pre` is what
    ada_linear saved (not needed for act "none")."""
    if stream is not None:
        return _on(stream, ada_linear_backward, dy, x, w, pre, act, dx, dw, dbias, want_dx, want_dw, want_dbias,
                   workspace)
    rows, d_out, d_in = _sizes(x, w)
    code, dc, dt, dev = _act(act), _dtype(x), x.dtype, x.get_device()
    if code == 0:
        pre = None
    elif pre is None:
        raise ValueError("pre is needed for the slope of the activation")
    pdy, lddy = _mat(dy, rows, d_out, dt, dev, "dy")
    px, ldx = _mat(x, rows, d_in, dt, dev, "x")
    pw, ldw = _mat(w, d_out, d_in, dt, dev, "w")
    pp, ldp = _mat(pre, rows, d_out, dt, dev, "pre")
    pdx, lddx = _mat(dx, rows, d_in, dt, dev, "dx")
    pdw, lddw = _mat(dw, d_out, d_in, dt, dev, "dw")
    pdb = _vec(dbias, d_out, dt, dev, "dbias")
    _current(dev)
    if dx is None and want_dx:
        dx = torch.empty((rows, d_in), dtype=dt, device=x.device)
        pdx, lddx = dx.data_ptr(), d_in
    if dw is None and want_dw:
        dw = torch.empty((d_out, d_in), dtype=dt, device=x.device)
        pdw, lddw = dw.data_ptr(), d_in
    if dbias is None and want_dbias:
        dbias = torch.empty(d_out, dtype=dt, device=x.device)
        pdb = dbias.data_ptr()
    ws, nbytes, _keep = _workspace(_workspace_bytes("ada_linear_backward_workspace", rows, d_out, d_in, code, dc),
                                   workspace, dev)
    args = AdaLinearGradArgs(pdy, px, pw, pp, pdx, pdw, pdb, lddy, ldx, ldw, ldp, lddx, lddw, rows, d_out, d_in)
    _check(_lib.load().ada_linear_backward(args, code, dc, ws, nbytes, _raw_stream(dev)), "ada_linear_backward")
    return dx, dw, dbias


def ada_glu(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, bias_gate=None, bias_up=None,
            act: str = "silu", y=None, pre=None, workspace=None, stream=None):
    """y = act(g) u with g = x w_gate^T + bias_gate and u = x w_up^T + bias_up, in one pass;
    `pre`, if given, is a pair (g, u) of matrices to receive them for the backward pass."""
    if stream is not None:
        return _on(stream, ada_glu, x, w_gate, w_up, bias_gate, bias_up, act, y, pre, workspace)
    rows, d_out, d_in = _sizes(x, w_gate)
    code, dc, dt, dev = _act(act), _dtype(x), x.dtype, x.get_device()
    px, ldx = _mat(x, rows, d_in, dt, dev, "x")
    pg, ldg = _mat(w_gate, d_out, d_in, dt, dev, "w_gate")
    pu, ldu = _mat(w_up, d_out, d_in, dt, dev, "w_up")
    pbg = _vec(bias_gate, d_out, dt, dev, "bias_gate")
    pbu = _vec(bias_up, d_out, dt, dev, "bias_up")
    gate_pre, up_pre = pre if pre is not None else (None, None)
    ppg, ldpg = _mat(gate_pre, rows, d_out, dt, dev, "gate_pre")
    ppu, ldpu = _mat(up_pre, rows, d_out, dt, dev, "up_pre")
    if y is not None:
        py, ldy = _mat(y, rows, d_out, dt, dev, "y")
    _current(dev)
    if y is None:
        y = torch.empty((rows, d_out), dtype=dt, device=x.device)
        py, ldy = y.data_ptr(), d_out
    ws, nbytes, _keep = _workspace(_workspace_bytes("ada_glu_workspace", rows, d_out, d_in, dc), workspace, dev)
    args = AdaGluArgs(px, pg, pu, pbg, pbu, py, ppg, ppu, ldx, ldg, ldu, ldy, ldpg, ldpu, rows, d_out, d_in)
    _check(_lib.load().ada_glu(args, code, dc, ws, nbytes, _raw_stream(dev)), "ada_glu")
    return y


def ada_glu_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, gate_pre, up_pre,
                     act: str = "silu", dx=None, dw_gate=None, dw_up=None, dbias_gate=None, dbias_up=None,
                     want_dx: bool = True, want_dw: bool = True, want_dbias: bool = False, workspace=None,
                     stream=None):
    """(dx, dw_gate, dw_up, dbias_gate, dbias_up) of ada_glu, given g and u as it saved them:
    dg = dy u act'(g), du = dy act(g), dx = dg w_gate + du w_up, dw = d^T x, dbias the sums
    over rows; None for what is neither passed nor wanted."""
    if stream is not None:
        return _on(stream, ada_glu_backward, dy, x, w_gate, w_up, gate_pre, up_pre, act, dx, dw_gate, dw_up,
                   dbias_gate, dbias_up, want_dx, want_dw, want_dbias, workspace)
    rows, d_out, d_in = _sizes(x, w_gate)
    code, dc, dt, dev = _act(act), _dtype(x), x.dtype, x.get_device()
    if gate_pre is None or up_pre is None:
        raise ValueError("gate_pre and up_pre are needed for the slopes")
    pdy, lddy = _mat(dy, rows, d_out, dt, dev, "dy")
    px, ldx = _mat(x, rows, d_in, dt, dev, "x")
    pg, ldg = _mat(w_gate, d_out, d_in, dt, dev, "w_gate")
    pu, ldu = _mat(w_up, d_out, d_in, dt, dev, "w_up")
    ppg, ldpg = _mat(gate_pre, rows, d_out, dt, dev, "gate_pre")
    ppu, ldpu = _mat(up_pre, rows, d_out, dt, dev, "up_pre")
    pdx, lddx = _mat(dx, rows, d_in, dt, dev, "dx")
    pdg, lddg = _mat(dw_gate, d_out, d_in, dt, dev, "dw_gate")
    pdu, lddu = _mat(dw_up, d_out, d_in, dt, dev, "dw_up")
    pbg = _vec(dbias_gate, d_out, dt, dev, "dbias_gate")
    pbu = _vec(dbias_up, d_out, dt, dev, "dbias_up")
    _current(dev)

    def made(t, p, ld, *shape):
        if t is not None:
            return t, p, ld
        t = torch.empty(shape, dtype=dt, device=x.device)
        return t, t.data_ptr(), shape[-1]

    if want_dx:
        dx, pdx, lddx = made(dx, pdx, lddx, rows, d_in)
    if want_dw:
        dw_gate, pdg, lddg = made(dw_gate, pdg, lddg, d_out, d_in)
        dw_up, pdu, lddu = made(dw_up, pdu, lddu, d_out, d_in)
    if want_dbias:
        dbias_gate, pbg, _ = made(dbias_gate, pbg, 0, d_out)
        dbias_up, pbu, _ = made(dbias_up, pbu, 0, d_out)
    ws, nbytes, _keep = _workspace(_workspace_bytes("ada_glu_backward_workspace", rows, d_out, d_in, code, dc),
                                   workspace, dev)
    args = AdaGluGradArgs(pdy, px, pg, pu, ppg, ppu, pdx, pdg, pdu, pbg, pbu, lddy, ldx, ldg, ldu, ldpg, ldpu, lddx,
                          lddg, lddu, rows, d_out, d_in)
    _check(_lib.load().ada_glu_backward(args, code, dc, ws, nbytes, _raw_stream(dev)), "ada_glu_backward")
    return dx, dw_gate, dw_up, dbias_gate, dbias_up


# ---- norms, dropout, and the router for many rows ------------------------------------
_NORMS = {"layer": 0, "rms": 1}
_M64 = (1 << 64) - 1


def _kind(kind: str) -> int:
    try:
        return _NORMS[kind]
    except KeyError:
        raise ValueError(f"unknown norm {kind!r}; expected one of {', '.join(_NORMS)}") from None


def _drop(p: float, seed, offset: int, dev: int):
    """The C call's dropout; a seed that is a tensor is the generator's state on the device."""
    if seed is None:
        if p != 0:
            raise ValueError("dropout needs a seed")
        return 0.0, 0, 0, None
    if not isinstance(seed, torch.Tensor):
        return p, index(seed) & _M64, index(offset) & _M64, None
    if seed.dtype is not torch.int64 or seed.shape != (2,) or seed.stride(0) != 1:
        raise TypeError("a seed on the device must be int64 [2]: the seed and the offset's start")
    if seed.get_device() != dev:
        raise ValueError(f"seed is on {seed.device}, not with the other tensors")
    return p, 0, index(offset) & _M64, seed.data_ptr()


def _shape(x: torch.Tensor, name: str):
    s = x.shape
    if len(s) != 2:
        raise ValueError(f"{name} must be [rows, d]")
    return s


def _like(t, shape, dt, dev: int, name: str):
    """Pointer and row stride of a matrix of this shape (as _mat, which it leaves the rest to)."""
    if t is not None and t.shape == shape and t.dtype is dt and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), shape[1]
    return _mat(t, shape[0], shape[1], dt, dev, name)


def ada_dropout(x: torch.Tensor, p: float, seed, offset: int = 0, residual=None, y=None, stream=None):
    """y = residual + dropout(x) for x [rows, d]: an element is zero with probability p (to the nearest 2^-16),
    else divided by 1 - p.  y may be x or the residual itself.

    The mask is a function of (seed, offset), whole numbers, and the element's place, and is not stored: give the
    backward pass the same numbers, and every call of a step an offset of its own.  `seed` may be
    an int64 [2] tensor on the device, (seed, start of the offset): a captured call then draws
    anew whenever that tensor changes.  `stream` as in ada_linear."""
    if stream is not None:
        return _on(stream, ada_dropout, x, p, seed, offset, residual, y)
    shape = _shape(x, "x")
    rows, d = shape
    dc, dt, dev = _dtype(x), x.dtype, x.get_device()
    px, ldx = _like(x, shape, dt, dev, "x")
    pr, ldr = _like(residual, shape, dt, dev, "residual")
    if y is not None:
        py, ldy = _like(y, shape, dt, dev, "y")
    drop = _drop(p, seed, offset, dev)
    _current(dev)
    if y is None:
        y = torch.empty((rows, d), dtype=dt, device=x.device)
        py, ldy = y.data_ptr(), d
    args = AdaDropoutArgs(px, pr, py, ldx, ldr, ldy, rows, d, *drop)
    _check(_lib.load().ada_dropout(args, dc, _raw_stream(dev)), "ada_dropout")
    return y


def ada_dropout_backward(dy: torch.Tensor, p: float, seed, offset: int = 0, dx=None, stream=None):
    """dx of ada_dropout with the same p, seed and offset (dx may be dy itself); the gradient of
    the residual is dy."""
    if stream is not None:
        return _on(stream, ada_dropout_backward, dy, p, seed, offset, dx)
    shape = _shape(dy, "dy")
    rows, d = shape
    dc, dt, dev = _dtype(dy), dy.dtype, dy.get_device()
    pdy, lddy = _like(dy, shape, dt, dev, "dy")
    if dx is not None:
        pdx, lddx = _like(dx, shape, dt, dev, "dx")
    drop = _drop(p, seed, offset, dev)
    _current(dev)
    if dx is None:
        dx = torch.empty((rows, d), dtype=dt, device=dy.device)
        pdx, lddx = dx.data_ptr(), d
    args = AdaDropoutGradArgs(pdy, pdx, lddy, lddx, rows, d, *drop)
    _check(_lib.load().ada_dropout_backward(args, dc, _raw_stream(dev)), "ada_dropout_backward")
    return dx


def ada_norm(x: torch.Tensor, weight=None, bias=None, residual=None, kind: str = "layer", eps: float = 1e-5,
             p: float = 0.0, seed=None, offset: int = 0, y=None, hidden=None, stats=None, stream=None):
    """y = (h - mean) rstd weight + bias over each row of h = residual + dropout(x), for x [rows, d]
    with d at most 32768; kind "rms" has no mean.  rstd = 1 / sqrt(mean of (h - mean)^2 + eps).

    `hidden` receives h, the new residual stream; `stats` is a pair (mean, rstd) of fp32 [rows]
    vectors to receive them (either may be None), both for the backward pass.  y and hidden may be
    x or the residual itself.  p, seed and offset as in ada_dropout, `stream` as in ada_linear."""
    if stream is not None:
        return _on(stream, ada_norm, x, weight, bias, residual, kind, eps, p, seed, offset, y, hidden, stats)
    shape = _shape(x, "x")
    rows, d = shape
    code, dc, dt, dev = _kind(kind), _dtype(x), x.dtype, x.get_device()
    px, ldx = _like(x, shape, dt, dev, "x")
    pr, ldr = _like(residual, shape, dt, dev, "residual")
    pw = _vec(weight, d, dt, dev, "weight")
    pb = _vec(bias, d, dt, dev, "bias")
    ph, ldh = _like(hidden, shape, dt, dev, "hidden")
    mean, rstd = stats if stats is not None else (None, None)
    pm = _vec(mean, rows, torch.float32, dev, "mean")
    ps = _vec(rstd, rows, torch.float32, dev, "rstd")
    if y is not None:
        py, ldy = _like(y, shape, dt, dev, "y")
    drop = _drop(p, seed, offset, dev)
    _current(dev)
    if y is None:
        y = torch.empty((rows, d), dtype=dt, device=x.device)
        py, ldy = y.data_ptr(), d
    args = AdaNormArgs(px, pr, pw, pb, py, ph, pm, ps, ldx, ldr, ldy, ldh, rows, d, code, eps, *drop)
    _check(_lib.load().ada_norm(args, dc, _raw_stream(dev)), "ada_norm")
    return y


def norm_backward_workspace_bytes(rows: int, d: int, dtype: torch.dtype) -> int:
    """Bytes of workspace ada_norm_backward needs at these sizes (none without dweight and dbias)."""
    return _workspace_bytes("ada_norm_backward_workspace", rows, d, _DT[dtype])


def ada_norm_backward(dy: torch.Tensor, hidden: torch.Tensor, stats, weight=None, dhidden=None, kind: str = "layer",
                      p: float = 0.0, seed=None, offset: int = 0, dx=None, dresidual=None, dweight=None, dbias=None,
                      want_dx: bool = True, want_dresidual: bool = False, want_dweight: bool = True,
                      want_dbias: bool = False, workspace=None, stream=None):
    """(dx, dresidual, dweight, dbias) of ada_norm, given h and (mean, rstd) as it saved them (h is x
    where there was neither residual nor dropout) and `dhidden`, the gradient that reaches h past
    the norm; None for what is neither passed nor wanted.

    dresidual is the gradient of h, dx that behind the dropout: without dropout dx is both.  dx and
    dresidual may be dy or dhidden itself."""
    if stream is not None:
        return _on(stream, ada_norm_backward, dy, hidden, stats, weight, dhidden, kind, p, seed, offset, dx, dresidual,
                   dweight, dbias, want_dx, want_dresidual, want_dweight, want_dbias, workspace)
    shape = _shape(dy, "dy")
    rows, d = shape
    code, dc, dt, dev = _kind(kind), _dtype(dy), dy.dtype, dy.get_device()
    mean, rstd = stats
    if rstd is None or (mean is None and code == 0):
        raise ValueError("stats must hold what ada_norm saved: rstd, and mean unless the norm is rms")
    pdy, lddy = _like(dy, shape, dt, dev, "dy")
    ph, ldh = _like(hidden, shape, dt, dev, "hidden")
    pdh, lddh = _like(dhidden, shape, dt, dev, "dhidden")
    pw = _vec(weight, d, dt, dev, "weight")
    pm = _vec(mean, rows, torch.float32, dev, "mean")
    ps = _vec(rstd, rows, torch.float32, dev, "rstd")
    pdx, lddx = _like(dx, shape, dt, dev, "dx")
    pdr, lddr = _like(dresidual, shape, dt, dev, "dresidual")
    pdw = _vec(dweight, d, dt, dev, "dweight")
    pdb = _vec(dbias, d, dt, dev, "dbias")
    drop = _drop(p, seed, offset, dev)
    _current(dev)
    if dx is None and want_dx:
        dx = torch.empty((rows, d), dtype=dt, device=dy.device)
        pdx, lddx = dx.data_ptr(), d
    if dresidual is None and want_dresidual:
        dresidual = torch.empty((rows, d), dtype=dt, device=dy.device)
        pdr, lddr = dresidual.data_ptr(), d
    if dweight is None and want_dweight:
        dweight = torch.empty(d, dtype=dt, device=dy.device)
        pdw = dweight.data_ptr()
    if dbias is None and want_dbias:
        dbias = torch.empty(d, dtype=dt, device=dy.device)
        pdb = dbias.data_ptr()
    need = 0 if dweight is None and dbias is None else _workspace_bytes("ada_norm_backward_workspace", rows, d, dc)
    ws, nbytes, _keep = _workspace(need, workspace, dev)
    args = AdaNormGradArgs(pdy, ph, pdh, pw, pm, ps, pdx, pdr, pdw, pdb, lddy, ldh, lddh, lddx, lddr, rows, d, code,
                           *drop)
    _check(_lib.load().ada_norm_backward(args, dc, ws, nbytes, _raw_stream(dev)), "ada_norm_backward")
    return dx, dresidual, dweight, dbias


class Routing(NamedTuple):
    """What ada_route writes.  The last four are None where no balance was asked for."""

    idx: torch.Tensor      # int32 [rows, k], -1 where nothing was picked
    gate: torch.Tensor     # fp32 [rows, k]
    counts: torch.Tensor   # int32 [E]: rows that picked each expert
    prob: torch.Tensor     # fp32 [E]: mean probability of each
    loss: torch.Tensor     # fp32 [1]: the balance loss
    used: torch.Tensor     # int32 [1]: the rows that count


def _table(t: torch.Tensor, shape, dt, dev: int, name: str):
    """Pointer of a contiguous table."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dt or t.get_device() != dev:
        _refuse(t, shape, dt, dev, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def route_workspace_bytes(rows: int, E: int) -> int:
    """Bytes of workspace ada_route needs at these sizes (none without a balance)."""
    return _workspace_bytes("ada_route_workspace", rows, E)


def ada_route(logits: torch.Tensor, k: int, renorm: bool = True, valid=None, balance: bool = True, out=None,
              workspace=None, stream=None) -> Routing:
    """ada_pregate's choice for every row of logits [rows, E], and the balance the router is
    trained on: how many rows picked each expert, the mean probability of each, and
    loss = E sum_e (counts_e / (k n)) prob_e over the n rows that count.

    A logit of -inf closes its expert to the row.  `valid` (bool or uint8 [rows]) marks the rows that
    count; the others, rows with every expert closed, and slots without an open expert left get
    index -1 and gate 0.  `out` is a Routing (or six tensors; without balance the last four may be None) to write
    to; `stream` as in ada_linear."""
    if stream is not None:
        return _on(stream, ada_route, logits, k, renorm, valid, balance, out, workspace)
    rows, E = _shape(logits, "logits")
    dc, dev = _dtype(logits), logits.get_device()
    pl, ld = _mat(logits, rows, E, logits.dtype, dev, "logits")
    pv = None
    if valid is not None:
        if valid.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"valid must be bool or uint8, got {valid.dtype}")
        pv = _vec(valid, rows, valid.dtype, dev, "valid")
    i32, f32 = torch.int32, torch.float32
    if out is None:
        _current(dev)
        one = logits.device
        out = Routing(torch.empty((rows, k), dtype=i32, device=one), torch.empty((rows, k), dtype=f32, device=one),
                      *((torch.empty(E, dtype=i32, device=one), torch.empty(E, dtype=f32, device=one),
                         torch.empty(1, dtype=f32, device=one), torch.empty(1, dtype=i32, device=one))
                        if balance else (None,) * 4))
    else:
        out = Routing(*out)
    pi = _table(out.idx, (rows, k), i32, dev, "idx")
    pg = _table(out.gate, (rows, k), f32, dev, "gate")
    pc = pp = po = pu = None
    if not balance:
        out = Routing(out.idx, out.gate, None, None, None, None)
    else:
        pc = _vec(out.counts, E, i32, dev, "counts")
        pp = _vec(out.prob, E, f32, dev, "prob")
        po = _vec(out.loss, 1, f32, dev, "loss")
        pu = _vec(out.used, 1, i32, dev, "used")
        if pc is None or pp is None or po is None or pu is None:
            raise ValueError("out has no tensors for the balance: counts, prob, loss and used are needed")
    _current(dev)
    ws, nbytes, _keep = _workspace(_workspace_bytes("ada_route_workspace", rows, E) if balance else 0, workspace, dev)
    args = AdaRouteArgs(pl, pv, pi, pg, pc, pp, po, pu, ld, rows, E, k, bool(renorm))
    _check(_lib.load().ada_route(args, dc, ws, nbytes, _raw_stream(dev)), "ada_route")
    return out


def ada_route_backward(logits: torch.Tensor, out, dgate=None, dloss=None, renorm: bool = True, dlogits=None,
                       stream=None):
    """dlogits of ada_route, given its logits and what it wrote: `dgate` (fp32 [rows, k]) is the
    gradient of the gates, `dloss` (fp32 [1]) that of the loss; either may be None.  The counts
    are constants."""
    if stream is not None:
        return _on(stream, ada_route_backward, logits, out, dgate, dloss, renorm, dlogits)
    rows, E = _shape(logits, "logits")
    dc, dt, dev = _dtype(logits), logits.dtype, logits.get_device()
    idx, gate, counts, _, _, used = out
    i32, f32 = torch.int32, torch.float32
    if idx.dim() != 2:
        raise ValueError("idx must be [rows, k]")
    k = idx.shape[1]
    if dgate is None and dloss is None:
        raise ValueError("dgate or dloss is needed")
    pl, ld = _mat(logits, rows, E, dt, dev, "logits")
    pi = _table(idx, (rows, k), i32, dev, "idx")
    pg = _table(gate, (rows, k), f32, dev, "gate")
    pdg = _table(dgate, (rows, k), f32, dev, "dgate")
    pc = pu = pdl = None
    if dloss is not None:
        if counts is None or used is None:
            raise ValueError("the loss was not computed: ada_route was called without balance")
        pc = _vec(counts, E, i32, dev, "counts")
        pu = _vec(used, 1, i32, dev, "used")
        pdl = _vec(dloss, 1, f32, dev, "dloss")
    if dlogits is not None:
        po, ldo = _mat(dlogits, rows, E, dt, dev, "dlogits")
    _current(dev)
    if dlogits is None:
        dlogits = torch.empty((rows, E), dtype=dt, device=logits.device)
        po, ldo = dlogits.data_ptr(), E
    args = AdaRouteGradArgs(pl, pi, pg, pc, pu, pdg, pdl, po, ld, ldo, rows, E, k, bool(renorm))
    _check(_lib.load().ada_route_backward(args, dc, _raw_stream(dev)), "ada_route_backward")
    return dlogits
