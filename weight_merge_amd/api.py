"""Python binding of libadafuse: argument marshalling only.

Every computation runs in the HIP kernels behind the C ABI; this module turns torch
tensors (device memory) and the current torch stream into the pointers and sizes the
C calls take, and turns negative status codes into exceptions.  Output tensors a
caller does not pass are allocated here with torch, outside the C calls.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import (ADA_BF16, ADA_F32, AdaGemvProj, AdaGluArgs, AdaGluGradArgs, AdaLinearArgs, AdaLinearGradArgs,
                   AdaLoraProj, AdaProj)

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
    if t.shape != (rows, cols) or t.dtype is not dt or t.get_device() != dev or t.stride(1) != 1:
        _refuse(t, (rows, cols), dt, dev, name)
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def _vec(t, n: int, dt, dev: int, name: str):
    """Pointer of an [n] vector."""
    if t is None:
        return None
    if t.shape != (n,) or t.dtype is not dt or t.get_device() != dev or t.stride(0) != 1:
        _refuse(t, (n,), dt, dev, name)
    return t.data_ptr()


def _sizes(x: torch.Tensor, w: torch.Tensor):
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [rows, d_in] and the weights [d_out, d_in]")
    return x.shape[0], w.shape[0], w.shape[1]


def _current(dev: int):
    if dev < 0:
        raise ValueError("tensors must be on the device")
    if dev != torch.cuda.current_device():
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
