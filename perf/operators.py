"""The products around a decoder layer's projections, as cases to measure: linear (bias, activation and residual in
one pass), the gated feed-forward pair, and the backward pass of both.

Layouts: x [rows, d_in], weights [d_out, d_in] (y = x W^T), everything of one storage type (bf16 or fp32).
  linear           z = x W^T + b, y = act(z) + residual
  linear_backward  dz = dy act'(z), dx = dz W, dw = dz^T x, dbias = sum over rows of dz
  glu              g = x Wg^T + bg, u = x Wu^T + bu, y = act(g) u
  glu_backward     dg = dy u act'(g), du = dy act(g), dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, and the biases'
The backward calls take z, g and u as the forward calls saved them, in the storage type.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
_TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
_SIZES = {BF16: 2, FP32: 4}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _case(name, op, rows, d_out, d_in, act, dtype, bias=False, residual=False, save=False):
    c = {"op": op, "rows": rows, "d_out": d_out, "d_in": d_in, "act": act, "dtype": dtype, "bias": bias,
         "residual": residual, "save": save}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decode token through the 7B-shaped output projection, added to the residual stream
        _case("linear_decode", "linear", 1, 4096, 4096, "none", BF16, residual=True),
        # 24 requests decoding together through the 7B-shaped down projection
        _case("linear_decode_batch", "linear", 24, 4096, 11008, "none", BF16, residual=True),
        # a prompt of odd length through a biased projection with its activation
        _case("linear_prompt_ragged", "linear", 509, 4096, 4096, "gelu", BF16, bias=True),
        # a long prompt through the 70B-shaped down projection, added to the residual stream
        _case("linear_prompt_long", "linear", 4096, 8192, 28672, "none", BF16, residual=True),
        # a small stack kept in fp32, sizes off every power of two, everything in the epilogue
        _case("linear_fp32", "linear", 300, 1032, 2056, "gelu_tanh", FP32, bias=True, residual=True),
        # training one biased projection on sequences of odd length
        _case("linear_backward", "linear_backward", 2047, 4096, 4096, "gelu", BF16, bias=True, save=True),
        # the same in fp32 on a small stack
        _case("linear_backward_fp32", "linear_backward", 257, 1288, 520, "silu", FP32, bias=True, save=True),
        # one decode token through the 7B-shaped gate and up projections
        _case("glu_decode", "glu", 1, 11008, 4096, "silu", BF16),
        # 48 requests on one GPU's eighth of the 70B-shaped gate and up projections
        _case("glu_decode_batch", "glu", 48, 3584, 8192, "silu", BF16),
        # the forward pass of a training step, which keeps what its backward pass reads
        _case("glu_train", "glu", 4096, 11008, 4096, "silu", BF16, save=True),
        # ... and that backward pass
        _case("glu_backward", "glu_backward", 4096, 11008, 4096, "silu", BF16, save=True),
        # a small gated block with biases in fp32
        _case("glu_backward_fp32", "glu_backward", 333, 1032, 520, "gelu_tanh", FP32, bias=True, save=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("linear", "linear", "linear_backward", "glu", "glu", "glu_backward"))
    dtype = rng.choice((BF16, BF16, BF16, FP32))
    most = 2.0 ** 38 if dtype == BF16 else 2.0 ** 33  # rows * d_out * d_in * products
    products = {"linear": 1, "linear_backward": 2, "glu": 2, "glu_backward": 4}[op]
    while True:
        rows = spread(1, 4096)
        d_out, d_in = 8 * spread(8, 3584), 8 * spread(8, 3584)
        if rows * d_out * d_in * products <= most and d_out * d_in <= 28672 * 8192:
            break
    acts = _ACTS[1:] if op.startswith("glu") else _ACTS
    return _case(None, op, rows, d_out, d_in, rng.choice(acts), dtype, bias=rng.random() < 0.5,
                 residual=op == "linear" and rng.random() < 0.5,
                 save=op.endswith("backward") or rng.random() < 0.3)


def prepare(case, seed):
    dt = _TYPES[case["dtype"]]
    rows, n, k = case["rows"], case["d_out"], case["d_in"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dt)

    def out(*shape):
        return torch.empty(shape, dtype=dt, device="cuda")

    s = {"case": case, "x": normal((rows, k), 1.0)}  # hidden states behind a norm
    gated = case["op"].startswith("glu")
    names = ("gate", "up") if gated else ("",)
    for p in names:
        s["w" + p] = normal((n, k), 0.02)
        s["b" + p] = normal((n,), 0.1) if case["bias"] else None
        if case["op"].endswith("backward"):  # the pre-activations that the forward pass kept
            z = s["x"].float() @ s["w" + p].float().t()
            s["pre" + p] = (z + s["b" + p].float() if case["bias"] else z).to(dt)
            s["dw" + p] = out(n, k)
            s["db" + p] = out(n) if case["bias"] else None
        else:
            s["pre" + p] = out(rows, n) if case["save"] else None
    if case["op"].endswith("backward"):
        s["dy"] = normal((rows, n), 0.05)
        s["dx"] = out(rows, k)
    else:
        s["residual"] = normal((rows, n), 1.0) if case["residual"] else None
        s["y"] = out(rows, n)
    return s


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _product(x, w, b):
    z = x.float() @ w.float().t()
    return z if b is None else z + b.float()


def _plain(s):
    c = s["case"]
    op, act, dt = c["op"], c["act"], s["x"].dtype
    if op == "linear":
        z = _product(s["x"], s["w"], s["b"])
        y = _act(z, act)
        y = y if s["residual"] is None else y + s["residual"].float()
        return {"y": y.to(dt), **({"pre": z.to(dt)} if c["save"] else {})}
    if op == "glu":
        g, u = _product(s["x"], s["wgate"], s["bgate"]), _product(s["x"], s["wup"], s["bup"])
        y = (_act(g, act) * u).to(dt)
        return {"y": y, **({"pregate": g.to(dt), "preup": u.to(dt)} if c["save"] else {})}
    x, dy = s["x"].float(), s["dy"].float()
    if op == "linear_backward":
        dz = dy * _slope(s["pre"].float(), act)
        got = {"dx": dz @ s["w"].float(), "dw": dz.t() @ x}
        if c["bias"]:
            got["db"] = dz.sum(0, dtype=torch.float64)
    else:
        g, u = s["pregate"].float(), s["preup"].float()
        dg, du = dy * u * _slope(g, act), dy * _act(g, act)
        got = {"dx": dg @ s["wgate"].float() + du @ s["wup"].float(), "dwgate": dg.t() @ x, "dwup": du.t() @ x}
        if c["bias"]:
            got["dbgate"], got["dbup"] = dg.sum(0, dtype=torch.float64), du.sum(0, dtype=torch.float64)
    return {k: v.to(dt) for k, v in got.items()}


def _framework(s):
    import weight_merge_amd as ada

    c = s["case"]
    op, act = c["op"], c["act"]
    if op == "linear":
        ada.ada_linear(s["x"], s["w"], bias=s["b"], residual=s["residual"], act=act, y=s["y"], pre=s["pre"])
        return {"y": s["y"], **({"pre": s["pre"]} if c["save"] else {})}
    if op == "glu":
        pre = (s["pregate"], s["preup"]) if c["save"] else None
        ada.ada_glu(s["x"], s["wgate"], s["wup"], bias_gate=s["bgate"], bias_up=s["bup"], act=act, y=s["y"], pre=pre)
        return {"y": s["y"], **({"pregate": s["pregate"], "preup": s["preup"]} if c["save"] else {})}
    if op == "linear_backward":
        ada.ada_linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], act=act, dx=s["dx"], dw=s["dw"], dbias=s["db"])
        return {"dx": s["dx"], "dw": s["dw"], **({"db": s["db"]} if c["bias"] else {})}
    ada.ada_glu_backward(s["dy"], s["x"], s["wgate"], s["wup"], s["pregate"], s["preup"], act=act, dx=s["dx"],
                         dw_gate=s["dwgate"], dw_up=s["dwup"], dbias_gate=s["dbgate"], dbias_up=s["dbup"])
    return {"dx": s["dx"], "dwgate": s["dwgate"], "dwup": s["dwup"],
            **({"dbgate": s["dbgate"], "dbup": s["dbup"]} if c["bias"] else {})}


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    e, r, n, k = _SIZES[case["dtype"]], case["rows"], case["d_out"], case["d_in"]
    parts = 2 if case["op"].startswith("glu") else 1
    bias = parts * n if case["bias"] else 0
    if case["op"].endswith("backward"):
        # dy and the saved pre-activations (a linear product without an activation reads none), x, w; dx, dw, dbias
        saved = parts if case["op"] == "glu_backward" or case["act"] != "none" else 0
        values = r * n * (1 + saved) + r * k + parts * n * k + r * k + parts * n * k + bias
        return {"bytes": e * values, "flops": 4 * parts * r * n * k}
    values = r * k + parts * n * k + bias + r * n * (1 + bool(case["residual"]) + (parts if case["save"] else 0))
    return {"bytes": e * values, "flops": 2 * parts * r * n * k}


def exact(case, seed):
    """The definition in 64 bits; the slopes come from differentiating the activation itself."""
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}

    def activation(t):
        name = case["act"]
        if name == "silu":
            return t * torch.sigmoid(t)
        if name == "gelu":
            return t * (1 + torch.erf(t / 2 ** 0.5)) / 2
        if name == "gelu_tanh":
            return t / 2 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3)))
        return torch.where(t > 0, t, torch.zeros_like(t)) if name == "relu" else t * 1

    def affine(p):
        t = torch.mm(v["x"], v["w" + p].t().contiguous())
        return t if s["b" + p] is None else t + v["b" + p][None, :]

    if case["op"] == "linear":
        z = affine("")
        y = activation(z)
        if s["residual"] is not None:
            y = y + v["residual"]
        return {"y": y, "pre": z} if case["save"] else {"y": y}
    if case["op"] == "glu":
        g, u = affine("gate"), affine("up")
        y = activation(g) * u
        return {"y": y, "pregate": g, "preup": u} if case["save"] else {"y": y}
    names = ("gate", "up") if case["op"] == "glu_backward" else ("",)
    leaves = [v["pre" + p].requires_grad_() for p in names]
    out = activation(leaves[0]) if len(leaves) == 1 else activation(leaves[0]) * leaves[1]
    slopes = torch.autograd.grad(out, leaves, v["dy"])
    got = {"dx": sum(torch.mm(d, v["w" + p]) for p, d in zip(names, slopes))}
    for p, d in zip(names, slopes):
        got["dw" + p] = torch.mm(d.t().contiguous(), v["x"])
        if case["bias"]:
            got["db" + p] = d.sum(0)
    return got
