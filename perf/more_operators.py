"""What stands around the projections of a routed decoder layer, as cases to measure: the norms with the residual stream
and the dropout before them, dropout by itself, and the router's choice with its balance loss; each with its backward pass.

Matrices are row-major; x, y, weights and gradients of one storage type (bf16 or fp32), statistics, gates and losses fp32.
  norm              h = residual + dropout(x), mean and rstd over a row of h, y = (h - mean) rstd w + b ("rms" has no mean)
  norm_backward     dh = dhidden + the gradient through the norm, dresidual = dh, dx = dropout(dh), dw, db: sums over rows
  dropout           y = residual + x keep / (1 - p); keep from a counter-based generator, the same wherever it is asked for
  dropout_backward  dx = dy keep / (1 - p)
  route             the k largest of a row's E logits, their gates (softmax), how often each expert was picked, the mean
                    probability of each, and the balance loss E sum_e f_e P_e
  route_backward    dlogits from the gradients of the gates and of the loss

The generator is Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011): counter
(g, offset) and key seed, 64 bits each; its four words are the eight 16-bit numbers of elements 8 g .. 8 g + 7 of the
matrix (row-major, without what lies between rows), low half first. An element is kept where its number is at least
round(65536 p), and scaled by 65536 / (65536 - round(65536 p)).
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
_TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
_SIZES = {BF16: 2, FP32: 4}
_M32 = 0xFFFFFFFF
_MULTIPLY = (0xD2511F53, 0xCD9E8D57)
_WEYL = (0x9E3779B9, 0xBB67AE85)


def _norm(name, op, rows, cols, kind, dtype, p=0.0, residual=False, bias=False, save=False):
    c = {"op": op, "rows": rows, "cols": cols, "kind": kind, "dtype": dtype, "p": p, "residual": residual, "bias": bias,
         "save": save}
    return {"name": name, **c} if name else c


def _dropout(name, op, rows, cols, dtype, p, residual=False):
    c = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual}
    return {"name": name, **c} if name else c


def _route(name, op, rows, experts, k, dtype, renorm=True, padded=False, closed=False):
    c = {"op": op, "rows": rows, "experts": experts, "k": k, "dtype": dtype, "renorm": renorm, "padded": padded,
         "closed": closed}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decode token of the 7B-shaped stack: the residual stream is added to and normed
        _norm("norm_decode", "norm", 1, 4096, "rms", BF16, residual=True),
        # a training step's rows of the 70B-shaped stack, dropout on what the block before gave
        _norm("norm_train", "norm", 4096, 8192, "layer", BF16, p=0.1, residual=True, bias=True, save=True),
        # a small stack kept in fp32, sizes off every power of two
        _norm("norm_fp32", "norm", 300, 1032, "layer", FP32, bias=True, save=True),
        # the backward pass of norm_train
        _norm("norm_backward", "norm_backward", 4096, 8192, "layer", BF16, p=0.1, residual=True, bias=True),
        # sequences of odd length through the 7B-shaped stack's norm
        _norm("norm_backward_rms", "norm_backward", 2047, 4096, "rms", BF16, residual=True),
        # the small stack's
        _norm("norm_backward_fp32", "norm_backward", 257, 520, "layer", FP32, bias=True),
        # a prompt of odd length, added to the residual stream
        _dropout("dropout_residual", "dropout", 509, 4096, BF16, 0.1, residual=True),
        # inside the feed-forward block of the 70B-shaped stack
        _dropout("dropout_wide", "dropout", 4096, 28672, BF16, 0.05),
        # its backward pass on a small fp32 stack
        _dropout("dropout_backward_fp32", "dropout_backward", 2047, 1032, FP32, 0.1),
        # 48 requests of the 7B-shaped stack with eight adapters
        _route("route_requests", "route", 48, 8, 2, BF16),
        # a training step that routes every token, the largest bank, padded sequences, experts closed to some tokens
        _route("route_train", "route", 16384, 64, 8, FP32, padded=True, closed=True),
        # the backward pass with sixteen adapters and four of them picked
        _route("route_backward", "route_backward", 8191, 16, 4, BF16, padded=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "norm", "norm_backward", "norm_backward", "dropout", "dropout_backward", "route",
                     "route_backward"))
    dtype = rng.choice((BF16, BF16, FP32))
    if op.startswith("route"):
        experts = spread(2, 64)
        return _route(None, op, spread(1, 32768), experts, rng.randint(1, min(experts, 8)), dtype,
                      renorm=rng.random() < 0.7, padded=rng.random() < 0.5, closed=rng.random() < 0.3)
    most = 4096 * 8192 if op.startswith("norm") else 4096 * 28672
    while True:
        rows, cols = spread(1, 16384), 8 * spread(1, 3584)
        if rows * cols * _SIZES[dtype] <= most * 2:
            break
    p = rng.choice((0.0, 0.0, round(rng.uniform(0.01, 0.5), 3))) if op.startswith("norm") else round(rng.uniform(0.01, 0.5), 3)
    if op.startswith("dropout"):
        return _dropout(None, op, rows, cols, dtype, p, residual=op == "dropout" and rng.random() < 0.5)
    kind = rng.choice(("layer", "rms"))
    return _norm(None, op, rows, cols, kind, dtype, p=p, residual=p > 0 or rng.random() < 0.5, bias=kind == "layer",
                 save=op == "norm" and rng.random() < 0.5)


def prepare(case, seed):
    dt = _TYPES[case["dtype"]]
    rows, op = case["rows"], case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std=1.0, mean=0.0, to=dt):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen).to(to)

    def out(*shape, to=dt):
        return torch.empty(shape, dtype=to, device="cuda")

    s = {"case": case}
    if op.startswith("route"):
        e, k = case["experts"], case["k"]
        logits = normal((rows, e), 1.0, to=torch.float32)
        logits += normal((e,), 0.7, to=torch.float32)  # some experts are liked better
        if case["closed"]:
            logits[normal((rows, e), to=torch.float32) > 1.0] = -math.inf
        s["logits"] = logits.to(dt)
        # the end of a sequence is padding, about one row in eight
        s["valid"] = (torch.arange(rows, device="cuda") % 512 < 448) if case["padded"] else None
        if op == "route":
            s["out"] = (out(rows, k, to=torch.int32), out(rows, k, to=torch.float32), out(e, to=torch.int32),
                        out(e, to=torch.float32), out(1, to=torch.float32), out(1, to=torch.int32))
        else:
            s["out"] = tuple(_plain_route(s).values())
            s["dgate"] = normal((rows, k), 0.1, to=torch.float32)
            s["dloss"] = torch.full((1,), 0.01, dtype=torch.float32, device="cuda")
            s["dlogits"] = out(rows, e)
        return s
    cols, p = case["cols"], case["p"]
    # one generator a run, a step and a call of it; the norms of a step keep it on the device
    s["seed"], s["offset"] = (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63, 7 * seed + 3
    spread = torch.exp(normal((cols,), 0.5, to=torch.float32))  # the residual stream has channels of many sizes
    if op == "norm":
        s["state"] = torch.tensor([s["seed"], s["offset"]], dtype=torch.int64, device="cuda") if p else None
        s["x"] = normal((rows, cols), 1.0, 0.1)
        s["residual"] = (normal((rows, cols), 2.0, 0.1, to=torch.float32) * spread).to(dt) if case["residual"] else None
        s["weight"], s["bias"] = normal((cols,), 0.1, 1.0), normal((cols,), 0.1) if case["bias"] else None
        s["y"] = out(rows, cols)
        s["hidden"] = out(rows, cols) if case["residual"] else None
        s["stats"] = (out(rows, to=torch.float32) if case["kind"] == "layer" else None, out(rows, to=torch.float32)) \
            if case["save"] else None
    elif op == "norm_backward":
        s["state"] = torch.tensor([s["seed"], s["offset"]], dtype=torch.int64, device="cuda") if p else None
        s["hidden"] = (normal((rows, cols), 2.0, 0.1, to=torch.float32) * spread).to(dt)
        s["weight"] = normal((cols,), 0.1, 1.0)
        s["stats"] = _statistics(s["hidden"].float(), case["kind"])
        s["dy"] = normal((rows, cols), 0.05)
        s["dhidden"] = normal((rows, cols), 0.05) if case["residual"] else None
        s["dx"], s["dw"] = out(rows, cols), out(cols)
        s["dresidual"] = out(rows, cols) if p else None  # without dropout dx is the residual's gradient too
        s["db"] = out(cols) if case["bias"] else None
    elif op == "dropout":
        s["x"] = normal((rows, cols), 1.0)
        s["residual"] = (normal((rows, cols), 2.0, to=torch.float32) * spread).to(dt) if case["residual"] else None
        s["y"] = out(rows, cols)
    else:
        s["dy"] = normal((rows, cols), 0.05)
        s["dx"] = out(rows, cols)
    return s


_EPS = 1e-5


def _statistics(h, kind):
    mean = h.mean(1) if kind == "layer" else None
    square = (h * h if mean is None else (h - mean[:, None]) ** 2).mean(1)
    return mean, 1.0 / torch.sqrt(square + _EPS)


def _kept(rows, cols, p, seed, offset, device="cuda"):
    """1 / (1 - p) where an element is kept, else 0; seed and offset are whole numbers or tensors of one."""
    least = int(round(65536 * p))
    g = torch.arange(rows * cols // 8, dtype=torch.int64, device=device)
    c = [g & _M32, g >> 32, (offset & _M32) + torch.zeros_like(g), ((offset >> 32) & _M32) + torch.zeros_like(g)]
    key = [seed & _M32, (seed >> 32) & _M32]
    for r in range(10):
        a, b = c[0] * _MULTIPLY[0], c[2] * _MULTIPLY[1]  # modulo 2^64
        c = [((b >> 32) & _M32) ^ c[1] ^ key[0], b & _M32, ((a >> 32) & _M32) ^ c[3] ^ key[1], a & _M32]
        key = [(q + w) & _M32 for q, w in zip(key, _WEYL)]
    halves = [h for w in c for h in (w & 0xFFFF, w >> 16)]
    numbers = torch.stack(halves, 1).reshape(rows, cols)
    return torch.where(numbers >= least, 65536.0 / (65536 - least), 0.0)


def _drop(v, keep):
    return torch.where(keep > 0, v * keep, 0.0)  # what is dropped is zero, whatever it was


def _plain_route(s):
    c, z = s["case"], s["logits"].float()
    rows, e, k = z.shape[0], c["experts"], c["k"]
    open_ = z > -math.inf
    used = open_.any(1) if s["valid"] is None else open_.any(1) & s["valid"]
    top = torch.where(used, z.max(1).values, 0.0)
    x = torch.where(open_ & used[:, None], torch.exp(z - top[:, None]), 0.0)
    total = torch.where(used, x.sum(1), 1.0)
    prob = x / total[:, None]
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]  # equal logits: the lower index first
    picked = torch.gather(open_, 1, order) & used[:, None]
    gate = torch.where(picked, torch.gather(x if c["renorm"] else prob, 1, order), 0.0)
    if c["renorm"]:
        gate = gate / torch.where(used, gate.sum(1), 1.0)[:, None]
    idx = torch.where(picked, order, -1)
    counts = (idx[:, :, None] == torch.arange(e, device=z.device)).sum((0, 1))
    n = used.sum()
    some = torch.clamp(n, min=1)
    mean = prob.sum(0, dtype=torch.float64) / some
    loss = e * (counts.double() / (k * some) * mean).sum().reshape(1)
    return {"idx": idx.int(), "gate": gate, "counts": counts.int(), "prob": mean.float(), "loss": loss.float(),
            "used": n.int().reshape(1)}


def _plain(s):
    c = s["case"]
    op, dt = c["op"], _TYPES[c["dtype"]]
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        idx, gate, counts, _, _, used = s["out"]
        z, e, k = s["logits"].float(), c["experts"], c["k"]
        rows_used, picked = idx[:, 0] >= 0, idx >= 0
        at = torch.where(picked, idx, 0).long()
        top = torch.where(rows_used, z.max(1).values, 0.0)
        x = torch.where(rows_used[:, None], torch.exp(z - top[:, None]), 0.0)
        prob = x / torch.where(rows_used, x.sum(1), 1.0)[:, None]
        some = torch.clamp(used, min=1).double()
        dprob = (s["dloss"] * (e * counts.double() / (k * some * some))).float().expand_as(prob)
        dgate = torch.where(picked, s["dgate"], 0.0)
        grad = torch.zeros_like(z)
        if c["renorm"]:
            inner = gate * (dgate - (gate * dgate).sum(1, keepdim=True))
            grad.scatter_add_(1, at, torch.where(picked, inner, 0.0))
        else:
            dprob = dprob.scatter_add(1, at, dgate)
        grad += prob * (dprob - (prob * dprob).sum(1, keepdim=True))
        return {"dlogits": grad.to(dt)}
    rows, cols, p = c["rows"], c["cols"], c["p"]
    if op == "dropout":
        y = _drop(s["x"].float(), _kept(rows, cols, p, s["seed"], s["offset"]))
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(dt)}
    if op == "dropout_backward":
        return {"dx": _drop(s["dy"].float(), _kept(rows, cols, p, s["seed"], s["offset"])).to(dt)}
    keep = _kept(rows, cols, p, s["state"][0], s["state"][1]) if p else None
    w = s["weight"].float()
    if op == "norm":
        h = s["x"].float()
        h = _drop(h, keep) if p else h
        h = h if s["residual"] is None else h + s["residual"].float()
        mean, rstd = _statistics(h, c["kind"])
        y = (h if mean is None else h - mean[:, None]) * rstd[:, None] * w
        got = {"y": (y if s["bias"] is None else y + s["bias"].float()).to(dt)}
        if c["residual"]:
            got["hidden"] = h.to(dt)
        if c["save"]:
            got["rstd"] = rstd
            if mean is not None:
                got["mean"] = mean
        return got
    mean, rstd = s["stats"]
    h, dy = s["hidden"].float(), s["dy"].float()
    xhat = (h if mean is None else h - mean[:, None]) * rstd[:, None]
    t = dy * w
    inner = t - xhat * (t * xhat).mean(1, keepdim=True)
    dh = rstd[:, None] * (inner if mean is None else inner - t.mean(1, keepdim=True))
    dh = dh if s["dhidden"] is None else dh + s["dhidden"].float()
    got = {"dx": (_drop(dh, keep) if p else dh).to(dt), "dw": (dy * xhat).sum(0, dtype=torch.float64).to(dt)}
    if p:
        got["dresidual"] = dh.to(dt)
    if c["bias"]:
        got["db"] = dy.sum(0, dtype=torch.float64).to(dt)
    return got


def _framework(s):
    import weight_merge_amd as ada

    c = s["case"]
    op = c["op"]
    if op == "route":
        out = ada.ada_route(s["logits"], c["k"], renorm=c["renorm"], valid=s["valid"], out=s["out"])
        return dict(zip(("idx", "gate", "counts", "prob", "loss", "used"), out))
    if op == "route_backward":
        ada.ada_route_backward(s["logits"], s["out"], dgate=s["dgate"], dloss=s["dloss"], renorm=c["renorm"],
                               dlogits=s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "dropout":
        ada.ada_dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"], y=s["y"])
        return {"y": s["y"]}
    if op == "dropout_backward":
        ada.ada_dropout_backward(s["dy"], c["p"], s["seed"], s["offset"], dx=s["dx"])
        return {"dx": s["dx"]}
    if op == "norm":
        ada.ada_norm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], kind=c["kind"], eps=_EPS, p=c["p"],
                     seed=s["state"], y=s["y"], hidden=s["hidden"], stats=s["stats"])
        got = {"y": s["y"]}
        if c["residual"]:
            got["hidden"] = s["hidden"]
        if c["save"]:
            got["rstd"] = s["stats"][1]
            if c["kind"] == "layer":
                got["mean"] = s["stats"][0]
        return got
    ada.ada_norm_backward(s["dy"], s["hidden"], s["stats"], s["weight"], dhidden=s["dhidden"], kind=c["kind"], p=c["p"],
                          seed=s["state"], dx=s["dx"], dresidual=s["dresidual"], dweight=s["dw"], dbias=s["db"])
    return {"dx": s["dx"], "dw": s["dw"], **({"dresidual": s["dresidual"]} if c["p"] else {}),
            **({"db": s["db"]} if c["bias"] else {})}


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    e, rows, op = _SIZES[case["dtype"]], case["rows"], case["op"]
    if op.startswith("route"):
        n, k = case["experts"], case["k"]
        if op == "route":
            # logits and the rows' flags; indexes and gates; counts, probabilities, loss, rows
            return {"bytes": rows * (n * e + 8 * k + bool(case["padded"])) + 8 * n + 8, "flops": 6 * rows * n}
        # logits, indexes, gates and their gradients, counts, dloss, rows; dlogits
        return {"bytes": rows * (2 * n * e + 12 * k) + 4 * n + 8, "flops": 8 * rows * n}
    cols, p = case["cols"], case["p"]
    if op.startswith("dropout"):
        return {"bytes": e * rows * cols * (2 + bool(case["residual"])), "flops": 2 * rows * cols}
    vectors = cols * (1 + bool(case["bias"]))
    if op == "norm":
        stats = 4 * rows * ((case["kind"] == "layer") + 1) if case["save"] else 0
        return {"bytes": e * (rows * cols * (2 + 2 * bool(case["residual"])) + vectors) + stats, "flops": 8 * rows * cols}
    # dy, hidden, dhidden, statistics, weight; dx, dresidual, dw, db
    mats = 3 + bool(case["residual"]) + (p > 0)
    stats = 4 * rows * ((case["kind"] == "layer") + 1)
    return {"bytes": e * (rows * cols * mats + cols + vectors) + stats, "flops": 14 * rows * cols}


def _kept64(case, seed, offset):
    """The generator in words of 16 bits: products of 32 by 16 bits, which stay below 2^49."""
    rows, cols, p = case["rows"], case["cols"], case["p"]
    g = torch.arange(rows * cols // 8, dtype=torch.int64, device="cuda")
    words = [g % 2 ** 32, g // 2 ** 32, torch.full_like(g, offset % 2 ** 32), torch.full_like(g, offset // 2 ** 32)]
    k0, k1 = seed % 2 ** 32, seed // 2 ** 32

    def times(v, constant):
        low = v * (constant % 65536)
        high = v * (constant // 65536) + low // 65536
        return high // 65536, (high % 65536) * 65536 + low % 65536

    for _ in range(10):
        h0, l0 = times(words[0], 3528531795)
        h1, l1 = times(words[2], 3449720151)
        words = [torch.bitwise_xor(torch.bitwise_xor(h1, words[1]), k0), l1,
                 torch.bitwise_xor(torch.bitwise_xor(h0, words[3]), k1), l0]
        k0, k1 = (k0 + 2654435769) % 2 ** 32, (k1 + 3144134277) % 2 ** 32
    keep = torch.empty((g.numel(), 8), dtype=torch.bool, device="cuda")
    limit = int(round(65536 * p))
    for i, w in enumerate(words):
        keep[:, 2 * i] = w % 65536 >= limit
        keep[:, 2 * i + 1] = w // 65536 >= limit
    return keep.reshape(rows, cols), 65536.0 / (65536 - limit)


def exact(case, seed):
    """The definitions in 64 bits; the norms' and the router's gradients come from differentiating the forward formula."""
    s = prepare(case, seed)
    op = case["op"]
    v = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if op.startswith("route"):
        e, k = case["experts"], case["k"]
        z = v["logits"].requires_grad_(op == "route_backward")
        live = torch.isfinite(z).any(1)
        if op == "route_backward":
            idx = s["out"][0].long()
            live = idx[:, 0] >= 0
        else:
            live = live if s["valid"] is None else live & s["valid"]
            ranked = z + 0.0
            idx = torch.full((case["rows"], k), -1, dtype=torch.int64, device="cuda")
            for j in range(k):  # the first of the largest that are left
                best = ranked.max(1, keepdim=True).values
                rank = torch.arange(e, device="cuda").expand_as(ranked)
                first = torch.where(ranked == best, rank, e).min(1).values
                idx[:, j] = torch.where(live & torch.isfinite(best[:, 0]), first, -1)
                ranked = ranked.masked_fill(rank == first[:, None], -math.inf)
        prob = torch.zeros_like(z)
        prob[live] = torch.softmax(z[live], 1)
        one = torch.zeros((case["rows"], e + 1), dtype=torch.float64, device="cuda")
        one.scatter_(1, torch.where(idx < 0, e, idx), 1.0)
        hit = one[:, :e] > 0
        counts = s["out"][2].double() if op == "route_backward" else hit.sum(0).double()
        n = max(int(live.sum()), 1)
        if case["renorm"]:
            share = torch.zeros_like(z)
            share[live] = torch.softmax(z[live].masked_fill(~hit[live], -math.inf), 1)
        else:
            share = prob
        gate = torch.where(idx >= 0, torch.gather(share, 1, idx.clamp(min=0)), 0.0)
        loss = (e * (counts / (k * n)) * (prob.sum(0) / n)).sum().reshape(1)
        if op == "route":
            return {"idx": idx.int(), "gate": gate, "counts": counts.int(), "prob": prob.sum(0) / n, "loss": loss,
                    "used": live.sum().int().reshape(1)}
        total = loss.sum() * v["dloss"][0] + (gate * v["dgate"]).sum()
        return {"dlogits": torch.autograd.grad(total, z)[0]}
    keep, scale = _kept64(case, s["seed"], s["offset"]) if case["p"] else (None, 1.0)

    def dropped(t):
        return t if keep is None else (t * scale).masked_fill(~keep, 0.0)

    if op == "dropout":
        y = dropped(v["x"])
        return {"y": y if s["residual"] is None else y + v["residual"]}
    if op == "dropout_backward":
        return {"dx": dropped(v["dy"])}
    if op == "norm":
        h = dropped(v["x"])
        if s["residual"] is not None:
            h = v["residual"] + h
        mean = h.sum(1) / case["cols"] if case["kind"] == "layer" else torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        centred = h - mean[:, None]
        rstd = (torch.linalg.vector_norm(centred, dim=1) ** 2 / case["cols"] + _EPS) ** -0.5
        y = centred * (rstd[:, None] * v["weight"])
        got = {"y": y if s["bias"] is None else y + v["bias"]}
        if case["residual"]:
            got["hidden"] = h
        if case["save"]:
            got["rstd"] = rstd
            if case["kind"] == "layer":
                got["mean"] = mean
        return got
    h, w = v["hidden"].requires_grad_(), v["weight"].requires_grad_()
    centred = h if case["kind"] == "rms" else h - h.sum(1, keepdim=True) / case["cols"]
    y = centred / ((centred * centred).sum(1, keepdim=True) / case["cols"] + _EPS).sqrt() * w
    dh, dw = torch.autograd.grad(y, (h, w), v["dy"])
    if s["dhidden"] is not None:
        dh = dh + v["dhidden"]
    got = {"dx": dropped(dh), "dw": dw}
    if case["p"]:
        got["dresidual"] = dh
    if case["bias"]:
        got["db"] = v["dy"].sum(0)
    return got
