"""A routed decoder block's training step through the calls as they are used together: norm with the
residual stream and dropout, gated pair, projection, norm, dropout, router product, choice and balance loss,
and every gradient back; against the same step in fp64 with torch's own differentiation."""
import pytest
import torch

import layer_helpers as H
from linear_helpers import growth
from oracle import layer as OL
from weight_merge_amd import api as A

DEV = "cuda"
D, F, E, K = 256, 512, 16, 4
P, EPS, BALANCE = 0.1, 1e-5, 0.1
SEED = 1234
STAGES = 14  # calls between an input and the furthest gradient


def tensors(rows, dtype, seed):
    def n(i, shape, std):
        return H.normal(seed + i, shape, std, dtype)

    return dict(x=n(0, (rows, D), 1.0), res=n(1, (rows, D), 1.0), w1=n(2, (D,), 0.1) + 1, b1=n(3, (D,), 0.1),
                wg=n(4, (F, D), D ** -0.5), wu=n(5, (F, D), D ** -0.5), wd=n(6, (D, F), F ** -0.5), w2=n(7, (D,), 0.1) + 1,
                router=n(8, (E, D), D ** -0.5))


def step(t, valid, c1, c2, state):
    """(outputs, gradients) from the library's calls."""
    rows = t["x"].shape[0]
    like = torch.empty_like
    dt = t["x"].dtype
    hidden, hidden2 = like(t["x"]), like(t["x"])
    stats = (torch.empty(rows, device=DEV), torch.empty(rows, device=DEV))
    stats2 = (None, torch.empty(rows, device=DEV))
    pre = (torch.empty((rows, F), dtype=dt, device=DEV), torch.empty((rows, F), dtype=dt, device=DEV))
    y = A.ada_norm(t["x"], t["w1"], bias=t["b1"], residual=t["res"], eps=EPS, p=P, seed=state, offset=0, hidden=hidden,
                   stats=stats)
    a = A.ada_glu(y, t["wg"], t["wu"], pre=pre)
    z = A.ada_linear(a, t["wd"])
    y2 = A.ada_norm(z, t["w2"], residual=hidden, kind="rms", eps=EPS, p=P, seed=state, offset=1, hidden=hidden2,
                    stats=stats2)
    y3 = A.ada_dropout(y2, P, state, 2)
    logits = A.ada_linear(y3, t["router"])
    out = A.ada_route(logits, K, valid=valid)

    dlogits = A.ada_route_backward(logits, out, dgate=c2, dloss=torch.full((1,), BALANCE, device=DEV))
    dy3, drouter, _ = A.ada_linear_backward(dlogits, y3, t["router"])
    dy2 = A.ada_dropout_backward(dy3, P, state, 2)
    dz, dhidden, dw2, _ = A.ada_norm_backward(dy2, hidden2, stats2, t["w2"], dhidden=c1, kind="rms", p=P, seed=state,
                                              offset=1, want_dresidual=True)
    da, dwd, _ = A.ada_linear_backward(dz, a, t["wd"])
    dy, dwg, dwu, _, _ = A.ada_glu_backward(da, y, t["wg"], t["wu"], *pre)
    dx, dres, dw1, db1 = A.ada_norm_backward(dy, hidden, stats, t["w1"], dhidden=dhidden, p=P, seed=state, offset=0,
                                             want_dresidual=True, want_dbias=True)
    return dict(hidden=hidden2, logits=logits, gate=out.gate, loss=out.loss, prob=out.prob), dict(
        x=dx, res=dres, w1=dw1, b1=db1, wg=dwg, wu=dwu, wd=dwd, w2=dw2, router=drouter), out


def reference(t, valid, c1, c2, idx):
    """The same in fp64 on the host, given the experts that were picked."""
    v = {k: x.double().requires_grad_() for k, x in t.items()}
    rows = v["x"].shape[0]

    def drop(x, offset):
        kept, scale = OL.dropout_mask(rows, x.shape[1], P, SEED, offset)
        return torch.where(torch.from_numpy(kept), x * scale, 0.0)

    def norm(h, w, centred):
        c = h - h.mean(1, keepdim=True) if centred else h
        return c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * w

    h = v["res"] + drop(v["x"], 0)
    y = norm(h, v["w1"], True) + v["b1"]
    a = torch.nn.functional.silu(y @ v["wg"].t()) * (y @ v["wu"].t())
    h2 = h + drop(a @ v["wd"].t(), 1)
    logits = drop(norm(h2, v["w2"], False), 2) @ v["router"].t()
    p = torch.softmax(logits, 1)
    picked = torch.gather(p, 1, idx.clamp(min=0))
    gate = torch.where(valid[:, None], picked / picked.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(idx[valid].flatten(), minlength=E).double()
    n = valid.sum()
    prob = p[valid].mean(0)
    loss = E * (counts / (K * n) * prob).sum()
    total = (h2 * c1.double()).sum() + (gate * c2.double()).sum() + BALANCE * loss
    grads = torch.autograd.grad(total, list(v.values()))
    return dict(hidden=h2, logits=logits, gate=gate, loss=loss[None], prob=prob), dict(zip(v, grads)), logits


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("rows", (1, 37, 1100))
def test_training_step_of_a_routed_block(rows, dtype):
    """Each call is off by no more than the usual bound of its deepest sum (fp32, F products) or by one
    rounding of its results, doubled for the operand that the products' backward rounds (bf16); a step
    of STAGES calls by STAGES times that, in the 2-norm of each result."""
    t = tensors(rows, dtype, rows)
    valid = torch.arange(rows) % 5 != 4
    c1, c2 = H.normal(90, (rows, D), 0.1, dtype), H.normal(91, (rows, K), 1.0, "fp32")
    state = torch.tensor([SEED, 0], dtype=torch.int64, device=DEV)
    dev = {k: x.to(DEV) for k, x in t.items()}
    got, grads, out = step(dev, valid.to(DEV), c1.to(DEV), c2.to(DEV), state)
    idx = out.idx.cpu().long()
    assert (idx[~valid] == -1).all() and int(out.used) == int(valid.sum())
    ref, rgrads, logits = reference(t, valid, c1, c2, idx)
    if dtype == "fp32":  # away from ties the fp64 logits pick the same
        top = torch.sort(logits, 1, descending=True)
        clear = valid & ((top.values[:, :K] - top.values[:, 1:K + 1]).min(1).values > 1e-3)
        assert torch.equal(idx[clear], top.indices[clear][:, :K])
    tol = STAGES * (growth(F) if dtype == "fp32" else 2 * H.half_step(dtype))
    for what, pairs in (("", (got, ref)), ("gradient of ", (grads, rgrads))):
        for name, g in pairs[0].items():
            r = pairs[1][name].detach()
            off = (g.cpu().double() - r).norm() / r.norm()
            assert off <= tol, f"{what}{name}: off by {off:.2e}, allowed {tol:.2e}"
