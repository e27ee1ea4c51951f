"""A training step of a layer of experts through every call it takes: the assignments in the experts'
order, two products with bias, activation and residual, the balance loss, all gradients, clipping and the
optimizer step; against float64 automatic differentiation, eager and as a replayed graph."""
import math

import pytest
import torch

import layer_ref
import muon_newton_schulz_amd as mns
import oracle
from grouped_ref import ULP
from helpers import check_weight, to_f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
C5 = [(3.4445, -4.7750, 2.0315)] * 5
TOKENS, H, F, E, TOP = 300, 40, 56, 5, 2


def _state(dtype, seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=g) * scale).to(dt).cuda()

    st = dict(X=r(TOKENS, H), W1=r(E, F, H, scale=0.2), b1=r(E, F, scale=0.3), W2=r(E, H, F, scale=0.2),
              b2=r(E, H, scale=0.3), logits=r(TOKENS, E, dt=F32), C=r(TOKENS, H),
              mix=torch.rand(TOKENS, TOP, generator=g).to(dtype).cuda(),
              M1=torch.zeros(E, F, H, device="cuda"), M2=torch.zeros(E, H, F, device="cuda"))
    st["ids"] = torch.topk(st["logits"], TOP).indices
    st["ids"][5:12] = -1                              # padded tokens
    st["ids"][20, 1] = E                              # one dropped assignment
    return st


def _step(s, max_norm=0.5):
    """Everything a program calls; no value is read by the host."""
    counts, offsets, order = mns.expert_order(s["ids"], E)
    token = order // TOP
    Xs, share = s["X"][token], s["mix"].reshape(-1)[order][:, None]
    Hs, Z = mns.grouped_linear(Xs, s["W1"], offsets, bias=s["b1"], activation="gelu", keep_z=True)
    Y = mns.grouped_linear(Hs, s["W2"], offsets, bias=s["b2"], residual=Xs)
    out = torch.zeros_like(s["X"], dtype=F32).index_add_(0, token, (Y * share).float())
    loss, dlogits = mns.balance_loss(s["logits"], s["ids"], counts, scale=0.1)
    dY = s["C"][token] * share
    dZ = mns.grouped_input_grad(dY, s["W2"], offsets, activation="gelu", Z=Z)
    grads = [mns.grouped_weight_grad(dZ, Xs, offsets), mns.grouped_bias_grad(dZ, offsets),
             mns.grouped_weight_grad(dY, Hs, offsets), mns.grouped_bias_grad(dY, offsets), dlogits]
    dX = mns.grouped_input_grad(dZ, s["W1"], offsets, residual=dY)
    raw = [g.clone() for g in grads]
    norm = mns.clip_grad_norm(grads, max_norm)
    mns.muon_step(list(s["W1"]) + list(s["W2"]), list(s["M1"]) + list(s["M2"]),
                  list(grads[0]) + list(grads[2]), mu=0.9, lr=0.02, coeffs=C5)
    return dict(offsets=offsets, order=order, out=out, loss=loss, dX=dX, raw=raw, grads=grads, norm=norm)


def _reference(s, got):
    """Gradients of <C, sum of mix Y> + balance loss by float64 automatic differentiation, for sorted rows,
    and their elementwise bounds: every product and activation is off by its reduction's length times
    2^-23 of the same chain of magnitudes (|gelu(z)| <= |z|, |gelu'| <= 1.13, |gelu''| <= 0.8)."""
    b = got["offsets"].tolist()
    order = got["order"].cpu()
    d = {k: v.cpu().double() for k, v in s.items() if k not in ("ids",)}
    names = ("W1", "b1", "W2", "b2", "logits")
    for k in names:
        d[k].requires_grad_(True)
    token = order // TOP
    share = d["mix"].reshape(-1)[order][:, None]
    Xs = d["X"][token].clone().requires_grad_(True)
    total = torch.zeros((), dtype=torch.float64)
    out = torch.zeros(TOKENS, H, dtype=torch.float64)
    bound = {k: torch.zeros_like(d[k]) for k in ("W1", "b1", "W2", "b2")}
    bound["dX"] = torch.zeros_like(Xs)
    for e, (lo, hi) in enumerate(zip(b, b[1:])):
        z = Xs[lo:hi] @ d["W1"][e].t() + d["b1"][e]
        h = 0.5 * z * torch.erfc(-z / math.sqrt(2))
        y = h @ d["W2"][e].t() + d["b2"][e] + Xs[lo:hi]
        out.index_add_(0, token[lo:hi], (y * share[lo:hi]).detach())
        total = total + (d["C"][token[lo:hi]] * share[lo:hi] * y).sum()
        with torch.no_grad():
            n = hi - lo
            x, dy = Xs[lo:hi].abs(), (d["C"][token[lo:hi]] * share[lo:hi]).abs()
            zm = x @ d["W1"][e].abs().t() + d["b1"][e].abs()
            ez = (H + 4) * ULP * zm
            eh = 1.13 * ez + 20 * ULP * zm
            dh = dy @ d["W2"][e].abs()
            edz = 1.13 * (H + 3) * ULP * dh + dh * (0.8 * ez + 20 * ULP * (1 + zm))
            edy = 2 * ULP * dy
            edz = edz + 1.13 * (edy @ d["W2"][e].abs())
            dz = 1.13 * dh
            bound["W1"][e] = edz.t() @ x + (n + 2) * ULP * (dz.t() @ x)
            bound["b1"][e] = edz.sum(0) + (n + 2) * ULP * dz.sum(0)
            bound["W2"][e] = dy.t() @ eh + edy.t() @ zm + (n + 2) * ULP * (dy.t() @ zm)
            bound["b2"][e] = edy.sum(0) + (n + 2) * ULP * dy.sum(0)
            bound["dX"][lo:hi] = (edz @ d["W1"][e].abs() + (F + 3) * ULP * (dz @ d["W1"][e].abs()) + edy
                                  + 2 * ULP * dy)
    ids = s["ids"].cpu()
    c = torch.tensor([float((ids == e).sum()) for e in range(E)], dtype=torch.float64)
    a = ((ids >= 0) & (ids < E)).sum(1).double()
    balance = 0.1 * E / c.sum() ** 2 * (a * (torch.softmax(d["logits"], 1) * c).sum(1)).sum()
    (total + balance).backward()
    return out, float(balance), {k: d[k].grad for k in names} | {"dX": Xs.grad}, bound


def test_step_against_automatic_differentiation():
    s = _state(F32)
    before = {k: to_f64(s[k]) for k in ("W1", "W2")}
    kept = {k: s[k].clone() for k in s}
    got = _step(s)
    out, balance, want, bound = _reference(kept, got)
    last = got["offsets"][-1].item()
    assert last == TOP * (TOKENS - 7) - 1
    assert (got["out"].cpu().double() - out).abs().max() < 1e-4          # (its parts are checked below)
    assert abs(got["loss"].item() - balance) <= 40 * ULP * abs(balance)
    for name, g in zip(("W1", "b1", "W2", "b2"), got["raw"]):
        over = ((g.cpu().double() - want[name]).abs() - bound[name]).max().item()
        assert over <= 0, (name, over)
    over = ((got["dX"].cpu().double() - want["dX"]).abs() - bound["dX"])[:last].max().item()
    assert over <= 0 and (got["dX"][last:] == 0).all()
    counts, _, _ = layer_ref.order(kept["ids"], E)
    _, _, wl, el = layer_ref.balance(kept["logits"], kept["ids"], counts, 0.1)
    assert ((got["raw"][4].cpu().double() - wl).abs() <= el).all()
    norm, factor = layer_ref.clip(got["raw"], 0.5, 1e-6)
    assert abs(got["norm"].item() - norm) <= 2.0 ** -23 * norm and factor < 1
    for g, r in zip(got["grads"], got["raw"]):
        w, err = layer_ref.clipped(r, factor)
        assert ((g.cpu().double() - w).abs() <= err).all()
    for name, i in (("W1", 0), ("W2", 2)):
        for e in range(E):
            step = oracle.muon_step(before[name][e], 0 * before[name][e], to_f64(got["grads"][i][e]),
                                    mu=0.9, lr=0.02, coeffs=C5)
            check_weight(to_f64(s[name][e]), before[name][e], step["W_exact"] - before[name][e], "f32",
                         (name, e))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_captured_step_follows_its_inputs(dtype):
    """One graph of the whole step, replayed on new tokens and routings with eager work in between: every
    replay equals the eager step, bit for bit."""
    s = _state(dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step({k: v.clone() for k, v in s.items()})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(s)
    for seed in (1, 2, 3):
        new = _state(dtype, seed)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = _step(new)
        for k in ("offsets", "order", "loss", "dX", "norm"):
            assert torch.equal(got[k], want[k]), (seed, k)
        for a, b in zip(got["raw"] + got["grads"] + [s["W1"], s["W2"], s["M1"]],
                        want["raw"] + want["grads"] + [new["W1"], new["W2"], new["M1"]]):
            assert torch.equal(a, b), seed
