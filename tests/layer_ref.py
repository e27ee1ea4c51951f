"""Plain float64 forms of the expert layers, their bias gradient, the ordered assignments, the balance
loss and clipping, with the error an implementation may make: results and bounds element by element.

Activations. A value off by d before the activation is off by at most L d behind it, L the largest slope
between (relu 1; relu2 2 (|z| + d); gelu 1.13; silu 1.1). The activations themselves, A = a relative
error: float32 storage evaluates exp and erfc to a few units in the last place (2^-23 each), and erfc's
and exp's arguments are rounded, which moves erfc(-z / sqrt 2) by up to z^2 2^-23 in the tail: A = (16 + z^2)
2^-23. bfloat16 storage uses approximations: gelu = max(z, 0) - |z| Q with Q = Phi(-|z|) off by up to 2e-4 of
itself for |z| <= 5, 6e-4 up to 8 and 8e-3 beyond (and less than 1e-40 past 13.3), evaluated with 10 roundings
of a logarithm up to 132: 10 132 2^-24 = 8e-5; its slope and silu are within 2.9e-5 and 8 roundings: A = 2^-14.
The slopes are sums of two such terms, each off by A of itself; silu's 1 - s is off by up to 2^-23 of 1
besides."""
import math

import torch

from grouped_ref import HALF_STEP, ULP, stored

ACTS = ["relu", "relu2", "gelu", "silu"]


def act(name, z):
    """(value, slope, Lipschitz constant near z) in float64."""
    one = torch.ones_like(z)
    if name is None:
        return z, one, one
    if name == "relu":
        return z.clamp(min=0), (z > 0).double(), one
    if name == "relu2":
        p = z.clamp(min=0)
        return p * p, 2 * p, 2 * p + 1e-3
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 1.13 * one
    s = torch.sigmoid(z)
    return z * s, s + z * s * torch.sigmoid(-z), 1.1 * one


def act_error(name, z, dtype):
    """Error of the activation's evaluation at z, and of its slope's."""
    if name in (None, "relu", "relu2"):
        return act(name, z)[0].abs() * 2 * ULP, act(name, z)[1].abs() * 2 * ULP
    rel = (16 + z * z) * ULP if dtype == torch.float32 else 2.0 ** -14
    # Far out in the tail e^(-z^2 / 2), e^-|z| or erfc lies below the normal numbers, 2^-126, and may be
    # flushed to zero: Phi, phi and s are off by as much, the value z Phi or z s by |z| of it, the slopes
    # Phi + z phi and s (1 + z (1 - s)) by 1 + |z| of it.
    flush = 2.0 ** -126 * (1 + z.abs())
    value = act(name, z)[0].abs() * rel + flush
    if name == "gelu" and dtype != torch.float32:
        far = z.abs()
        q = torch.where(far <= 5, 2.8e-4, torch.where(far <= 8, 6.8e-4, 8.1e-3))
        value = far * 0.5 * torch.erfc(far / math.sqrt(2)) * q + ULP * z.abs() + flush
    if name == "gelu":
        parts = 0.5 * torch.erfc(-z / math.sqrt(2)) + z.abs() * torch.exp(-z * z / 2)
        return value, parts * rel + flush
    s = torch.sigmoid(z)
    return value, s * (1 + z.abs() * torch.sigmoid(-z)) * rel + s * z.abs() * ULP + flush


def linear(X, W, bounds, bias, name, R, start, start_z):
    """(Y, its bound, Z, its bound): rows of no expert keep `start` and `start_z`."""
    Xd, Wd = X.cpu().double(), W.cpu().double()
    Y, Z = start.cpu().double().clone(), start_z.cpu().double().clone()
    eY, eZ = torch.zeros_like(Y), torch.zeros_like(Z)
    r = Xd.shape[1]
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi <= lo:
            continue
        z = Xd[lo:hi] @ Wd[e].t()
        mag = Xd[lo:hi].abs() @ Wd[e].t().abs()
        if bias is not None:
            z = z + bias[e].cpu().double()
            mag = mag + bias[e].cpu().double().abs()
        d = (r + 3) * ULP * mag
        v, _, lip = act(name, z)
        ev, _ = act_error(name, z, X.dtype)
        extra = 2 * d if name == "relu2" else 0.0
        ev = ev + (lip + extra) * d
        if R is not None:
            res = R[lo:hi].cpu().double()
            v = v + res
            ev = ev + ULP * (v.abs() + res.abs())
        Y[lo:hi], Z[lo:hi] = v, z
        eY[lo:hi], eZ[lo:hi] = stored(v, ev, X.dtype), stored(z, d, X.dtype)
    return Y, eY, Z, eZ


def input_grad(dY, W, bounds, name, Zin, R, start):
    Yd, Wd = dY.cpu().double(), W.cpu().double()
    out = start.cpu().double().clone()
    err = torch.zeros_like(out)
    r = Yd.shape[1]
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi <= lo:
            continue
        g = Yd[lo:hi] @ Wd[e]
        d = (r + 2) * ULP * (Yd[lo:hi].abs() @ Wd[e].abs())
        if name is not None:
            z = Zin[lo:hi].cpu().double()
            s, es = act(name, z)[1], act_error(name, z, dY.dtype)[1]
            d = d * (s.abs() + es) + g.abs() * es + ULP * (g * s).abs()
            g = g * s
        if R is not None:
            res = R[lo:hi].cpu().double()
            g = g + res
            d = d + ULP * (g.abs() + res.abs())
        out[lo:hi], err[lo:hi] = g, stored(g, d, dY.dtype)
    return out, err


def bias_grad(dY, bounds, name, Zin, out_dtype, start):
    """(db, its bound, dZ, its bound): dZ's rows of no expert keep `start`."""
    Yd = dY.cpu().double()
    dZ = start.cpu().double().clone()
    eZ = torch.zeros_like(dZ)
    db = torch.zeros(len(bounds) - 1, Yd.shape[1], dtype=torch.float64)
    eb = torch.zeros_like(db)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        g = Yd[lo:hi]
        d = torch.zeros_like(g)
        if name is not None:
            z = Zin[lo:hi].cpu().double()
            s, es = act(name, z)[1], act_error(name, z, dY.dtype)[1]
            d = g.abs() * es + ULP * (g * s).abs()
            g = g * s
        dZ[lo:hi], eZ[lo:hi] = g, stored(g, d, dY.dtype)
        db[e] = g.sum(0)
        eb[e] = d.sum(0) + (hi - lo) * ULP * g.abs().sum(0)
        eb[e] = stored(db[e], eb[e], out_dtype)
    return db, eb, dZ, eZ


def order(ids, experts):
    """(counts, offsets, order), whole numbers."""
    flat = ids.reshape(-1).cpu().tolist()
    members = [[] for _ in range(experts + 1)]
    for i, e in enumerate(flat):
        members[e if 0 <= e < experts else experts].append(i)
    counts = [len(m) for m in members[:experts]]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    flat_order = [i for m in members for i in m]
    return (torch.tensor(counts, dtype=torch.int64), torch.tensor(offsets, dtype=torch.int64),
            torch.tensor(flat_order, dtype=torch.int64))


def balance(logits, ids, counts, scale):
    """(loss, bound, dlogits, bound). Errors: the exponentials by 2 units and the rounding of their
    argument (|x - max| 2^-24 of them), a sum of E terms by E units, s and the quotients by 3 more; c - s loses
    what cancels, so its error is that of c plus s's."""
    T, E = logits.shape
    x, c = logits.cpu().double(), counts.cpu().double()
    a = ((ids >= 0) & (ids < E)).sum(1).cpu().double()
    n = c.sum().item()
    factor = scale * E / (n * n) if n > 0 else 0.0
    loss, el = 0.0, 0.0
    grad, eg = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        if a[t] == 0 or bool((x[t] == -math.inf).all()):
            continue
        m = x[t].max()
        p = torch.exp(x[t] - m)
        p = p / p.sum()
        s = (p * c).sum()
        far = (m - x[t]).clamp(max=120.0)
        rel = (E + 8 + 2 * float((far * p).sum()) + far) * ULP
        es = float(((rel + (E + 4) * ULP) * p * c).sum())
        loss += a[t] * s
        el += a[t] * es
        grad[t] = factor * a[t] * p * (c - s)
        eg[t] = abs(factor) * a[t] * p * (es + ULP * (c + s) + (2 * rel + 6 * ULP) * (c - s).abs())
    loss, el = factor * loss, abs(factor) * float(el)
    el = el + 2 * ULP * abs(float(loss)) + 1e-38
    return torch.tensor(float(loss), dtype=torch.float64), torch.tensor(el), grad, stored(
        grad, eg, logits.dtype)


def clip(grads, max_norm, eps):
    """(norm, factor) in float64."""
    total = sum(float((g.cpu().double() ** 2).sum()) for g in grads)
    norm = math.sqrt(total)
    return norm, (1.0 if norm + eps == 0 else min(1.0, max_norm / (norm + eps)))


def clipped(g, factor):
    """(result, bound): the factor's rounding, the product's and the dtype's."""
    v = g.cpu().double() * factor
    return v, stored(v, v.abs() * ULP, g.dtype)
