"""What the timed passes of the expert layers' further operators and of gradient clipping compute.

Five calls around the products of `perf/operators.py`, each in a plain form of elementary torch
operations in float32 (`own` false) and through the package (`own` true):

  linear    rows sorted by expert through a layer, Z_e = X_e W_e^T + b_e, Y = act(Z) + R
  dinput    its input's gradient with the activation before it, dX_e = (dY_e W_e) act'(Z) + R
  dbias     its bias's gradient, dZ = dY act'(Z), db_e = the sum of dZ's rows of expert e
  balance   a router's bookkeeping: the assignments counted and ordered by expert, the balance loss
            E / N^2 sum_e c_e sum_t a_t softmax(logits_t)_e and its gradient (c_e assignments of
            expert e, a_t of token t, N in all)
  clip      the global norm over many gradients, each scaled by min(1, max_norm / (norm + 1e-6))
"""
from __future__ import annotations

import math

import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_ACTS = ["relu", "relu2", "gelu", "silu"]
EPS = 1e-6


def _layer(name, op, dtype, experts, rows, n, k, route, act, tail=0, residual=False, keep=False,
           bias=True):
    """A case of an expert layer: one n x k matrix an expert, `rows` tokens routed (`route`), `tail`
    more rows behind the last expert's. keep: the forward also returns Z."""
    return {"name": name, "op": op, "dtype": dtype, "experts": experts, "rows": rows, "n": n,
            "k": k, "route": route, "act": act, "tail": tail, "residual": residual, "keep": keep,
            "bias": bias}


def _balance(name, dtype, tokens, experts, top, pad, skew):
    return {"name": name, "op": "balance", "dtype": dtype, "tokens": tokens, "experts": experts,
            "top": top, "pad": pad, "skew": skew}


def _clip(name, shapes, dtypes, max_norm, scale):
    """`shapes`: sizes joined by "x", with an optional "count*" before them, comma separated;
    `dtypes`: one for all, or "mixed" (vectors float32, matrices bfloat16)."""
    return {"name": name, "op": "clip", "shapes": shapes, "dtypes": dtypes, "max_norm": max_norm,
            "scale": scale}


def listed():
    return [
        # one decoded batch of 16 tokens over 32 experts of 8192 x 1024: the weights' bytes count
        _layer("linear_decode", "linear", "bf16", 32, 16, 8192, 1024, "spread", "silu"),
        # the first product of a training batch's experts, unevenly routed; Z is kept for the backward
        _layer("linear_train", "linear", "bf16", 32, 16384, 8192, 1024, "skewed", "gelu", keep=True),
        # odd everything, float32, experts without rows, rows behind the last expert
        _layer("linear_odd_f32", "linear", "f32", 9, 613, 777, 331, "gaps", "relu2", tail=37,
               residual=True, keep=True),
        # back through the second product (1024 x 8192 an expert) and the activation before it
        _layer("dinput_train", "dinput", "bf16", 32, 16384, 1024, 8192, "skewed", "gelu"),
        # odd sizes in bfloat16, a residual's gradient added: no row starts on a 16-byte boundary
        _layer("dinput_odd", "dinput", "bf16", 5, 1021, 513, 1277, "gaps", "silu", tail=3,
               residual=True),
        # the bias of a training batch's first product, when no product follows its activation
        _layer("dbias_train", "dbias", "bf16", 32, 16384, 8192, 1024, "skewed", "gelu"),
        # a small batch's bias without an activation: launches count
        _layer("dbias_small", "dbias", "bf16", 16, 384, 2048, 2048, "uniform", "none"),
        # a few decoded tokens: launches count
        _balance("balance_small", "f32", 61, 32, 2, 3, 1.0),
        # a training batch of bfloat16 logits, a few padded tokens
        _balance("balance_train", "bf16", 16384, 32, 2, 100, 1.0),
        # many experts, a long batch
        _balance("balance_large", "f32", 65536, 256, 8, 1000, 0.5),
        # a handful of small float32 gradients, odd sizes among them: launches count
        _clip("clip_small", "256x1024,1024,3*333x17,257,1", "f32", 1.0, 0.02),
        # a model's matrices and vectors: 1.5 GB of gradients
        _clip("clip_large", "8*4096x4096,2*4096x16384,2*5120x13824,32x1024x8192,4*2048x8192,40*4096,"
              "1000x777", "mixed", 1.0, 0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "dinput", "dbias", "balance", "clip"])
    if op == "balance":
        experts, tokens = _log(rng, 2, 512), _log(rng, 1, 65536)
        tokens = max(1, min(tokens, 65536 * 256 // experts))
        return {"op": op, "dtype": rng.choice(["bf16", "f32"]), "tokens": tokens,
                "experts": experts, "top": rng.randint(1, min(8, experts)),
                "pad": rng.choice([0, rng.randint(0, tokens)]), "skew": rng.choice([0.0, 0.5, 2.0])}
    if op == "clip":
        shapes, total = [], 0
        for _ in range(_log(rng, 1, 60)):
            r, c = _log(rng, 1, 5120), _log(rng, 1, 16384)
            if total + r * c > 700_000_000:
                r, c = 1, min(c, 4096)
            total += r * c
            shapes.append(f"{r}x{c}" if rng.random() < 0.7 else f"{c}")
        return {"op": op, "shapes": ",".join(shapes), "dtypes": rng.choice(["f32", "bf16", "mixed"]),
                "max_norm": rng.choice([1.0, 1.0, 1e6]), "scale": rng.choice([1e-4, 1e-2, 1.0])}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n, k = _log(rng, 48, 8192), _log(rng, 48, 8192)
    if rng.random() < 0.7:          # most models' widths are multiples of 64
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    experts = _log(rng, 1, 64)
    rows = _log(rng, 1, 16384)
    while experts > 1 and experts * n * k > 32 * 8192 * 1024:
        experts = (experts + 1) // 2
    cap = 2.0 * 16384 * 8192 * 1024 / (1 if dtype == "bf16" else 16)
    rows = max(1, min(rows, int(cap / (2.0 * n * k))))
    act = rng.choice(_ACTS + ["none"])
    return {"op": op, "dtype": dtype, "experts": experts, "rows": rows, "n": n, "k": k,
            "route": rng.choice(["uniform", "skewed", "gaps"]), "act": act,
            "tail": rng.choice([0, 0, rng.randint(1, 100)]),
            "residual": op != "dbias" and rng.random() < 0.5,
            "keep": op == "linear" and act != "none" and rng.random() < 0.5,
            "bias": rng.random() < 0.8}


def _sizes(case, gen):
    """Rows of each expert (host), adding up to case['rows']."""
    e, r, route = case["experts"], case["rows"], case["route"]
    if route == "spread":            # each token to an expert of its own while they last
        s = torch.full((e,), r // e, dtype=torch.int64)
        s[torch.randperm(e, generator=gen)[:r % e]] += 1
        return s
    p = torch.ones(e)
    if route == "skewed":            # a few experts take most of the rows
        p = 1.0 / (1.0 + torch.randperm(e, generator=gen).float()) ** 0.7
    elif route == "gaps":            # a third of the experts get none
        p[torch.randperm(e, generator=gen)[:e // 3]] = 0.0
    pick = torch.multinomial(p, r, replacement=True, generator=gen)
    return torch.bincount(pick, minlength=e)


def _randn(shape, dtype, gen, scale=1.0):
    """Normal values of `dtype` on the GPU, in pieces so that no large float32 copy is made."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), device="cuda", generator=gen) * scale)
    return out


def _tensors(case):
    """(shape, dtype name) of each gradient of a clip case."""
    out = []
    for item in case["shapes"].split(","):
        count, _, size = item.rpartition("*")
        shape = tuple(int(s) for s in size.split("x"))
        d = case["dtypes"]
        if d == "mixed":
            d = "f32" if len(shape) == 1 else "bf16"
        out += [(shape, d)] * int(count or 1)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "clip":
        grads = [_randn(s, _TORCH[d], gen, case["scale"]) for s, d in _tensors(case)]
        return {"case": case, "grads": grads, "out": [torch.empty_like(g) for g in grads]}
    dtype = _TORCH[case["dtype"]]
    if case["op"] == "balance":
        t, e = case["tokens"], case["experts"]
        lean = torch.randn(e, device="cuda", generator=gen) * case["skew"]
        logits = (torch.randn(t, e, device="cuda", generator=gen) + lean).to(dtype)
        ids = torch.topk(logits.float(), case["top"], dim=1).indices
        if case["pad"]:              # padded tokens go nowhere
            ids[torch.randperm(t, device="cuda", generator=gen)[:case["pad"]]] = -1
        return {"case": case, "logits": logits, "ids": ids}
    e, n, k = case["experts"], case["n"], case["k"]
    sizes = _sizes(case, torch.Generator().manual_seed(seed))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)])
    total = case["rows"] + case["tail"]
    act = None if case["act"] == "none" else case["act"]
    st = {"case": case, "act": act, "offsets": offsets.cuda(), "bias": None, "r": None, "z": None}
    if case["op"] == "dbias":
        st["dy"] = _randn((total, n), dtype, gen, 1e-2)
        st["z"] = _randn((total, n), dtype, gen) if act else None
        return st
    st["w"] = _randn((e, n, k), dtype, gen, 1.0 / math.sqrt(k if case["op"] == "linear" else n))
    if case["op"] == "linear":
        st["x"] = _randn((total, k), dtype, gen)
        st["bias"] = _randn((e, n), dtype, gen, 0.5) if case["bias"] else None
        st["r"] = _randn((total, n), dtype, gen) if case["residual"] else None
    else:
        st["dy"] = _randn((total, n), dtype, gen, 1e-2)
        st["z"] = _randn((total, k), dtype, gen) if act else None
        st["r"] = _randn((total, k), dtype, gen, 1e-2) if case["residual"] else None
    return st


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import muon_newton_schulz_amd as mns
    case = st["case"]
    op = case["op"]
    if op == "clip":
        norm = mns.clip_grad_norm(st["grads"], case["max_norm"], eps=EPS, out=st["out"])
        return [norm] + st["out"]
    if op == "balance":
        counts, offsets, order = mns.expert_order(st["ids"], case["experts"])
        loss, dlogits = mns.balance_loss(st["logits"], st["ids"], counts, scale=0.01)
        return counts, offsets, order, loss, dlogits
    if op == "linear":
        return mns.grouped_linear(st["x"], st["w"], st["offsets"], bias=st["bias"],
                                  activation=st["act"], residual=st["r"], keep_z=case["keep"])
    if op == "dinput":
        return mns.grouped_input_grad(st["dy"], st["w"], st["offsets"], activation=st["act"],
                                      Z=st["z"], residual=st["r"])
    return mns.grouped_bias_grad(st["dy"], st["offsets"], activation=st["act"], Z=st["z"])


def _act(name, z):
    if name is None:
        return z
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "relu2":
        return torch.where(z <= 0, torch.zeros_like(z), z * z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z * torch.sigmoid(z)


def _slope(name, z):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return torch.where(z <= 0, torch.zeros_like(z), 2 * z)
    if name == "gelu":
        return (0.5 * torch.erfc(z * -math.sqrt(0.5))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    s = torch.sigmoid(z)
    return s * (1 + z * torch.sigmoid(-z))


def _run_plain(st):
    op = st["case"]["op"]
    if op == "clip":
        return _plain_clip(st)
    if op == "balance":
        return _plain_balance(st)
    bounds = st["offsets"].tolist()
    act = st["act"]
    if op == "dbias":
        dy, z = st["dy"], st["z"]
        db = torch.zeros(len(bounds) - 1, dy.shape[1], dtype=dy.dtype, device=dy.device)
        dz = torch.zeros_like(dy) if act else None
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if hi > lo:
                d = dy[lo:hi].float()
                if act:
                    d = d * _slope(act, z[lo:hi].float())
                    dz[lo:hi] = d
                db[e] = d.sum(0)
        return (db, dz) if act else db
    x, w = (st["x"], st["w"]) if op == "linear" else (st["dy"], st["w"])
    out = torch.zeros(x.shape[0], w.shape[1 if op == "linear" else 2], device=x.device,
                      dtype=x.dtype)
    kept = torch.zeros_like(out) if st["case"]["keep"] else None
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi == lo:
            continue
        if op == "linear":
            y = x[lo:hi].float() @ w[e].float().t()
            if st["bias"] is not None:
                y = y + st["bias"][e].float()
            if kept is not None:
                kept[lo:hi] = y
            y = _act(act, y)
        else:
            y = x[lo:hi].float() @ w[e].float()
            if act:
                y = y * _slope(act, st["z"][lo:hi].float())
        if st["r"] is not None:
            y = y + st["r"][lo:hi].float()
        out[lo:hi] = y
    return out if kept is None else (out, kept)


def _plain_balance(st):
    e, ids = st["case"]["experts"], st["ids"]
    logits = st["logits"].float()
    valid = (ids >= 0) & (ids < e)
    key = torch.where(valid, ids, torch.full_like(ids, e)).reshape(-1)
    counts = torch.bincount(key, minlength=e + 1)[:e]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), counts.cumsum(0)])
    order = torch.argsort(key, stable=True)
    a = valid.sum(1).float()
    p = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    c = counts.float()
    n = c.sum()
    factor = torch.where(n > 0, 0.01 * e / (n * n), torch.zeros_like(n))
    s = (p * c).sum(1)
    loss = factor * (a.double() * s.double()).sum().float()
    grad = factor * a[:, None] * p * (c - s[:, None])
    return counts, offsets, order, loss, grad.to(st["logits"].dtype)


def _plain_clip(st):
    case = st["case"]
    total = sum((g.float() ** 2).sum().double() for g in st["grads"])
    norm = total.sqrt().float()
    factor = torch.clamp(case["max_norm"] / (norm + EPS), max=1.0)
    for o, g in zip(st["out"], st["grads"]):
        o.copy_(g.float() * factor)
    return [norm] + st["out"]


def _exact_act(name, z):
    """Value and slope in 64 bits."""
    if name is None:
        return z, torch.ones_like(z)
    if name in ("relu", "relu2"):
        up = torch.clamp(z, min=0)
        on = (z > 0).double()
        return (up, on) if name == "relu" else (up * up, 2 * up)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = 1 / (1 + torch.exp(-z))
    return z * s, s + z * s / (1 + torch.exp(z))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(sum(float(torch.dot(p, p)) for g in st["grads"]
                             for p in g.reshape(-1).double().split(1 << 26)))
        factor = min(1.0, case["max_norm"] / (norm + EPS))
        return [torch.tensor(norm, dtype=torch.float64, device="cuda")] + [
            g.double() * factor for g in st["grads"]]
    if op == "balance":
        return _exact_balance(case, st)
    b = st["offsets"].cpu().numpy()
    experts = range(case["experts"])
    if op == "dbias":
        d = st["dy"].double()
        d[b[-1]:] = 0
        if st["act"]:
            d *= _exact_act(st["act"], st["z"].double())[1]
        db = torch.stack([d[b[e]:b[e + 1]].sum(0) for e in experts])
        return (db, d) if st["act"] else db
    forward = op == "linear"
    x = st["x" if forward else "dy"].double()
    out = torch.zeros(x.shape[0], case["n" if forward else "k"], dtype=torch.float64,
                      device=x.device)
    for e in experts:
        if b[e + 1] > b[e]:
            we = st["w"][e].double()
            out[b[e]:b[e + 1]] = torch.mm(x[b[e]:b[e + 1]], we.t() if forward else we)
            if st["bias"] is not None:
                out[b[e]:b[e + 1]] += st["bias"][e].double()
    kept = out.clone() if case["keep"] else None
    last = b[-1]
    if forward:
        out = _exact_act(st["act"], out)[0]
    elif st["act"]:
        out *= _exact_act(st["act"], st["z"].double())[1]
    if st["r"] is not None:
        out[:last] += st["r"][:last].double()
    return out if kept is None else (out, kept)


def _exact_balance(case, st):
    e = case["experts"]
    ids, logits = st["ids"].cpu(), st["logits"].cpu().double()
    flat = ids.reshape(-1)
    members = [torch.nonzero(flat == j).reshape(-1) for j in range(e)]
    counts = torch.tensor([len(m) for m in members])
    offsets = torch.zeros(e + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(counts, 0)
    order = torch.cat(members + [torch.nonzero((flat < 0) | (flat >= e)).reshape(-1)])
    n = float(counts.sum())
    logits.requires_grad_(True)
    a = ((ids >= 0) & (ids < e)).sum(1).double()
    p = torch.softmax(logits, 1)
    mean = (a[:, None] * p).sum(0)
    loss = 0.01 * e / (n * n) * (counts.double() * mean).sum() if n else (0 * p).sum()
    (grad,) = torch.autograd.grad(loss, logits)
    return tuple(t.detach().cuda() for t in (counts, offsets, order, loss, grad))


def work(case):
    op = case["op"]
    if op == "clip":
        size = [(math.prod(s), _SIZE[d]) for s, d in _tensors(case)]
        # read for the norm, then read and written; a square and a product an element
        return {"bytes": sum(2 * n * b for n, b in size), "flops": 3 * sum(n for n, _ in size)}
    s = _SIZE[case["dtype"]]
    if op == "balance":
        t, e, top = case["tokens"], case["experts"], case["top"]
        return {"bytes": 2 * t * e * s + t * top * 16 + 16 * e, "flops": 8 * t * e}
    e, r, n, k = case["experts"], case["rows"], case["n"], case["k"]
    total = r + case["tail"]
    if op == "dbias":
        if case["act"] == "none":
            return {"bytes": r * n * s + e * n * s, "flops": r * n}
        return {"bytes": (2 * r + total) * n * s + e * n * s, "flops": 10 * r * n}
    width, inner = (n, k) if op == "linear" else (k, n)
    # experts with rows are at most the rows and, routed over gaps, two thirds of all
    used = min(r, e - e // 3 if case["route"] == "gaps" else e)
    moved = r * inner + used * n * k + total * width * (2 if case["keep"] else 1)
    moved += r * width * (int(case["residual"]) + int(op == "dinput" and case["act"] != "none"))
    moved += used * n * int(op == "linear" and case["bias"])
    return {"bytes": moved * s, "flops": 2 * r * n * k}
