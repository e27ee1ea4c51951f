"""What the timed passes of the expert products and of the Newton-Schulz gradient compute.

Four calls, each in a plain form of elementary torch operations in float32 (`own` false) and
through the package (`own` true):

  matmul   rows sorted by expert times that expert's matrix, Y_e = X_e W_e^T
  dgrad    the same rows' gradient, dX_e = dY_e W_e
  wgrad    the experts' weight gradients, G_e = beta C_e + dY_e^T X_e
  nsgrad   the gradient of O = NS_T(X / ||X||_F), the quintic Newton-Schulz map
"""
from __future__ import annotations

import math

import torch

own = False

QUINTIC = (3.4445, -4.7750, 2.0315)
COEFFS = [QUINTIC] * 5
_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def _rows(name, op, dtype, experts, rows, n, k, route, tail=0, accum=False):
    """A case of the expert products. n x k is one expert's matrix; `rows` tokens are routed to
    `experts` of them (`route`), and `tail` more rows lie behind the last expert's."""
    return {"name": name, "op": op, "dtype": dtype, "experts": experts, "rows": rows, "n": n,
            "k": k, "route": route, "tail": tail, "accum": accum}


def _ns(name, dtype, batch, rows, cols, dist):
    return {"name": name, "op": "nsgrad", "dtype": dtype, "batch": batch, "rows": rows,
            "cols": cols, "dist": dist}


def listed():
    return [
        # one decoded batch of 16 tokens over 32 experts of 8192 x 1024: the weights' bytes count
        _rows("matmul_decode", "matmul", "bf16", 32, 16, 8192, 1024, "spread"),
        # a short prompt, about 64 rows an expert: between the two bounds
        _rows("matmul_prompt", "matmul", "bf16", 8, 512, 4096, 2048, "uniform"),
        # a training batch, unevenly routed
        _rows("matmul_train", "matmul", "bf16", 32, 16384, 8192, 1024, "skewed"),
        # odd everything, float32, experts without rows, rows behind the last expert
        _rows("matmul_odd_f32", "matmul", "f32", 9, 613, 777, 331, "gaps", tail=37),
        # the training batch's input gradient
        _rows("dgrad_train", "dgrad", "bf16", 32, 16384, 8192, 1024, "skewed"),
        # odd sizes in bfloat16: no row starts on a 16-byte boundary
        _rows("dgrad_odd", "dgrad", "bf16", 5, 1021, 513, 1277, "gaps", tail=3),
        # the training batch's weight gradient
        _rows("wgrad_train", "wgrad", "bf16", 32, 16384, 8192, 1024, "skewed"),
        # a small batch added to the float32 momentum: the momentum's bytes count
        _rows("wgrad_momentum", "wgrad", "bf16", 16, 384, 2048, 2048, "uniform", accum=True),
        # one small float32 matrix: launches count
        _ns("nsgrad_single_f32", "f32", 1, 256, 1024, "normal"),
        # tall, odd, float16-side arithmetic
        _ns("nsgrad_odd_tall", "bf16", 3, 1111, 333, "student_t"),
        # a few experts of 1024 x 8192
        _ns("nsgrad_experts", "bf16", 8, 1024, 8192, "normal"),
        # one large low-rank-plus-noise matrix
        _ns("nsgrad_large", "bf16", 1, 4096, 16384, "lowrank"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "dgrad", "wgrad", "wgrad", "nsgrad"])
    if op == "nsgrad":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        top = 4096 if dtype == "bf16" else 1500
        n, m = sorted((_log(rng, 16, top), _log(rng, 16, 3 * top)))
        batch = max(1, min(_log(rng, 1, 24), int(2.0e12 / (50.0 * n * n * m)) if dtype == "bf16"
                           else int(1.0e11 / (50.0 * n * n * m))))
        rows, cols = (n, m) if rng.random() < 0.7 else (m, n)
        return {"op": op, "dtype": dtype, "batch": batch, "rows": rows, "cols": cols,
                "dist": rng.choice(["normal", "student_t", "lowrank"])}
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
    return {"op": op, "dtype": dtype, "experts": experts, "rows": rows, "n": n, "k": k,
            "route": rng.choice(["uniform", "skewed", "gaps"]),
            "tail": rng.choice([0, 0, rng.randint(1, 100)]),
            "accum": op == "wgrad" and rng.random() < 0.4}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TORCH[case["dtype"]]
    if case["op"] == "nsgrad":
        b, r, c = case["batch"], case["rows"], case["cols"]
        if case["dist"] == "lowrank":     # rank 64 plus a tenth of noise
            q = min(64, r, c)
            x = torch.randn(b, r, q, device="cuda", generator=gen) / math.sqrt(q)
            x = x @ torch.randn(b, q, c, device="cuda", generator=gen)
            x += 0.1 * torch.randn(b, r, c, device="cuda", generator=gen)
        else:
            x = torch.randn(b, r, c, device="cuda", generator=gen)
            if case["dist"] == "student_t":
                z = sum(torch.randn(b, r, c, device="cuda", generator=gen) ** 2 for _ in range(3))
                x /= torch.sqrt(z / 3.0)
        return {"case": case, "x": x.to(dtype), "do": _randn((b, r, c), dtype, gen, 1e-2)}
    e, n, k = case["experts"], case["n"], case["k"]
    cpu = torch.Generator().manual_seed(seed)
    sizes = _sizes(case, cpu)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)])
    total = case["rows"] + case["tail"]
    st = {"case": case, "offsets": offsets.cuda()}
    if case["op"] == "wgrad":
        st["dy"] = _randn((total, n), dtype, gen, 1e-2)
        st["x"] = _randn((total, k), dtype, gen)
        st["c"] = _randn((e, n, k), torch.float32, gen, 1e-2) if case["accum"] else None
    else:
        st["w"] = _randn((e, n, k), dtype, gen, 1.0 / math.sqrt(k))
        st["x"] = _randn((total, k if case["op"] == "matmul" else n), dtype, gen)
    return st


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import muon_newton_schulz_amd as mns
    op = state["case"]["op"]
    if op == "matmul":
        return mns.grouped_matmul(state["x"], state["w"], state["offsets"])
    if op == "dgrad":
        return mns.grouped_matmul(state["x"], state["w"], state["offsets"], transpose_w=True)
    if op == "wgrad":
        if state["c"] is None:
            return mns.grouped_weight_grad(state["dy"], state["x"], state["offsets"])
        return mns.grouped_weight_grad(state["dy"], state["x"], state["offsets"], C=state["c"],
                                       beta=0.95)
    return mns.ns_orthogonalize_backward(state["x"], state["do"], COEFFS)


def _run_plain(state):
    op = state["case"]["op"]
    if op == "nsgrad":
        return _plain_nsgrad(state["x"], state["do"])
    x = state["x"]
    bounds = state["offsets"].tolist()
    if op == "wgrad":
        dy, c = state["dy"], state["c"]
        out = torch.empty(len(bounds) - 1, dy.shape[1], x.shape[1], device=x.device,
                          dtype=x.dtype if c is None else torch.float32)
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            g = dy[lo:hi].float().t() @ x[lo:hi].float()
            out[e] = g if c is None else 0.95 * c[e] + g
        return out
    w = state["w"]
    out = torch.zeros(x.shape[0], w.shape[1 if op == "matmul" else 2], device=x.device,
                      dtype=x.dtype)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            we = w[e].float()
            out[lo:hi] = x[lo:hi].float() @ (we.t() if op == "matmul" else we)
    return out


def _mm(a, b):
    """Products of a batch, one matrix at a time."""
    return torch.stack([p @ q for p, q in zip(a, b)])


def _plain_nsgrad(x, do):
    """The textbook way: keep every iterate, walk back through them."""
    dtype = x.dtype
    tall = x.shape[1] > x.shape[2]
    x, g = x.float(), do.float()
    if tall:
        x, g = x.transpose(1, 2).contiguous(), g.transpose(1, 2).contiguous()
    norm = torch.sqrt((x * x).sum((1, 2), keepdim=True))
    inv = torch.where(norm > 0, 1.0 / norm, torch.zeros_like(norm))
    x0 = x * inv
    eye = torch.eye(x.shape[1], device=x.device)
    saved, y = [], x0
    for i, (a, b, c) in enumerate(COEFFS):
        s = _mm(y, y.transpose(1, 2).contiguous())
        p = a * eye + b * s + c * _mm(s, s)
        saved.append((y, s, p))
        if i < len(COEFFS) - 1:
            y = _mm(p, y)
    for (a, b, c), (y, s, p) in zip(reversed(COEFFS), reversed(saved)):
        dp = _mm(g, y.transpose(1, 2).contiguous())
        dp = dp + dp.transpose(1, 2)
        sd = _mm(s, dp)
        g = _mm(p, g) + _mm(b * dp + c * (sd + sd.transpose(1, 2)), y)
    g = (g - x0 * (x0 * g).sum((1, 2), keepdim=True)) * inv
    return (g.transpose(1, 2).contiguous() if tall else g).to(dtype)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "nsgrad":
        outs = []
        for xi, gi in zip(st["x"], st["do"]):
            v = xi.double().requires_grad_(True)
            y = v / torch.linalg.norm(v)
            if y.shape[0] > y.shape[1]:
                y = y.t()
            for a, b, c in COEFFS:
                s = y @ y.t()
                y = a * y + (b * s + c * (s @ s)) @ y
            y = y.t() if xi.shape[0] > xi.shape[1] else y
            (grad,) = torch.autograd.grad(y, v, gi.double())
            outs.append(grad)
        return torch.stack(outs)
    x, b = st["x"].double(), st["offsets"].cpu().numpy()
    if case["op"] == "wgrad":
        dy, c = st["dy"].double(), st["c"]
        out = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64,
                          device=x.device)
        for e in range(case["experts"]):
            torch.mm(dy[b[e]:b[e + 1]].t(), x[b[e]:b[e + 1]], out=out[e])
            if c is not None:
                out[e].add_(c[e].double(), alpha=0.95)
        return out
    width = case["n"] if case["op"] == "matmul" else case["k"]
    out = torch.zeros(x.shape[0], width, dtype=torch.float64, device=x.device)
    for e in range(case["experts"]):
        if b[e + 1] > b[e]:
            we = st["w"][e].double()
            out[b[e]:b[e + 1]] = torch.mm(x[b[e]:b[e + 1]], we.t() if case["op"] == "matmul" else we)
    return out


def work(case):
    s = _SIZE[case["dtype"]]
    if case["op"] == "nsgrad":
        n, m = sorted((case["rows"], case["cols"]))
        t = len(COEFFS)
        # per iteration X X^T and A^2 (symmetric: half), E X^T, A S, P E + Q X and P X (not in
        # the last one)
        flops = t * (n * n * m + n ** 3 + 2 * n * n * m + 2 * n ** 3 + 4 * n * n * m + 2 * n * n * m)
        return {"bytes": case["batch"] * 3 * n * m * s,
                "flops": case["batch"] * (flops - 2 * n * n * m)}
    e, r, n, k = case["experts"], case["rows"], case["n"], case["k"]
    flops = 2 * r * n * k
    if case["op"] == "wgrad":
        return {"bytes": r * (n + k) * s + e * n * k * (8 if case["accum"] else s), "flops": flops}
    # experts with rows are at most the rows and, routed over gaps, two thirds of all
    used = min(r, e - e // 3 if case["route"] == "gaps" else e)
    total_out = (r + case["tail"]) * (n if case["op"] == "matmul" else k)
    return {"bytes": (r * (k if case["op"] == "matmul" else n) + used * n * k + total_out) * s,
            "flops": flops}
