"""Refusals of the expert layers, the router's bookkeeping and clipping that need no GPU: the binding's
checks of tensors and the library's of sizes, pointers and alignment, made before any HIP call. The plain
forms' slopes against differences."""
import ctypes

import pytest
import torch

import layer_ref
import muon_newton_schulz_amd as mns
from muon_newton_schulz_amd import _abi

BF, I64 = torch.bfloat16, torch.int64
BAD_DTYPE, BAD_SHAPE, BAD_PARAM, BAD_NULL = (_abi.MNS_ERR_DTYPE, _abi.MNS_ERR_SHAPE,
                                             _abi.MNS_ERR_PARAM, _abi.MNS_ERR_NULL)


def _layer():
    rows, n, k, e = 12, 16, 24, 3
    z = lambda *s: torch.zeros(*s, dtype=BF)
    return dict(X=z(rows, k), W=z(e, n, k), dY=z(rows, n), bias=z(e, n), Yn=z(rows, n), Yk=z(rows, k),
                offsets=torch.zeros(e + 1, dtype=I64))


@pytest.mark.parametrize("change,error", [
    (lambda c: {}, ValueError),                                        # CPU tensors
    (lambda c: {"X": c["X"].half()}, TypeError),
    (lambda c: {"W": c["W"].float()}, TypeError),
    (lambda c: {"X": c["X"][:, :23]}, ValueError),
    (lambda c: {"W": c["W"].transpose(1, 2)}, ValueError),
    (lambda c: {"W": c["W"][0]}, ValueError),
    (lambda c: {"offsets": c["offsets"].int()}, ValueError),
    (lambda c: {"bias": c["bias"].float()}, ValueError),
    (lambda c: {"bias": c["bias"][0]}, ValueError),
    (lambda c: {"bias": torch.zeros(16, 3, dtype=BF).t()}, ValueError),
    (lambda c: {"activation": "tanh"}, ValueError),
    (lambda c: {"keep_z": True}, ValueError),                          # without an activation
    (lambda c: {"residual": c["X"]}, ValueError),
    (lambda c: {"residual": c["Yn"].float()}, ValueError),
    (lambda c: {"residual": c["Yn"][:1].expand(12, 16)}, ValueError),  # overlapping rows
    (lambda c: {"out": c["X"][:, :16]}, ValueError),
    (lambda c: {"out_z": c["X"][:, :16], "activation": "relu"}, ValueError),
    (lambda c: {"out": c["Yn"], "out_z": c["Yn"], "activation": "relu"}, ValueError),
    (lambda c: {"residual": c["Yn"], "out_z": c["Yn"], "activation": "relu"}, ValueError),
    (lambda c: {"residual": torch.zeros(13, 16, dtype=BF)[1:], "out": None}, ValueError),
])
def test_linear_refusals(change, error):
    c = _layer()
    args = {"X": c["X"], "W": c["W"], "offsets": c["offsets"]}
    args.update(change(c))
    with pytest.raises(error):
        mns.grouped_linear(**args)


def test_linear_shifted_output_is_refused():
    c = _layer()
    buf = torch.zeros(13, 16, dtype=BF)
    with pytest.raises(ValueError, match="itself"):
        mns.grouped_linear(c["X"], c["W"], c["offsets"], residual=buf[:12], out=buf[1:])
    with pytest.raises(ValueError, match="GPU"):                       # the residual itself may be
        mns.grouped_linear(c["X"], c["W"], c["offsets"], residual=buf[:12], out=buf[:12])


@pytest.mark.parametrize("change,error", [
    (lambda c: {}, ValueError),
    (lambda c: {"dY": c["X"]}, ValueError),
    (lambda c: {"activation": "gelu"}, ValueError),                    # without Z
    (lambda c: {"Z": c["Yk"]}, ValueError),                            # without an activation
    (lambda c: {"activation": "gelu", "Z": c["Yn"]}, ValueError),
    (lambda c: {"residual": c["Yn"]}, ValueError),
    (lambda c: {"out": c["Yk"].float()}, ValueError),
    (lambda c: {"activation": "x", "Z": c["Yk"]}, ValueError),
])
def test_input_grad_refusals(change, error):
    c = _layer()
    args = {"dY": c["dY"], "W": c["W"], "offsets": c["offsets"]}
    args.update(change(c))
    with pytest.raises(error):
        mns.grouped_input_grad(**args)


@pytest.mark.parametrize("change,error", [
    (lambda c: {}, ValueError),
    (lambda c: {"dY": c["dY"].half()}, TypeError),
    (lambda c: {"offsets": c["offsets"][:1]}, ValueError),
    (lambda c: {"activation": "silu"}, ValueError),
    (lambda c: {"Z": c["Yn"]}, ValueError),
    (lambda c: {"out_dz": c["Yn"]}, ValueError),
    (lambda c: {"out": torch.zeros(3, 15, dtype=BF)}, ValueError),
    (lambda c: {"out_dtype": torch.float16}, TypeError),
    (lambda c: {"out": torch.zeros(16, 3, dtype=BF).t()}, ValueError),
    (lambda c: {"out": c["dY"][:3]}, ValueError),
    (lambda c: {"activation": "silu", "Z": c["Yn"], "out_dz": c["X"][:, :16][1:]}, ValueError),
])
def test_bias_grad_refusals(change, error):
    c = _layer()
    args = {"dY": c["dY"], "offsets": c["offsets"]}
    args.update(change(c))
    with pytest.raises(error):
        mns.grouped_bias_grad(**args)


def test_router_refusals():
    ids, counts = torch.zeros(6, 2, dtype=I64), torch.zeros(4, dtype=I64)
    logits = torch.zeros(6, 4)
    for bad in (ids.int(), ids.t(), ids):                             # the last: on the CPU
        with pytest.raises(ValueError):
            mns.expert_order(bad, 4)
    for args in ((logits.half(), ids, counts), (logits, ids[:5], counts), (logits, ids, counts[:3]),
                 (logits, ids, counts.int()), (logits, ids.int(), counts), (logits[0], ids, counts),
                 (logits, ids[:, 0], counts), (logits, ids, counts)):
        with pytest.raises((ValueError, TypeError)):
            mns.balance_loss(*args)
    with pytest.raises(ValueError):
        mns.balance_loss(logits, ids, counts, grad=False, out=torch.zeros(6, 4))
    with pytest.raises(ValueError):
        mns.balance_loss(logits, ids, counts, out=torch.zeros(6, 4, dtype=BF))


def test_clip_refusals():
    g = torch.zeros(5, 4)
    for bad in ([], [g.half()], [g.t()], [g]):
        with pytest.raises((ValueError, TypeError)):
            mns.grad_norm(bad)
        with pytest.raises((ValueError, TypeError)):
            mns.clip_grad_norm(bad, 1.0)
    for out in ([], [torch.zeros(4, 5)], [g.to(BF)], [torch.zeros(4, 5).t()], [g, g]):
        with pytest.raises(ValueError):
            mns.clip_grad_norm([g], 1.0, out=out)


def _linear(lib, **kw):
    a = dict(X=0x100000, ldx=24, W=0x200000, b=0x300000, act=3, R=0x400000, ldr=16, Z=0x500000, ldz=16,
             Y=0x600000, ldy=16, dtype=1, off=0x700000, groups=3, rows=12, n=16, k=24, fill=0)
    a.update(kw)
    return lib.grouped_linear(a["X"], a["ldx"], a["W"], a["b"], a["act"], a["R"], a["ldr"], a["Z"],
                              a["ldz"], a["Y"], a["ldy"], a["dtype"], a["off"], a["groups"], a["rows"],
                              a["n"], a["k"], a["fill"], None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), BAD_DTYPE), (dict(groups=0), BAD_SHAPE), (dict(rows=-1), BAD_SHAPE),
    (dict(n=0), BAD_SHAPE), (dict(ldx=23), BAD_SHAPE), (dict(ldr=15), BAD_SHAPE),
    (dict(ldz=(1 << 21) + 1), BAD_SHAPE), (dict(ldy=15), BAD_SHAPE), (dict(act=5), BAD_PARAM),
    (dict(act=-1), BAD_PARAM), (dict(fill=2), BAD_PARAM), (dict(X=None), BAD_NULL),
    (dict(W=None), BAD_NULL), (dict(Y=None), BAD_NULL), (dict(off=None), BAD_NULL),
    (dict(b=0x300001), BAD_PARAM), (dict(R=0x400001), BAD_PARAM), (dict(Z=0x500001), BAD_PARAM),
    (dict(off=0x700004), BAD_PARAM), (dict(Y=0x500000), BAD_PARAM), (dict(Y=0x100010), BAD_PARAM),
    (dict(Y=0x400020), BAD_PARAM), (dict(Y=0x400000, ldy=17), BAD_PARAM), (dict(Z=0x400000), BAD_PARAM),
    (dict(Y=0x300000), BAD_PARAM), (dict(Z=0x200000), BAD_PARAM), (dict(Y=0x6ffff0), BAD_PARAM),
    (dict(act=0), BAD_PARAM),
    (dict(rows=0, X=None, Y=None), 0),
])
def test_library_refuses_linear(kw, status):
    assert _linear(mns.load(), **kw) == status


def _input_grad(lib, **kw):
    a = dict(dY=0x100000, lddy=16, W=0x200000, act=3, Z=0x300000, ldz=24, R=0x400000, ldr=24,
             dX=0x500000, lddx=24, dtype=1, off=0x700000, groups=3, rows=12, n=16, k=24, fill=0)
    a.update(kw)
    return lib.grouped_input_grad(a["dY"], a["lddy"], a["W"], a["act"], a["Z"], a["ldz"], a["R"],
                                  a["ldr"], a["dX"], a["lddx"], a["dtype"], a["off"], a["groups"],
                                  a["rows"], a["n"], a["k"], a["fill"], None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), BAD_DTYPE), (dict(lddy=15), BAD_SHAPE), (dict(ldz=23), BAD_SHAPE),
    (dict(ldr=23), BAD_SHAPE), (dict(lddx=23), BAD_SHAPE), (dict(act=9), BAD_PARAM),
    (dict(act=0), BAD_PARAM), (dict(Z=None), BAD_NULL), (dict(dY=None), BAD_NULL),
    (dict(dX=0x100000), BAD_PARAM), (dict(dX=0x300030), BAD_PARAM),
    (dict(dX=0x300000, lddx=25), BAD_PARAM), (dict(dX=0x400002), BAD_PARAM),
    (dict(Z=0x300001), BAD_PARAM), (dict(rows=0, dY=None, dX=None, Z=None), 0),
])
def test_library_refuses_input_grad(kw, status):
    assert _input_grad(mns.load(), **kw) == status


def _bias_grad(lib, **kw):
    a = dict(dY=0x100000, lddy=16, act=3, Z=0x300000, ldz=16, dZ=0x400000, lddz=16, dtype=1,
             off=0x700000, groups=3, rows=1200, n=16, db=0x500000, od=0, fill=0, ws=None, wsb=0)
    a.update(kw)
    return lib.grouped_bias_grad(a["dY"], a["lddy"], a["act"], a["Z"], a["ldz"], a["dZ"], a["lddz"],
                                 a["dtype"], a["off"], a["groups"], a["rows"], a["n"], a["db"], a["od"],
                                 a["fill"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), BAD_DTYPE), (dict(od=7), BAD_DTYPE), (dict(dtype=0, od=1), BAD_DTYPE),
    (dict(groups=0), BAD_SHAPE), (dict(rows=(1 << 30) + 1), BAD_SHAPE), (dict(n=65537), BAD_SHAPE),
    (dict(lddy=15), BAD_SHAPE), (dict(ldz=15), BAD_SHAPE), (dict(lddz=15), BAD_SHAPE),
    (dict(act=0), BAD_PARAM), (dict(act=5), BAD_PARAM), (dict(Z=None), BAD_NULL),
    (dict(dY=None), BAD_NULL), (dict(db=None), BAD_NULL), (dict(off=None), BAD_NULL),
    (dict(db=0x500002), BAD_PARAM), (dict(dZ=0x100020), BAD_PARAM), (dict(db=0x100000), BAD_PARAM),
    (dict(dZ=0x500000), BAD_PARAM), (dict(), _abi.MNS_ERR_WORKSPACE),
    (dict(ws=0x900010, wsb=1 << 20), _abi.MNS_ERR_WORKSPACE), (dict(ws=0x900000, wsb=100),
                                                               _abi.MNS_ERR_WORKSPACE),
])
def test_library_refuses_bias_grad(kw, status):
    assert _bias_grad(mns.load(), **kw) == status


@pytest.mark.parametrize("args,status", [
    ((0x1000, 10, 0, 0x2000, 0x3000, 0x4000), BAD_SHAPE),
    ((0x1000, 10, 2049, 0x2000, 0x9000, 0xf000), BAD_SHAPE),
    ((0x1000, -1, 4, 0x2000, 0x3000, 0x4000), BAD_SHAPE),
    ((0x1000, (1 << 30) + 1, 4, 0x2000, 0x3000, 0x4000), BAD_SHAPE),
    ((None, 10, 4, 0x2000, 0x3000, 0x4000), BAD_NULL),
    ((0x1000, 10, 4, None, 0x3000, 0x4000), BAD_NULL),
    ((0x1000, 10, 4, 0x2000, None, 0x4000), BAD_NULL),
    ((0x1004, 10, 4, 0x2000, 0x3000, 0x4000), BAD_PARAM),
    ((0x1000, 10, 4, 0x2000, 0x2018, 0x4000), BAD_PARAM),
    ((0x1000, 10, 4, 0x2000, 0x3000, 0x1000), BAD_PARAM),
    ((0x100000, 10000, 4, 0x2000, 0x3000, 0x900000), _abi.MNS_ERR_WORKSPACE),
])
def test_library_refuses_order(args, status):
    assert mns.load().expert_order(*args, None, 0, None) == status


def _balance(lib, **kw):
    a = dict(l=0x100000, ldl=8, dtype=0, ids=0x200000, top=2, c=0x300000, T=10, E=8, scale=1.0,
             loss=0x400000, g=0x500000, ldg=8)
    a.update(kw)
    return lib.balance_loss(a["l"], a["ldl"], a["dtype"], a["ids"], a["top"], a["c"], a["T"], a["E"],
                            a["scale"], a["loss"], a["g"], a["ldg"], None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), BAD_DTYPE), (dict(E=0), BAD_SHAPE), (dict(E=2049, ldl=2049, ldg=2049), BAD_SHAPE),
    (dict(T=-1), BAD_SHAPE), (dict(top=0), BAD_SHAPE), (dict(top=1 << 28), BAD_SHAPE),
    (dict(ldl=7), BAD_SHAPE), (dict(ldg=7), BAD_SHAPE), (dict(scale=float("nan")), BAD_PARAM),
    (dict(scale=float("inf")), BAD_PARAM), (dict(l=None), BAD_NULL), (dict(ids=None), BAD_NULL),
    (dict(c=None), BAD_NULL), (dict(loss=None), BAD_NULL), (dict(l=0x100002), BAD_PARAM),
    (dict(loss=0x400002), BAD_PARAM), (dict(g=0x100020), BAD_PARAM), (dict(g=0x200000), BAD_PARAM),
    (dict(loss=0x100010), BAD_PARAM), (dict(g=0x100000, ldg=9), BAD_PARAM),
    (dict(T=5000), _abi.MNS_ERR_WORKSPACE),
])
def test_library_refuses_balance(kw, status):
    assert _balance(mns.load(), **kw) == status


def _clip(tensors, max_norm=1.0, eps=0.0, norm=0x900000, count=None, ws=None, wsb=0):
    arr = (_abi.MnsTensor * max(1, len(tensors)))(*tensors)
    return mns.load().clip_grad_norm(arr, len(tensors) if count is None else count, max_norm, eps, norm,
                                     ws, wsb, None)


@pytest.mark.parametrize("tensors,kw,status", [
    ([], dict(count=0), BAD_SHAPE), ([], dict(count=65537), BAD_SHAPE),
    ([(0x1000, 0x1000, -1, 0)], {}, BAD_SHAPE), ([(0x1000, 0x1000, 1 << 41, 0)], {}, BAD_SHAPE),
    ([(0x1000, 0x1000, 4, 2)], {}, BAD_DTYPE), ([(None, 0x1000, 4, 0)], {}, BAD_NULL),
    ([(0x1000, None, 4, 0)], {}, BAD_NULL), ([(0x1000, 0x1000, 4, 0)], dict(norm=None), BAD_NULL),
    ([(0x1002, 0x1002, 4, 0)], {}, BAD_PARAM), ([(0x1000, 0x1000, 4, 0)], dict(norm=0x900002), BAD_PARAM),
    ([(0x1000, 0x1000, 4, 0)], dict(max_norm=-1.0), BAD_PARAM),
    ([(0x1000, 0x1000, 4, 0)], dict(max_norm=float("nan")), BAD_PARAM),
    ([(0x1000, 0x1000, 4, 0)], dict(eps=-1.0), BAD_PARAM),
    ([(0x1000, 0x1000, 4, 0)], dict(eps=float("inf")), BAD_PARAM),
    ([(0x1000, 0x1000, 4, 0)] * 2, {}, BAD_PARAM),                     # the same twice
    ([(0x1000, 0x1000, 8, 0), (0x101c, 0x101c, 8, 0)], {}, BAD_PARAM),
    ([(0x1000, 0x1008, 8, 0)], {}, BAD_PARAM),                         # shifted over itself
    ([(0x1000, 0x2000, 8, 0), (0x2000, 0x3000, 8, 0)], {}, BAD_PARAM),  # out over another's input
    ([(0x1000, 0x2000, 8, 0), (0x3000, 0x2010, 8, 0)], {}, BAD_PARAM),
    ([(0x1000, 0x1000, 8, 0)], dict(norm=0x1010), BAD_PARAM),
    ([(0x1000, 0x1000, 8, 0), (0x1020, 0x1020, 8, 1)], {}, _abi.MNS_ERR_WORKSPACE),   # neighbours
    ([(0x1000, 0x5000, 8, 0), (0x1000, 0x6000, 8, 0)], {}, _abi.MNS_ERR_WORKSPACE),   # read twice
])
def test_library_refuses_clip(tensors, kw, status):
    assert _clip(tensors, **kw) == status


def test_workspace_queries():
    lib, out = mns.load(), ctypes.c_size_t(1)
    ref = ctypes.byref(out)
    assert lib.mns_grouped_bias_grad_workspace_size(3, 100, 16, ref) == 0 and out.value == 0
    assert lib.mns_grouped_bias_grad_workspace_size(3, 1000, 16, ref) == 0 and out.value > 0
    assert lib.mns_grouped_bias_grad_workspace_size(0, 100, 16, ref) == BAD_SHAPE
    assert lib.mns_expert_order_workspace_size(100, 8, ref) == 0 and out.value == 0
    assert lib.mns_expert_order_workspace_size(1 << 20, 8, ref) == 0 and out.value > 0
    assert lib.mns_balance_workspace_size(10, 4096, ref) == BAD_SHAPE
    assert lib.mns_clip_workspace_size(0, ref) == BAD_SHAPE
    size = lib.mns_grouped_layer_workspace_size
    assert size(0, _abi.MNS_BF16, 3, 12, 16, 24, ref) == 0 and out.value == 0
    assert size(1, _abi.MNS_F32, 3, 12, 4096, 24, ref) == 0 and out.value > 0      # parts of a reduction
    assert size(1, _abi.MNS_F32, 3, 0, 4096, 24, ref) == 0 and out.value == 0
    assert size(2, _abi.MNS_F32, 3, 12, 16, 24, ref) == BAD_PARAM
    assert size(0, 9, 3, 12, 16, 24, ref) == _abi.MNS_ERR_DTYPE
    assert size(0, _abi.MNS_F32, 0, 12, 16, 24, ref) == BAD_SHAPE
    assert size(0, _abi.MNS_F32, 3, 12, 16, 24, None) == BAD_NULL
    for query in (lambda: lib.mns_grouped_bias_grad_workspace_size(3, 100, 16, None),
                  lambda: lib.mns_expert_order_workspace_size(100, 8, None),
                  lambda: lib.mns_balance_workspace_size(10, 8, None),
                  lambda: lib.mns_clip_workspace_size(5, None)):
        assert query() == BAD_NULL


@pytest.mark.parametrize("name", layer_ref.ACTS)
def test_plain_slopes_against_differences(name):
    z = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    diff = (layer_ref.act(name, z + 1e-6)[0] - layer_ref.act(name, z - 1e-6)[0]) / 2e-6
    # values up to 81 off by 3 roundings of 2^-53, arguments up to 9 by one at a slope of 18, twice each,
    # over a step of 2e-6: 2 (81 * 3 + 9 * 18) 2^-53 / 2e-6 = 4.5e-8; curvature: 1e-12
    assert (diff - layer_ref.act(name, z)[1])[z.abs() > 1e-5].abs().max() < 5e-8
