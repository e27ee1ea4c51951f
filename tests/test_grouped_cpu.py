"""Refusals of the products grouped by expert that need no GPU: the binding's checks of tensors
and the library's checks of sizes, pointers and alignment, made before any HIP call."""
import ctypes

import pytest
import torch

import muon_newton_schulz_amd as mns
from muon_newton_schulz_amd import _abi

BF = torch.bfloat16


def _case(rows=12, n=16, k=24, e=3, dt=BF):
    return (torch.zeros(rows, k, dtype=dt), torch.zeros(e, n, k, dtype=dt),
            torch.zeros(rows, n, dtype=dt), torch.zeros(e + 1, dtype=torch.int64))


def test_cpu_tensors_are_refused():
    X, W, dY, off = _case()
    with pytest.raises(ValueError, match="GPU"):
        mns.grouped_matmul(X, W, off)
    with pytest.raises(ValueError, match="GPU"):
        mns.grouped_weight_grad(dY, X, off)


@pytest.mark.parametrize("change,error", [
    (lambda c: {"X": c["X"].half()}, TypeError),
    (lambda c: {"W": c["W"].float()}, TypeError),
    (lambda c: {"X": c["X"][:, :23]}, ValueError),                    # another width
    (lambda c: {"X": c["X"].reshape(3, 4, 24)}, ValueError),
    (lambda c: {"X": torch.zeros(24, 12, dtype=BF).t()}, ValueError),  # rows not contiguous
    (lambda c: {"X": c["X"][:1].expand(12, 24)}, ValueError),          # overlapping rows
    (lambda c: {"W": c["W"].transpose(1, 2)}, ValueError),
    (lambda c: {"W": c["W"][0]}, ValueError),
    (lambda c: {"W": torch.zeros(3, 24, 16, dtype=BF).transpose(1, 2)}, ValueError),
    (lambda c: {"offsets": c["offsets"].int()}, ValueError),
    (lambda c: {"offsets": c["offsets"][:3]}, ValueError),
    (lambda c: {"offsets": torch.zeros(8, dtype=torch.int64)[::2]}, ValueError),
    (lambda c: {"out": torch.zeros(12, 17, dtype=BF)}, ValueError),
    (lambda c: {"out": torch.zeros(12, 16)}, ValueError),
    (lambda c: {"out": c["X"][:, :16]}, ValueError),                  # overlaps X
])
def test_matmul_refusals(change, error):
    X, W, dY, off = _case()
    args = {"X": X, "W": W, "offsets": off}
    args.update(change(args))
    with pytest.raises(error):
        mns.grouped_matmul(**args)


@pytest.mark.parametrize("change,error", [
    (lambda c: {"dY": c["dY"].float()}, TypeError),
    (lambda c: {"X": c["X"].double()}, TypeError),
    (lambda c: {"dY": c["dY"][:11]}, ValueError),
    (lambda c: {"offsets": c["offsets"][:1]}, ValueError),
    (lambda c: {"C": torch.zeros(3, 16, 23)}, ValueError),
    (lambda c: {"C": torch.zeros(3, 16, 24), "out": torch.zeros(3, 16, 24, dtype=BF)}, ValueError),
    (lambda c: {"out": torch.zeros(3, 24, 16).transpose(1, 2)}, ValueError),
    (lambda c: {"out_dtype": torch.float16}, TypeError),
    (lambda c: {"X": c["X"].float(), "dY": c["dY"].float(), "out_dtype": BF}, TypeError),
    (lambda c: {"out": c["X"].view(-1)[:0].new_zeros(0).expand(0)}, ValueError),
])
def test_weight_grad_refusals(change, error):
    X, W, dY, off = _case()
    args = {"dY": dY, "X": X, "offsets": off}
    args.update(change(args))
    with pytest.raises(error):
        mns.grouped_weight_grad(**args)


def test_weight_grad_part_overlap_is_refused():
    X, W, dY, off = _case()
    buf = torch.zeros(4, 16, 24)
    with pytest.raises(ValueError, match="itself"):
        mns.grouped_weight_grad(dY, X, off, C=buf[:3], out=buf[1:])


def _call(lib, **kw):
    a = dict(X=0x10000, ldx=24, W=0x20000, Y=0x30000, ldy=16, dtype=_abi.MNS_BF16, off=0x40000,
             groups=3, rows=12, n=16, k=24, t=0, fill=0, ws=None, wsb=0)
    a.update(kw)
    return lib.grouped_matmul(a["X"], a["ldx"], a["W"], a["Y"], a["ldy"], a["dtype"], a["off"],
                              a["groups"], a["rows"], a["n"], a["k"], a["t"], a["fill"], a["ws"],
                              a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), _abi.MNS_ERR_DTYPE),
    (dict(groups=0), _abi.MNS_ERR_SHAPE),
    (dict(groups=65537), _abi.MNS_ERR_SHAPE),
    (dict(rows=-1), _abi.MNS_ERR_SHAPE),
    (dict(rows=1 << 31), _abi.MNS_ERR_SHAPE),
    (dict(rows=(1 << 30) + 1), _abi.MNS_ERR_SHAPE),
    (dict(n=0), _abi.MNS_ERR_SHAPE),
    (dict(k=65537, ldx=65537), _abi.MNS_ERR_SHAPE),
    (dict(ldx=23), _abi.MNS_ERR_SHAPE),
    (dict(ldy=15), _abi.MNS_ERR_SHAPE),
    (dict(ldx=(1 << 21) + 1), _abi.MNS_ERR_SHAPE),
    (dict(t=1), _abi.MNS_ERR_SHAPE),              # ldy is 16, the transposed output 24 wide
    (dict(t=2), _abi.MNS_ERR_PARAM),
    (dict(fill=-1), _abi.MNS_ERR_PARAM),
    (dict(X=None), _abi.MNS_ERR_NULL),
    (dict(W=None), _abi.MNS_ERR_NULL),
    (dict(Y=None), _abi.MNS_ERR_NULL),
    (dict(off=None), _abi.MNS_ERR_NULL),
    (dict(X=0x10001), _abi.MNS_ERR_PARAM),
    (dict(Y=0x30001), _abi.MNS_ERR_PARAM),
    (dict(off=0x40004), _abi.MNS_ERR_PARAM),
    (dict(dtype=_abi.MNS_F32, W=0x20002), _abi.MNS_ERR_PARAM),
    # nothing to do: no launch, so no device is needed either
    (dict(rows=0, X=None, Y=None), _abi.MNS_OK),
])
def test_library_refuses_matmul(kw, status):
    assert _call(mns.load(), **kw) == status


def _call_w(lib, **kw):
    a = dict(dY=0x10000, lddy=16, X=0x20000, ldx=24, dtype=_abi.MNS_BF16, off=0x40000, groups=3,
             rows=12, n=16, k=24, C=None, beta=0.5, G=0x50000, od=_abi.MNS_F32, ws=None, wsb=0)
    a.update(kw)
    return lib.grouped_weight_grad(a["dY"], a["lddy"], a["X"], a["ldx"], a["dtype"], a["off"],
                                   a["groups"], a["rows"], a["n"], a["k"], a["C"], a["beta"],
                                   a["G"], a["od"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), _abi.MNS_ERR_DTYPE),
    (dict(od=5), _abi.MNS_ERR_DTYPE),
    (dict(dtype=_abi.MNS_F32, od=_abi.MNS_BF16), _abi.MNS_ERR_DTYPE),
    (dict(beta=float("nan")), _abi.MNS_ERR_PARAM),
    (dict(beta=float("inf")), _abi.MNS_ERR_PARAM),
    (dict(lddy=15), _abi.MNS_ERR_SHAPE),
    (dict(ldx=1 << 22), _abi.MNS_ERR_SHAPE),
    (dict(groups=65536, n=65536, k=32767, lddy=65536, ldx=32767), _abi.MNS_ERR_SHAPE),
    (dict(dY=None), _abi.MNS_ERR_NULL),
    (dict(G=None), _abi.MNS_ERR_NULL),
    (dict(off=None), _abi.MNS_ERR_NULL),
    (dict(C=0x60002), _abi.MNS_ERR_PARAM),
    (dict(G=0x50002), _abi.MNS_ERR_PARAM),
])
def test_library_refuses_weight_grad(kw, status):
    assert _call_w(mns.load(), **kw) == status


def test_workspace_query():
    lib = mns.load()
    out = ctypes.c_size_t(1)
    assert lib.mns_grouped_workspace_size(0, _abi.MNS_BF16, 3, 12, 16, 24, ctypes.byref(out)) == 0
    assert lib.mns_grouped_workspace_size(2, 1, 3, 12, 16, 24, ctypes.byref(out)) == _abi.MNS_ERR_PARAM
    assert lib.mns_grouped_workspace_size(1, 9, 3, 12, 16, 24, ctypes.byref(out)) == _abi.MNS_ERR_DTYPE
    assert lib.mns_grouped_workspace_size(1, 1, 0, 12, 16, 24, ctypes.byref(out)) == _abi.MNS_ERR_SHAPE
    assert lib.mns_grouped_workspace_size(1, 1, 3, 12, 16, 24, None) == _abi.MNS_ERR_NULL
