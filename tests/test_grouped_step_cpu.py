"""Refusals of muon_step_grouped that need no GPU."""
import ctypes

import pytest
import torch

import muon_newton_schulz_amd as mns
from muon_newton_schulz_amd import _abi

BF = torch.bfloat16
C5 = [(3.4445, -4.7750, 2.0315)] * 5


def _case(e=3, r=16, c=24, t=12):
    return dict(W=torch.zeros(e, r, c, dtype=BF), M=torch.zeros(e, r, c),
                dY=torch.zeros(t, r, dtype=BF), X=torch.zeros(t, c, dtype=BF),
                offsets=torch.zeros(e + 1, dtype=torch.int64), v=torch.zeros(e, r))


@pytest.mark.parametrize("change,error,match", [
    ({}, ValueError, "GPU"),
    ({"M": torch.zeros(3, 16, 23)}, ValueError, "shape"),
    ({"M": torch.zeros(3, 16, 24, dtype=torch.float64)}, TypeError, "momentum"),
    ({"dY": torch.zeros(12, 16)}, TypeError, "storage dtype"),
    ({"dY": torch.zeros(12, 17, dtype=BF)}, ValueError, "rows of 16"),
    ({"X": torch.zeros(11, 24, dtype=BF)}, ValueError, "same rows"),
    ({"v": torch.zeros(48)}, ValueError, "v must be"),
    ({"v": None}, ValueError, "NorMuon"),
    ({"offsets": torch.zeros(3, dtype=torch.int64)}, ValueError, "offsets"),
    ({"W": torch.zeros(3, 24, 16, dtype=BF).transpose(1, 2)}, ValueError, "contiguous"),
])
def test_binding_refuses(change, error, match):
    a = {**_case(), **change}
    v = a.pop("v")
    with pytest.raises(error, match=match):
        mns.muon_step_grouped(**a, v=v, mu=0.9, lr=0.1, coeffs=C5, normuon=True)


def test_state_overlapping_an_input_is_refused():
    a = _case()
    a["W"] = a["X"].new_zeros(3 * 16 * 24 + 8)[:1152].view(3, 16, 24)
    a["dY"] = a["W"].view(-1)[:192].view(12, 16)
    with pytest.raises(ValueError, match="overlap"):
        mns.muon_step_grouped(**a, mu=0.9, lr=0.1, coeffs=C5)


def _hp(**kw):
    abc = (ctypes.c_float * 15)(*([3.4445, -4.775, 2.0315] * 5))
    a = dict(mu=0.95, lr=0.02, T=5, abc=ctypes.cast(abc, ctypes.POINTER(ctypes.c_float)), kind=0,
             restart_mask=0, normuon=0, beta2=0.95, eps=1e-8, row_fraction=1.0,
             dtype=_abi.MNS_BF16)
    a.update(kw)
    return _abi.MnsHparams(**a), abc


@pytest.mark.parametrize("hp_kw,kw,status", [
    (dict(row_fraction=0.5), {}, _abi.MNS_ERR_PARAM),
    (dict(dtype=4), {}, _abi.MNS_ERR_DTYPE),
    (dict(T=0), {}, _abi.MNS_ERR_PARAM),
    (dict(mu=float("inf")), {}, _abi.MNS_ERR_PARAM),
    (dict(normuon=1), dict(v=None), _abi.MNS_ERR_NULL),
    ({}, dict(groups=0), _abi.MNS_ERR_SHAPE),
    ({}, dict(rows=0), _abi.MNS_ERR_SHAPE),
    ({}, dict(W=None), _abi.MNS_ERR_NULL),
    ({}, dict(M=None), _abi.MNS_ERR_NULL),
    ({}, dict(X=None), _abi.MNS_ERR_NULL),
    ({}, dict(off=None), _abi.MNS_ERR_NULL),
    ({}, dict(lddy=15), _abi.MNS_ERR_SHAPE),
    ({}, dict(W=0x10008), _abi.MNS_ERR_PARAM),
    ({}, dict(ws=None), _abi.MNS_ERR_WORKSPACE),
    ({}, dict(wsb=64), _abi.MNS_ERR_WORKSPACE),
])
def test_library_refuses(hp_kw, kw, status):
    lib = mns.load()
    hp, _keep = _hp(**hp_kw)
    a = dict(W=0x10000, M=0x20000, v=0x30000, dY=0x40000, lddy=16, X=0x50000, ldx=24, off=0x60000,
             groups=3, total=12, rows=16, cols=24, ws=0x100000, wsb=1 << 40)
    a.update(kw)
    assert lib.muon_step_grouped(a["W"], a["M"], a["v"], a["dY"], a["lddy"], a["X"], a["ldx"],
                                 a["off"], a["groups"], a["total"], a["rows"], a["cols"],
                                 ctypes.byref(hp), a["ws"], a["wsb"], None) == status
    assert lib.muon_step_grouped(a["W"], a["M"], a["v"], a["dY"], a["lddy"], a["X"], a["ldx"],
                                 a["off"], a["groups"], a["total"], a["rows"], a["cols"], None,
                                 a["ws"], a["wsb"], None) == _abi.MNS_ERR_NULL
