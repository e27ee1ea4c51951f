"""Layers of experts (product, bias, activation, residual), their input and bias gradients, against float64
on the CPU, element by element with derived bounds (layer_ref), on every kernel and at the sizes where a
tile, a chunk or a group ends."""
import ctypes

import pytest
import torch

import grouped_ref
import layer_ref as ref
import muon_newton_schulz_amd as mns
from muon_newton_schulz_amd import _abi

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
check = grouped_ref.check


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _offsets(bounds):
    return torch.tensor(bounds, dtype=torch.int64, device="cuda")


def _strided(t, pitch, lead=0):
    """t's values in rows `pitch` apart, starting `lead` elements into a buffer of 7s."""
    buf = torch.full((lead + t.shape[0] * pitch + 8,), 7.0, dtype=t.dtype, device=t.device)
    view = buf.as_strided(t.shape, (pitch, 1), lead)
    view.copy_(t)
    return view, buf


def _both(sizes, front, tail, n, k, dtype, act, bias=True, residual=True, wscale=0.3):
    bounds = grouped_ref.bounds_of(sizes, front)
    rows, e = bounds[-1] + tail, len(sizes)
    off = _offsets(bounds)
    W = _rand((e, n, k), dtype, 1, wscale)
    X, b = _rand((rows, k), dtype, 2), _rand((e, n), dtype, 3) if bias else None
    R = _rand((rows, n), dtype, 4) if residual else None
    keep = act is not None
    print("case", sizes, front, tail, n, k, dtype, act, "forward", flush=True)
    got = mns.grouped_linear(X, W, off, bias=b, activation=act, residual=R, keep_z=keep)
    Y, Z = got if keep else (got, None)
    zero = torch.zeros(rows, n, dtype=dtype)
    wY, eY, wZ, eZ = ref.linear(X, W, bounds, b, act, R, zero, zero)
    check(Y, wY, eY, ("Y", n, k))
    if keep:
        check(Z, wZ, eZ, ("Z", n, k))
    dY, Zin = _rand((rows, n), dtype, 5), _rand((rows, k), dtype, 6) if act else None
    R = _rand((rows, k), dtype, 7) if residual else None
    print("case", sizes, front, tail, n, k, dtype, act, "input gradient", flush=True)
    dX = mns.grouped_input_grad(dY, W, off, activation=act, Z=Zin, residual=R)
    check(dX, *ref.input_grad(dY, W, bounds, act, Zin, R, torch.zeros(rows, k, dtype=dtype)),
          ("dX", n, k))


ROUTES = {
    "one_token": ([0, 0, 1, 0], 0, 0),
    "one_expert": ([200], 0, 0),
    "even": ([64] * 4, 0, 0),
    "ragged": ([1, 0, 129, 127, 0, 33, 256, 2], 0, 5),
    "front_and_tail": ([7, 140], 3, 150),
    "all_empty": ([0] * 5, 0, 9),
    "many": ([(i * 7) % 5 for i in range(150)], 2, 1),
    "long": ([700, 3, 1100], 0, 0),
}
WIDTHS = [(64, 128), (1, 1), (65, 33), (256, 320), (130, 72), (24, 520)]


@pytest.mark.parametrize("route", sorted(ROUTES))
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_routes_and_widths(route, dtype):
    for i, (n, k) in enumerate(WIDTHS):
        _both(*ROUTES[route], n, k, dtype, (ref.ACTS + [None])[(i + len(route)) % 5])


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257])
def test_weights_between_dwords(k, lead):
    """An odd pitch, or weights that start between two dwords: the input gradient on both kernels that take
    any alignment, next to the tiles' widths; nothing of the neighbours gets into a column."""
    for sizes, n in (([20, 1], 70), ([20, 1], 2100), ([6200, 0, 5200], 70)):
        bounds = grouped_ref.bounds_of(sizes, 1)
        rows, e = bounds[-1] + 2, len(sizes)
        buf = torch.full((lead + e * n * k + 9,), float("nan"), dtype=BF, device="cuda")
        W = buf[lead:lead + e * n * k].view(e, n, k)
        W.copy_(_rand((e, n, k), BF, 1))
        dY, R = _rand((rows, n), BF, 2), _rand((rows, k), BF, 3)
        print("case", sizes, n, k, lead, flush=True)
        zero = torch.zeros(rows, k, dtype=BF)
        got = mns.grouped_input_grad(dY, W, _offsets(bounds), residual=R)
        check(got, *ref.input_grad(dY, W, bounds, None, None, R, zero), (n, k))
        got = mns.grouped_matmul(dY, W, _offsets(bounds), transpose_w=True)
        check(got, *grouped_ref.matmul(dY, W, bounds, True, zero), (n, k))


# Few tiles with a long reduction: cut into parts over the blocks, then joined. (route, output width,
# reduction, dtype); the forward takes this way beyond 96 rows an expert.
PARTS = [
    (([141], 0, 0), 70, 2100, BF), (([100, 130], 3, 70), 65, 1090, F32), (([300, 0, 200], 0, 1), 130, 2049, BF),
    (([1], 0, 0), 1, 2050, BF), (([0, 1, 0], 2, 66), 33, 1025, F32), (([1] * 9 + [0] * 60, 1, 2), 40, 1030, F32),
    (([64, 65, 32, 33], 0, 64), 64, 6500, BF), (([31, 97], 64, 0), 320, 6080, F32),
    (([120, 1, 0, 300], 3, 0), 200, 2048, BF), (([130], 0, 5), 64, 4096, BF), (([45] * 5, 1, 0), 72, 3968, BF),
]


@pytest.mark.parametrize("i", range(len(PARTS)))
def test_reduction_in_parts(i):
    route, width, red, dtype = PARTS[i]
    need = ctypes.c_size_t(0)
    rows = sum(route[0]) + route[1] + route[2]
    for back, n, k in ((1, red, width), (0, width, red)):
        _abi.check(mns.load().mns_grouped_layer_workspace_size(
            back, _abi.MNS_F32 if dtype == F32 else _abi.MNS_BF16, len(route[0]), rows, n, k,
            ctypes.byref(need)), "size")
        assert need.value > 0 or (not back and rows <= 96 * len(route[0]))
        _both(*route, n, k, dtype, (ref.ACTS + [None])[i % 5], wscale=0.05)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_parts_with_overlapping_offsets_stay_inside(dtype):
    """Every expert claims all rows: values unspecified, nothing outside the rows is written."""
    rows, e, n, k = 90, 7, 4100, 70
    off = torch.tensor([v for _ in range(4) for v in (0, rows)], dtype=torch.int64, device="cuda")
    buf = torch.full((rows + 8, k + 3), 7.0, dtype=dtype, device="cuda")
    mns.grouped_input_grad(_rand((rows, n), dtype, 1), _rand((e, n, k), dtype, 2), off,
                           residual=_rand((rows, k), dtype, 3), out=buf[4:4 + rows, :k])
    assert (buf[:4] == 7).all() and (buf[4 + rows:] == 7).all() and (buf[:, k:] == 7).all()


# (sizes, front, tail), n, k, dtype, the kernels that take the forward and the input gradient; the first
# rows: every tile of the kernel for few rows, in both types
KERNELS = [
    (([3, 0, 5], 1, 2), 96, 200, BF, "grouped_rows_bf16", "grouped_64_nn_bf16"),
    (([3, 0, 5], 1, 2), 97, 201, F32, "grouped_rows_f32", "grouped_64_nn_f32"),
    (([5] * 40, 0, 3), 1000, 96, BF, "grouped_rows_bf16", None),
    (([5] * 40, 0, 3), 1001, 97, F32, "grouped_rows_f32", None),
    (([5] * 40, 0, 3), 4096, 160, BF, "grouped_rows_bf16", "grouped_256_nn"),
    (([2] * 60, 0, 3), 8200, 96, F32, "grouped_rows_f32", None),
    (([30, 28], 0, 3), 520, 250, BF, "grouped_rows_bf16", None),
    (([30, 28], 0, 3), 520, 250, F32, "grouped_rows_f32", None),
    (([30] * 40, 0, 3), 900, 96, BF, "grouped_rows_bf16", None),
    (([30] * 40, 0, 3), 900, 96, F32, "grouped_rows_f32", None),
    (([25] * 40, 0, 3), 3200, 100, BF, "grouped_rows_bf16", None),
    (([25] * 40, 0, 3), 3200, 100, F32, "grouped_rows_f32", None),
    (([50, 60], 0, 3), 260, 100, BF, "grouped_rows_bf16", None),
    (([60] * 8, 0, 3), 90, 96, F32, "grouped_rows_f32", None),
    (([50] * 40, 0, 3), 1100, 72, BF, "grouped_rows_bf16", None),
    (([50] * 40, 0, 3), 1100, 72, F32, "grouped_rows_f32", None),
    (([60] * 20, 0, 3), 6400, 72, BF, "grouped_rows_bf16", "grouped_256_nn"),
    (([60] * 20, 0, 3), 6400, 72, F32, "grouped_rows_f32", None),
    (([300, 220], 2, 3), 130, 72, BF, "grouped_64_nt_bf16", "grouped_64_nn_bf16"),
    (([300, 220], 2, 3), 130, 72, F32, "grouped_64_nt_f32", "grouped_64_nn_f32"),
    (([900, 1300], 2, 3), 1283, 1410, BF, "grouped_128_nt_bf16", "grouped_128_nn_bf16"),
    (([900, 1300], 2, 3), 1284, 1408, F32, "grouped_128_nt_f32", "grouped_128_nn_f32"),
    (([70, 40, 90], 3, 4), 512, 640, BF, "grouped_ring_nt", "grouped_ring_nn"),
    (([100] * 8, 3, 4), 4160, 1024, BF, "grouped_ring_nt", "grouped_ring_nn"),
    (([100] * 8, 3, 4), 1024, 4160, BF, "grouped_ring_nt", "grouped_ring_nn"),
    (([2000, 1700, 0, 800], 5, 6), 2048, 2304, BF, "grouped_256_nt", "grouped_256_nn"),
    (([700, 900], 3, 9), 520, 2560, BF, "grouped_256_nt", None),         # in parts, joined
    (([700, 900], 3, 9), 2560, 520, BF, None, "grouped_256_nn"),
    (([1100, 800, 0, 500], 0, 1), 5376, 1600, BF, "grouped_256_nt", None),   # a whole round, then parts
    (([1100, 800, 0, 500], 0, 1), 1600, 5376, BF, None, "grouped_256_nn"),
]


@pytest.mark.parametrize("i", range(len(KERNELS)))
def test_every_kernel(i):
    route, n, k, dtype, forward, back = KERNELS[i]
    mns.profile_begin()
    try:
        _both(*route, n, k, dtype, ref.ACTS[i % 4], wscale=0.05)
    finally:
        names = [r["name"] for r in mns.profile_end()]
    if forward:
        assert names[0] == forward, names
    if back:
        assert names[-1] == back, names


@pytest.mark.parametrize("act", [None] + ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_activations_over_their_range(act, dtype):
    """Values from the tails to the middle, through a product with the identity."""
    n = 64
    z = torch.cat([torch.linspace(-14, 14, 190 * n - 8), torch.tensor(
        [0.0, -0.0, 1e-30, -1e-30, -100.0, 100.0, 1e-4, -1e-4])]).reshape(190, n).to(dtype).cuda()
    W = torch.eye(n, dtype=dtype, device="cuda")[None].contiguous()
    off = _offsets([0, 190])
    got = mns.grouped_linear(z, W, off, activation=act)
    want, err, _, _ = ref.linear(z, W, [0, 190], None, act, None, torch.zeros(190, n),
                                 torch.zeros(190, n))
    check(got, want, err, act)
    if act is None:
        return
    g = _rand((190, n), dtype, 3)
    check(mns.grouped_input_grad(g, W, off, activation=act, Z=z),
          *ref.input_grad(g, W, [0, 190], act, z, None, torch.zeros(190, n)), act)
    db, dZ = mns.grouped_bias_grad(g, off, activation=act, Z=z, out_dtype=F32)
    wb, eb, wz, ez = ref.bias_grad(g, [0, 190], act, z, F32, torch.zeros(190, n))
    check(db, wb, eb, act)
    check(dZ, wz, ez, act)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [([40, 0, 90], 65, 130), ([600, 900], 512, 256)])
def test_pitches_alignment_and_given_outputs(dtype, sizes, n, k):
    """Row pitches, addresses off the 16-byte grid; what lies around and behind stays as it was."""
    bounds = grouped_ref.bounds_of(sizes, 2)
    rows, e = bounds[-1] + 3, len(sizes)
    off = _offsets(bounds)
    W, b = _rand((e, n, k), dtype, 1, 0.2), _rand((e, n), dtype, 2)
    for lead, pad in ((0, 8), (1, 3), (3, 16)):
        X, _ = _strided(_rand((rows, k), dtype, 3), k + pad, lead)
        R, _ = _strided(_rand((rows, n), dtype, 4), n + 2 * pad, lead)
        out, buf = _strided(_rand((rows, n), dtype, 5), n + pad, lead)
        oz, bufz = _strided(_rand((rows, n), dtype, 6), n + 5, lead)
        old, oldz, before, beforez = out.clone(), oz.clone(), buf.clone(), bufz.clone()
        Y, Z = mns.grouped_linear(X, W, off, bias=b, activation="silu", residual=R, out=out, out_z=oz)
        assert Y is out and Z is oz
        wY, eY, wZ, eZ = ref.linear(X, W, bounds, b, "silu", R, old, oldz)
        check(Y, wY, eY, "Y")
        check(Z, wZ, eZ, "Z")
        out.copy_(old)
        oz.copy_(oldz)
        assert torch.equal(buf, before) and torch.equal(bufz, beforez)      # nothing else written
        dY, _ = _strided(_rand((rows, n), dtype, 7), n + pad, lead)
        Zin, _ = _strided(_rand((rows, k), dtype, 8), k + pad, lead)
        out, buf = _strided(_rand((rows, k), dtype, 9), k + 7, lead)
        old, before = out.clone(), buf.clone()
        mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Zin, out=out)
        check(out, *ref.input_grad(dY, W, bounds, "gelu", Zin, None, old), "dX")
        out.copy_(old)
        assert torch.equal(buf, before)


@pytest.mark.parametrize("dtype,sizes,n,k", [(BF, [30, 7], 72, 136), (F32, [30, 7], 72, 136),
                                             (BF, [2100, 1900], 1024, 512), (F32, [700, 900], 300, 257),
                                             (BF, [90, 100, 110], 512, 512)])
def test_in_place(dtype, sizes, n, k):
    bounds = grouped_ref.bounds_of(sizes)
    rows, e = bounds[-1] + 2, len(sizes)
    off, W = _offsets(bounds), _rand((e, n, k), dtype, 1, 0.1)
    X, R = _rand((rows, k), dtype, 2), _rand((rows, n), dtype, 3)
    want = mns.grouped_linear(X, W, off, activation="relu2", residual=R, out=R.clone())
    got = mns.grouped_linear(X, W, off, activation="relu2", residual=R, out=R)
    assert got is R and torch.equal(got, want)
    dY, Z = _rand((rows, n), dtype, 4), _rand((rows, k), dtype, 5)
    res = _rand((rows, k), dtype, 6)
    want = mns.grouped_input_grad(dY, W, off, activation="silu", Z=Z, residual=res, out=Z.clone())
    over_z = Z.clone()
    mns.grouped_input_grad(dY, W, off, activation="silu", Z=over_z, residual=res, out=over_z)
    assert torch.equal(over_z, want)
    over_r = res.clone()
    mns.grouped_input_grad(dY, W, off, activation="silu", Z=Z, residual=over_r, out=over_r)
    last = bounds[-1]
    assert torch.equal(over_r[:last], want[:last]) and torch.equal(over_r[last:], res[last:])
    g = _rand((rows, k), dtype, 7)
    db, dz = mns.grouped_bias_grad(g, off, activation="gelu", Z=Z)
    for which in ("dY", "Z"):
        g2, z2 = g.clone(), Z.clone()
        db2, dz2 = mns.grouped_bias_grad(g2, off, activation="gelu", Z=z2,
                                         out_dz=g2 if which == "dY" else z2)
        assert torch.equal(db, db2) and torch.equal(dz[:last], dz2[:last])


def test_mixed_given_and_new_outputs():
    bounds = [1, 20, 20, 31]
    W, X, off = _rand((3, 40, 24), BF, 1), _rand((35, 24), BF, 2), _offsets(bounds)
    zero = torch.zeros(35, 40, dtype=BF)
    wY, eY, wZ, eZ = ref.linear(X, W, bounds, None, "gelu", None, zero, zero)
    given = torch.full((35, 40), 3.0, dtype=BF, device="cuda")
    Y, Z = mns.grouped_linear(X, W, off, activation="gelu", keep_z=True, out=given)
    check(Z, wZ, eZ, "Z new")
    check(Y[1:31], wY[1:31], eY[1:31], "Y given")
    assert (Y[:1] == 3).all() and (Y[31:] == 3).all()
    given = torch.full((35, 40), 3.0, dtype=BF, device="cuda")
    Y, Z = mns.grouped_linear(X, W, off, activation="gelu", out_z=given)
    check(Y, wY, eY, "Y new")
    check(Z[1:31], wZ[1:31], eZ[1:31], "Z given")
    assert (Z[:1] == 3).all() and (Z[31:] == 3).all()


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)],
                         ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("route", sorted(ROUTES))
def test_bias_grad(route, dtype, out_dtype):
    sizes, front, tail = ROUTES[route]
    bounds = grouped_ref.bounds_of(sizes, front)
    rows, off = bounds[-1] + tail, _offsets(bounds)
    for i, n in enumerate((1, 8, 33, 256, 263, 600)):
        act = (ref.ACTS + [None])[i % 5]
        print("case", route, dtype, n, act, flush=True)
        dY, Z = _rand((rows, n), dtype, 1), _rand((rows, n), dtype, 2) if act else None
        got = mns.grouped_bias_grad(dY, off, activation=act, Z=Z, out_dtype=out_dtype)
        wb, eb, wz, ez = ref.bias_grad(dY, bounds, act, Z, out_dtype, torch.zeros(rows, n))
        if act:
            check(got[1], wz, ez, (route, n, "dZ"))
            got = got[0]
        check(got, wb, eb, (route, n, "db"))


@pytest.mark.parametrize("rows", [128, 129, 5000, 70000])
def test_bias_grad_chunks(rows):
    """One chunk, two, many, and so many rows that the chunks grow; equal calls give equal bits."""
    sizes = [rows // 3, 0, rows - rows // 3 - 1]
    bounds = grouped_ref.bounds_of(sizes, 1)
    off, n = _offsets(bounds), 40
    dY, Z = _rand((rows + 4, n + 3), F32, 1)[:, :n], _rand((rows + 4, n), F32, 2)
    db, dZ = mns.grouped_bias_grad(dY, off, activation="silu", Z=Z)
    wb, eb, wz, ez = ref.bias_grad(dY, bounds, "silu", Z, F32, torch.zeros(rows + 4, n))
    check(db, wb, eb, rows)
    check(dZ, wz, ez, rows)
    out = torch.empty_like(db)
    again, dz2 = mns.grouped_bias_grad(dY, off, activation="silu", Z=Z, out=out,
                                       out_dz=torch.zeros_like(dZ))
    assert again is out and torch.equal(again, db) and torch.equal(dz2, dZ)


def test_bias_grad_beyond_the_caches():
    """More than 256 MB, read and written past the caches, odd widths and pitches."""
    n, sizes = 8187, [1, 3000, 0, 4007]
    bounds = grouped_ref.bounds_of(sizes, 1)
    rows, off = bounds[-1] + 2, _offsets(bounds)
    g = torch.Generator("cuda").manual_seed(1)
    dY = torch.empty(rows, n + 3, dtype=BF, device="cuda").normal_(generator=g)[:, 1:n + 1]
    Z = torch.empty(rows, n, dtype=BF, device="cuda").normal_(generator=g)
    db, dZ = mns.grouped_bias_grad(dY, off, activation="relu", Z=Z, out_dtype=F32)
    want = torch.where(Z > 0, dY, torch.zeros_like(dY))             # exact
    want[:1], want[bounds[-1]:] = 0, 0
    assert torch.equal(dZ, want)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        part = want[lo:hi].double()
        err = (hi - lo + 1) * 2.0 ** -23 * part.abs().sum(0) + 1e-38
        assert ((db[e].double() - part.sum(0)).abs() <= err).all(), e


def test_widths_the_large_kernels_do_not_take():
    """A reduction of whole k-tiles with an odd output: no whole 16-byte pieces to store."""
    for sizes, n, k in (([700, 900], 1001, 1024), ([40, 50], 77, 256), ([300], 2049, 2048)):
        _both(sizes, 1, 2, n, k, BF, "silu", wscale=0.05)


def test_no_rows_at_all():
    W, off = _rand((3, 16, 24), BF, 1), _offsets([0, 0, 0, 0])
    X, dY = torch.empty(0, 24, dtype=BF, device="cuda"), torch.empty(0, 16, dtype=BF, device="cuda")
    Y, Z = mns.grouped_linear(X, W, off, activation="gelu", keep_z=True)
    assert Y.shape == Z.shape == (0, 16)
    assert mns.grouped_input_grad(dY, W, off).shape == (0, 24)
    db = mns.grouped_bias_grad(dY, off)
    assert db.shape == (3, 16) and (db == 0).all()


def test_wrong_offsets_stay_inside():
    """Offsets that overlap, run backwards or lie outside: unspecified values, no access outside."""
    W, X, dY = _rand((4, 512, 256), BF, 1), _rand((900, 256), BF, 2), _rand((900, 512), BF, 3)
    Z = _rand((900, 256), BF, 4)
    for bounds in ([0, 900, 0, 900, 0], [-5, 2 ** 40, 7, -(2 ** 50), 3], [900, 900, 0, 0, 900]):
        off = _offsets(bounds)
        mns.grouped_linear(X, W, off, activation="gelu", keep_z=True)
        mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Z)
        mns.grouped_bias_grad(X, off, activation="gelu", Z=Z)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_nan_and_infinity_stay_in_their_rows(dtype):
    bounds, n, k = [0, 70, 300], 96, 128
    off, W = _offsets(bounds), _rand((2, n, k), dtype, 1, 0.2)
    X, R = _rand((305, k), dtype, 2), _rand((305, n), dtype, 3)
    clean = mns.grouped_linear(X, W, off, activation="gelu", residual=R)
    X[5, 3], X[302] = float("nan"), float("nan")
    R[80, 7] = float("inf")
    got = mns.grouped_linear(X, W, off, activation="gelu", residual=R)
    assert got[5].isnan().all() and got[80, 7] == float("inf") and (got[300:] == 0).all()
    keep = [i for i in range(300) if i not in (5, 80)]
    assert torch.equal(got[keep], clean[keep])
    for act in ref.ACTS:
        z = torch.full((305, n), float("nan"), dtype=dtype, device="cuda")
        g = _rand((305, n), dtype, 4)
        db, dz = mns.grouped_bias_grad(g, off, activation=act, Z=z)
        assert (dz[300:] == 0).all()
        assert act in ("relu", "relu2") or dz[:300].isnan().all()
        y = mns.grouped_linear(X, W, off, activation=act)
        assert y[5].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(37, 45), (300, 129), (33, 515)])
@pytest.mark.parametrize("rows", [12, 300, 3000])
def test_what_follows_a_row_does_not_reach_it(dtype, n, k, rows):
    """Odd widths, whose last vectors of a row reach into the next one: NaN in every second row, in the
    other expert's weights and bias, and between the rows."""
    bounds = [0, rows, rows, 2 * rows]
    off = _offsets(bounds)
    W, b = _rand((3, n, k), dtype, 1, 0.2), _rand((3, n), dtype, 2)
    X, R, dY = _rand((2 * rows, k), dtype, 3), _rand((2 * rows, n), dtype, 4), _rand((2 * rows, n), dtype, 5)
    Z = _rand((2 * rows, k), dtype, 6)
    calls = (lambda: mns.grouped_linear(X, W, off, bias=b, activation="silu", residual=R),
             lambda: mns.grouped_input_grad(dY, W, off, activation="silu", Z=Z),
             lambda: mns.grouped_bias_grad(dY, off, activation="silu", Z=R)[1],
             lambda: mns.grouped_matmul(X, W, off), lambda: mns.grouped_matmul(dY, W, off, transpose_w=True))
    clean = [call() for call in calls]
    keep = torch.arange(0, rows, 2)
    nan = float("nan")
    for t in (X, R, dY, Z):
        t[1:rows:2] = nan
        t[rows:] = nan
    W[1:] = nan
    b[1:] = nan
    for i, (call, want) in enumerate(zip(calls, clean)):
        print("case", dtype, n, k, rows, i, flush=True)
        assert torch.equal(call()[keep], want[keep]), i
    g = mns.grouped_weight_grad(dY[:rows:2], X[:rows:2], _offsets([0, len(keep)]))
    assert torch.isfinite(g).all()


def test_gradients_against_differences():
    """The layer's calls together: dX, dW and db of L = <C, gelu(X W^T + b) + R> against central
    differences of the float64 form."""
    bounds, n, k = [0, 9, 9, 30], 20, 14
    off, rows = _offsets(bounds), 30
    X, W = _rand((rows, k), F32, 1), _rand((3, n, k), F32, 2, 0.4)
    b, R, C = _rand((3, n), F32, 3), _rand((rows, n), F32, 4), _rand((rows, n), F32, 5)
    Y, Z = mns.grouped_linear(X, W, off, bias=b, activation="gelu", residual=R, keep_z=True)
    db, dZ = mns.grouped_bias_grad(C, off, activation="gelu", Z=Z)
    dX = mns.grouped_input_grad(dZ, W, off)
    dW = mns.grouped_weight_grad(dZ, X, off)

    def loss(Xd, Wd, bd):
        total = 0.0
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            z = Xd[lo:hi] @ Wd[e].t() + bd[e]
            total += float((C[lo:hi].cpu().double() * (ref.act("gelu", z)[0]
                                                       + R[lo:hi].cpu().double())).sum())
        return total

    args = [t.cpu().double() for t in (X, W, b)]
    g = torch.Generator().manual_seed(9)
    for i, grad in enumerate((dX, dW, db)):
        for _ in range(3):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + 1e-5 * v, args[i] - 1e-5 * v
            diff = (loss(*up) - loss(*down)) / 2e-5
            mine = float((grad.cpu().double() * v).sum())
            # differences: 1e-10 curvature and 1e-16 |L| / 1e-5; float32 gradients: k + n + 20 roundings
            size = float((grad.cpu().double() * v).abs().sum())
            assert abs(mine - diff) <= (n + k + 20) * 2.0 ** -23 * size + 1e-6, (i, mine, diff)


def test_captured_and_replayed():
    """Captured calls follow the offsets and inputs of each replay."""
    n, k, rows = 256, 512, 700
    W, b = _rand((4, n, k), BF, 1, 0.1), _rand((4, n), BF, 2)
    X, off = _rand((rows, k), BF, 3), _offsets([0, 100, 100, 400, 690])
    dY, Zin = _rand((rows, n), BF, 4), _rand((rows, k), BF, 5)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step():
        Y, Z = mns.grouped_linear(X, W, off, bias=b, activation="gelu", keep_z=True, workspace=ws)
        dX = mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Zin, workspace=ws)
        db, dZ = mns.grouped_bias_grad(dY, off, activation="gelu", Z=Z, workspace=ws)
        return Y, Z, dX, db, dZ

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed, bounds in enumerate(([0, 100, 100, 400, 690], [0, 0, 650, 651, 700], [5, 9, 20, 20, 20])):
        off.copy_(_offsets(bounds))
        X.copy_(_rand((rows, k), BF, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want), (seed, bounds)


def test_two_streams_at_once():
    bounds, n, k = [0, 900, 1000, 2300], 768, 1024
    off, W = _offsets(bounds), _rand((3, n, k), BF, 1, 0.1)
    X, Z = _rand((2300, k), BF, 2), _rand((2300, n), BF, 3)
    torch.cuda.synchronize()

    def step(stream):
        Y = mns.grouped_linear(X, W, off, activation="gelu", stream=stream)
        return Y, *mns.grouped_bias_grad(Z, off, activation="silu", Z=Z, stream=stream)

    want = step(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[step(s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in outs:
        for got in pair:
            assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_parts_in_place_captured_and_on_two_streams(dtype):
    rows, e, n, k = 150, 3, 2500, 130
    W, off = _rand((e, n, k), dtype, 1, 0.1), _offsets([0, 40, 41, 150])
    dY, Z = _rand((rows, n), dtype, 2), _rand((rows, k), dtype, 3)

    def step(out=None, stream=None):
        return mns.grouped_input_grad(dY, W, off, activation="gelu", Z=Z if out is None else out, out=out,
                                      stream=stream)

    want = step()
    assert torch.equal(step(), want) and torch.equal(step(Z.clone()), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [step(stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for bounds in ([0, 0, 0, 150], [3, 60, 130, 140], [0, 150, 150, 150]):
        off.copy_(_offsets(bounds))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, step()), bounds
