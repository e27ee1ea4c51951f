"""Products grouped by expert against float64 on the CPU, element by element with derived bounds
(grouped_ref), at the sizes where a tile, a chunk or a group ends: no rows, one row, many empty
experts, odd widths, row pitches, addresses off the 16-byte grid, rows of no expert."""
import pytest
import torch

import grouped_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _offsets(bounds):
    return torch.tensor(bounds, dtype=torch.int64, device="cuda")


def _strided(t, pitch, lead=0):
    """t's values in rows `pitch` apart, starting `lead` elements into a buffer of 7s."""
    buf = torch.full((lead + t.shape[0] * pitch + 8,), 7.0, dtype=t.dtype, device=t.device)
    view = buf[lead:].as_strided(t.shape, (pitch, 1), lead)
    view.copy_(t)
    return view, buf


# sizes of the experts' row groups, rows before the first and behind the last
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
def test_matmul_both_ways(route, dtype):
    sizes, front, tail = ROUTES[route]
    bounds = ref.bounds_of(sizes, front)
    rows = bounds[-1] + tail
    for i, (n, k) in enumerate(WIDTHS):
        W = _rand((len(sizes), n, k), dtype, 100 + i, 0.3)
        for t in (False, True):
            print("case", route, dtype, n, k, "transpose_w", t, flush=True)
            X = _rand((rows, n if t else k), dtype, i)
            out = mns.grouped_matmul(X, W, _offsets(bounds), transpose_w=t)
            ref.check(out, *ref.matmul(X, W, bounds, t, torch.zeros_like(out)), (route, n, k, t))


@pytest.mark.parametrize("route", sorted(ROUTES))
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)],
                         ids=["bf16", "bf16_f32", "f32"])
def test_weight_grad(route, dtype, out_dtype):
    sizes, front, tail = ROUTES[route]
    bounds = ref.bounds_of(sizes, front)
    rows = bounds[-1] + tail
    for i, (n, k) in enumerate(WIDTHS):
        print("case", route, dtype, out_dtype, n, k, flush=True)
        dY, X = _rand((rows, n), dtype, i, 0.2), _rand((rows, k), dtype, 50 + i)
        out = mns.grouped_weight_grad(dY, X, _offsets(bounds), out_dtype=out_dtype)
        ref.check(out, *ref.weight_grad(dY, X, bounds, None, 0.0, out_dtype), (route, n, k))
        C = _rand((len(sizes), n, k), out_dtype, 70 + i)
        want = ref.weight_grad(dY, X, bounds, C, 0.95, out_dtype)
        got = mns.grouped_weight_grad(dY, X, _offsets(bounds), C=C, beta=0.95, out=C)
        assert got is C
        ref.check(C, *want, (route, n, k, "in place"))


# more than one tile in every direction, on both sides of whole ones, groups that end inside a
# row tile, rows enough for the large tiles (and, f32, the same shapes on the others)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(512, 576), (520, 320), (192, 1000), (640, 64), (257, 448)])
def test_many_tiles(dtype, n, k):
    for sizes, front, tail in (([1500, 0, 257, 63], 3, 300), ([256, 512], 0, 0)):
        bounds = ref.bounds_of(sizes, front)
        rows, e = bounds[-1] + tail, len(sizes)
        W, off = _rand((e, n, k), dtype, 1, 0.3), _offsets(bounds)
        X, dY = _rand((rows, k), dtype, 2), _rand((rows, n), dtype, 3)
        print("case", dtype, n, k, sizes, flush=True)
        Y = mns.grouped_matmul(X, W, off)
        ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), "forward")
        dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
        ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), "input gradient")
        for out_dtype in {dtype, F32}:
            C = _rand((e, n, k), out_dtype, 4)
            for c, beta in ((None, 0.0), (C, -0.7)):
                G = mns.grouped_weight_grad(dY, X, off, C=c, beta=beta, out_dtype=out_dtype)
                ref.check(G, *ref.weight_grad(dY, X, bounds, c, beta, out_dtype), "weight gradient")


@pytest.mark.parametrize("sizes", [[600, 150, 0, 400], [3000], [1100, 1500]])
def test_long_reductions_in_parts(sizes):
    """Few tiles and a long reduction: the tiles are computed in parts and joined."""
    n, k = 384, 2048
    bounds = ref.bounds_of(sizes, 1)
    rows, e = bounds[-1] + 2, len(sizes)
    off = _offsets(bounds)
    W, X = _rand((e, n, k), BF, 1, 0.3), _rand((rows, k), BF, 2)
    Y = mns.grouped_matmul(X, W, off)
    ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), "forward")
    W, dY = _rand((e, k, n), BF, 3, 0.3), _rand((rows, k), BF, 4)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), "input gradient")
    dY = _rand((rows, n), BF, 5)
    for out_dtype in (BF, F32):
        C = _rand((e, n, k), out_dtype, 6)
        G = mns.grouped_weight_grad(dY, X, off, C=C, beta=0.5)
        ref.check(G, *ref.weight_grad(dY, X, bounds, C, 0.5, out_dtype), "weight gradient")
    again = mns.grouped_weight_grad(dY, X, off, C=C, beta=0.5)
    assert torch.equal(again, G)


def test_more_experts_than_lanes_with_many_rows():
    sizes = [(i * 37) % 300 + (i % 3 == 0) * 90 for i in range(70)]
    n, k = 136, 192
    bounds = ref.bounds_of(sizes, 5)
    rows, off = bounds[-1] + 7, _offsets(bounds)
    assert rows >= 128 * len(sizes)
    W, X, dY = _rand((70, n, k), BF, 1, 0.3), _rand((rows, k), BF, 2), _rand((rows, n), BF, 3)
    Y = mns.grouped_matmul(X, W, off)
    ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), "forward")
    G = mns.grouped_weight_grad(dY, X, off)
    ref.check(G, *ref.weight_grad(dY, X, bounds, None, 0.0, BF), "weight gradient")
    W, dY = _rand((70, k, n), BF, 4, 0.3), _rand((rows, k), BF, 5)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), "input gradient")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_no_rows_at_all(dtype):
    W = _rand((3, 40, 24), dtype, 1)
    X = torch.empty(0, 24, dtype=dtype, device="cuda")
    off = _offsets([0, 0, 0, 0])
    assert mns.grouped_matmul(X, W, off).shape == (0, 40)
    G = mns.grouped_weight_grad(torch.empty(0, 40, dtype=dtype, device="cuda"), X, off)
    assert G.shape == (3, 40, 24) and not G.any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead,extra", [(0, 24), (1, 24), (3, 5)])
def test_row_pitches_and_addresses(dtype, lead, extra):
    sizes, n, k = [70, 0, 5, 130], 72, 136
    bounds = ref.bounds_of(sizes, 2)
    rows = bounds[-1] + 4
    X0, dY0 = _rand((rows, k), dtype, 1), _rand((rows, n), dtype, 2)
    X, _ = _strided(X0, k + extra, lead)
    dY, _ = _strided(dY0, n + extra, lead)
    Wbuf = torch.empty(4 * n * k + 8, dtype=dtype, device="cuda")
    W = Wbuf[lead:lead + 4 * n * k].view(4, n, k)
    W.copy_(_rand((4, n, k), dtype, 3, 0.3))
    off = _offsets(bounds)
    for t, src, width in ((False, X, n), (True, dY, k)):
        out, buf = _strided(torch.full((rows, width), 3.0, dtype=dtype, device="cuda"),
                            width + extra, lead)
        before = buf.clone()
        want, err = ref.matmul(src, W, bounds, t, out)
        assert mns.grouped_matmul(src, W, off, transpose_w=t, out=out) is out
        ref.check(out, want, err, ("pitch", lead, extra, t))
        # rows of no expert and the gaps between rows keep what they held
        touched = torch.zeros_like(buf, dtype=torch.bool)
        touched[lead:].as_strided(out.shape, (width + extra, 1), lead)[bounds[0]:bounds[-1]] = True
        assert torch.equal(buf[~touched], before[~touched])
    G = mns.grouped_weight_grad(dY, X, off)
    ref.check(G, *ref.weight_grad(dY, X, bounds, None, 0.0, dtype), ("pitch", lead, extra))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_nothing_leaks_between_experts(dtype):
    """NaN and infinity in one expert's rows, in the rows of no expert and in one expert's matrix
    stay there."""
    sizes, n, k = [20, 31, 0, 40], 48, 104
    bounds = ref.bounds_of(sizes, 5)
    rows = bounds[-1] + 6
    X, dY = _rand((rows, k), dtype, 1), _rand((rows, n), dtype, 2)
    W = _rand((4, n, k), dtype, 3)
    off = _offsets(bounds)
    clean = [mns.grouped_matmul(X, W, off), mns.grouped_matmul(dY, W, off, transpose_w=True),
             mns.grouped_weight_grad(dY, X, off)]
    for t in (X, dY):
        t[:5] = float("nan")
        t[bounds[1]:bounds[2]] = float("inf")
        t[bounds[-1]:] = float("nan")
    W[1] = float("nan")
    W[2] = float("inf")
    got = [mns.grouped_matmul(X, W, off), mns.grouped_matmul(dY, W, off, transpose_w=True),
           mns.grouped_weight_grad(dY, X, off)]
    keep = torch.ones(rows, dtype=torch.bool)
    keep[bounds[1]:bounds[2]] = False
    for c, g in zip(clean[:2], got[:2]):
        assert torch.equal(g.cpu()[keep], c.cpu()[keep])
        assert not torch.isfinite(g.cpu()[~keep]).any()
    assert torch.equal(got[2][[0, 2, 3]], clean[2][[0, 2, 3]])
    assert not torch.isfinite(got[2][1]).any()


def test_beta_zero_reads_no_addend():
    sizes, n, k = [3, 0, 9], 40, 72
    bounds = ref.bounds_of(sizes)
    dY, X = _rand((12, n), BF, 1), _rand((12, k), BF, 2)
    C = torch.full((3, n, k), float("nan"), device="cuda")
    G = mns.grouped_weight_grad(dY, X, _offsets(bounds), C=C, beta=0.0)
    ref.check(G, *ref.weight_grad(dY, X, bounds, None, 0.0, F32))


def test_offsets_out_of_range_stay_inside_the_buffers():
    """Offsets below zero, beyond the rows or decreasing are clamped; the valid experts' rows hold
    the right values."""
    n, k, rows = 40, 72, 60
    X, W = _rand((rows, k), BF, 1), _rand((4, n, k), BF, 2)
    dY = _rand((rows, n), BF, 3)
    off = _offsets([-(1 << 40), 20, 30, 1 << 40, -5])
    want = [0, 20, 30, 60, 60]
    out = mns.grouped_matmul(X, W, off)
    ref.check(out[:60], *ref.matmul(X, W, want, False, torch.zeros_like(out)))
    G = mns.grouped_weight_grad(dY, X, off)
    ref.check(G[:3], *[t[:3] for t in ref.weight_grad(dY, X, want, None, 0.0, BF)])
    torch.cuda.synchronize()


def _chain(X, W, dY, off, M):
    Y = mns.grouped_matmul(X, W, off)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    mns.grouped_weight_grad(dY, X, off, C=M, beta=0.5, out=M)
    return Y, dX


def test_captured_and_replayed_with_new_offsets():
    """A captured call reads the offsets and tokens of each replay."""
    n, k, rows = 200, 136, 300
    W = _rand((5, n, k), BF, 1, 0.3)
    X, dY = _rand((rows, k), BF, 2), _rand((rows, n), BF, 3)
    off = _offsets([0, 0, 60, 200, 200, 300])
    M = torch.zeros(5, n, k, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _chain(X, W, dY, off, M)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, dX = _chain(X, W, dY, off, M)
    for i, bounds in enumerate([[0, 10, 10, 250, 300, 300], [0, 300, 300, 300, 300, 300],
                                [0, 0, 60, 200, 200, 300]]):
        off.copy_(_offsets(bounds))
        X.copy_(_rand((rows, k), BF, 20 + i))
        M.copy_(_rand((5, n, k), F32, 30 + i))
        M2 = M.clone()
        Y2, dX2 = _chain(X, W, dY, off, M2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Y2) and torch.equal(dX, dX2) and torch.equal(M, M2), bounds


def test_two_streams_at_once_and_a_given_stream():
    n, k, rows = 320, 264, 500
    W = _rand((4, n, k), BF, 1, 0.3)
    off = _offsets([0, 100, 100, 420, 500])
    Xs = [_rand((rows, k), BF, 5 + i) for i in range(2)]
    alone = [mns.grouped_matmul(x, W, off) for x in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = [[mns.grouped_matmul(x, W, off, stream=s) for _ in range(4)]
           for x, s in zip(Xs, streams)]
    raw = mns.grouped_matmul(Xs[0], W, off, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    for a, outs in zip(alone, got):
        for o in outs:
            assert torch.equal(o, a)
    assert torch.equal(raw, alone[0])


def test_rows_beyond_32_bits_of_bytes():
    """Offsets of rows past 2^32 bytes into the token matrices."""
    k, n, rows = 4096, 64, 600_000
    X = torch.zeros(rows, k, dtype=BF, device="cuda")          # 4.9 GB
    W = _rand((2, n, k), BF, 1, 0.1)
    bounds = [0, rows - 150, rows]
    X[rows - 200:] = _rand((200, k), BF, 2)
    X[:3] = _rand((3, k), BF, 3)
    dY = torch.zeros(rows, n, dtype=BF, device="cuda")
    dY[rows - 200:] = _rand((200, n), BF, 4)
    off = _offsets(bounds)
    pick = torch.cat([torch.arange(3), torch.arange(rows - 200, rows)])
    small = [0, 53, 203]
    Y = mns.grouped_matmul(X, W, off)
    Xp = X[pick.cuda()]
    ref.check(Y[pick.cuda()], *ref.matmul(Xp, W, small, False, torch.zeros(203, n)))
    assert not Y[3:rows - 200].any()
    G = mns.grouped_weight_grad(dY, X, off)
    # adding the products of the all-zero rows is exact, so the bound is the picked rows'
    ref.check(G, *ref.weight_grad(dY[pick.cuda()], Xp, small, None, 0.0, BF), "long reduction")


@pytest.mark.parametrize("sizes", [[40, 0, 100, 61], [129, 3, 90], [33] * 9, [128, 127]])
@pytest.mark.parametrize("n,k", [(192, 512), (520, 128), (64, 1024)])
def test_some_dozens_of_rows(sizes, n, k):
    """Row counts around one tile of 128, reductions of a few k-tiles up to more than the ring holds."""
    bounds = ref.bounds_of(sizes, 2)
    rows, e = bounds[-1] + 3, len(sizes)
    off = _offsets(bounds)
    print("case", sizes, n, k, flush=True)
    W, X = _rand((e, n, k), BF, 1, 0.3), _rand((rows, k), BF, 2)
    Y = mns.grouped_matmul(X, W, off)
    ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), "forward")
    W, dY = _rand((e, k, n), BF, 3, 0.3), _rand((rows, k), BF, 4)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), "input gradient")


@pytest.mark.parametrize("sizes", [[300, 0, 150, 260], [40, 0, 100, 61], [9, 0, 3, 16]])
def test_row_pitches_on_aligned_sizes(sizes):
    """Pitches of whole 16 bytes and widths of whole k-tiles, in groups of many, some dozens and few
    rows: rows of no expert and the gaps between rows keep what they held."""
    n, k, extra = 320, 192, 72
    bounds = ref.bounds_of(sizes, 3)
    rows = bounds[-1] + 5
    X, _ = _strided(_rand((rows, k), BF, 1), k + extra)
    dY, _ = _strided(_rand((rows, n), BF, 2), n + extra)
    W, off = _rand((4, n, k), BF, 3, 0.3), _offsets(bounds)
    for t, src, width in ((False, X, n), (True, dY, k)):
        out, buf = _strided(torch.full((rows, width), 3.0, dtype=BF, device="cuda"), width + extra)
        before = buf.clone()
        want, err = ref.matmul(src, W, bounds, t, out)
        mns.grouped_matmul(src, W, off, transpose_w=t, out=out)
        ref.check(out, want, err, ("pitch", sizes, t))
        touched = torch.zeros_like(buf, dtype=torch.bool)
        touched.as_strided(out.shape, (width + extra, 1))[bounds[0]:bounds[-1]] = True
        assert torch.equal(buf[~touched], before[~touched])
    for out_dtype in (BF, F32):
        G = mns.grouped_weight_grad(dY, X, off, out_dtype=out_dtype)
        ref.check(G, *ref.weight_grad(dY, X, bounds, None, 0.0, out_dtype), ("pitch", sizes))


def test_short_reductions_over_many_tiles():
    """More tiles than blocks, two k-tiles each: a block goes from tile to tile at once."""
    n, k, sizes = 4096, 128, [2600, 5, 1300, 1200]
    bounds = ref.bounds_of(sizes)
    off = _offsets(bounds)
    W, X = _rand((4, n, k), BF, 1, 0.3), _rand((bounds[-1], k), BF, 2)
    Y = mns.grouped_matmul(X, W, off)
    ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), "forward")
    W, dY = _rand((4, k, n), BF, 3, 0.3), _rand((bounds[-1], k), BF, 4)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), "input gradient")


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradients_of_few_rows_over_many_tiles(out_dtype):
    """Experts with no row, one row, one k-tile and a little more, over more tiles than blocks."""
    n, k, sizes = 2048, 2000, [0, 1, 64, 65, 130, 3]
    bounds = ref.bounds_of(sizes, 2)
    off = _offsets(bounds)
    rows = bounds[-1] + 2
    dY, X = _rand((rows, n), BF, 1), _rand((rows, k), BF, 2)
    C = _rand((6, n, k), out_dtype, 3)
    for c, beta in ((None, 0.0), (C, 0.9)):
        G = mns.grouped_weight_grad(dY, X, off, C=c, beta=beta, out_dtype=out_dtype)
        ref.check(G, *ref.weight_grad(dY, X, bounds, c, beta, out_dtype), (out_dtype, beta))


def test_no_rows_but_a_workspace():
    """A batch without rows through the kernel that takes weight gradients of aligned sizes."""
    off = _offsets([0, 0, 0])
    empty = torch.empty(0, 256, dtype=BF, device="cuda")
    G = mns.grouped_weight_grad(empty, empty, off)
    assert G.shape == (2, 256, 256) and not G.any()
    C = _rand((2, 256, 256), F32, 1)
    G = mns.grouped_weight_grad(empty, empty, off, C=C, beta=2.0)
    assert torch.equal(G, 2.0 * C)


@pytest.mark.parametrize("n,k", [(257, 260), (258, 257), (260, 262), (258, 1000), (1, 264)])
@pytest.mark.parametrize("sizes", [[0, 1, 70, 300], [1500], [40, 0, 2]])
def test_weight_gradients_of_widths_inside_an_aligned_pitch(n, k, sizes):
    """Columns of wider, 16-byte aligned rows: the width ends inside a 16-byte piece, an odd one inside
    a dword. Every expert's last row and the last columns count; what lies behind them (NaN) does
    not. [1500] is computed in parts where the widths are even."""
    bounds = ref.bounds_of(sizes, 2)
    rows, e, off = bounds[-1] + 3, len(sizes), _offsets(bounds)
    print("case", n, k, sizes, flush=True)

    def columns(width, seed):
        pitch = (width + 15) // 8 * 8
        buf = torch.full((rows, pitch), float("nan"), dtype=BF, device="cuda")
        buf[:, :width] = _rand((rows, width), BF, seed)
        return buf[:, :width]

    dY, X = columns(n, 1), columns(k, 2)
    for out_dtype in (BF, F32):
        C = _rand((e, n, k), out_dtype, 3)
        for c, beta in ((None, 0.0), (C, 0.5)):
            G = mns.grouped_weight_grad(dY, X, off, C=c, beta=beta, out_dtype=out_dtype)
            ref.check(G, *ref.weight_grad(dY, X, bounds, c, beta, out_dtype), (n, k, sizes, out_dtype))


@pytest.mark.parametrize("transpose_w", [False, True])
def test_overlapping_offsets_take_no_more_rounds(transpose_w):
    """Experts that each claim all rows: unspecified values, but within the output, and not 32 times
    the work of the rows dealt out once (at most one part tile of 256 rows more per expert, which is
    about twice the tiles here)."""
    n, k, rows, e = 2048, 1024, 16384, 64
    W = _rand((e, n, k), BF, 1, 0.3)
    X = _rand((rows, n if transpose_w else k), BF, 2)
    width = k if transpose_w else n
    buf = torch.full((rows + 2, width), 7.0, dtype=BF, device="cuda")
    out = buf[1:-1]

    def time_of(bounds):
        off = _offsets(bounds)
        best = 1e9
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            mns.grouped_matmul(X, W, off, transpose_w=transpose_w, out=out)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    once = time_of([i * rows // e for i in range(e + 1)])
    over = time_of([0, rows] * (e // 2) + [0])
    print("once", once, "overlapping", over, flush=True)
    assert over <= 8 * once
    assert (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()


def _both_ways(sizes, out, red, what):
    bounds = ref.bounds_of(sizes, 1)
    rows, e, off = bounds[-1] + 2, len(sizes), _offsets(bounds)
    print("case", what, sizes, out, red, flush=True)
    W, X = _rand((e, out, red), BF, 1, 0.3), _rand((rows, red), BF, 2)
    Y = mns.grouped_matmul(X, W, off)
    ref.check(Y, *ref.matmul(X, W, bounds, False, torch.zeros_like(Y)), (what, "forward"))
    W, dY = _rand((e, red, out), BF, 3, 0.3), _rand((rows, red), BF, 4)
    dX = mns.grouped_matmul(dY, W, off, transpose_w=True)
    ref.check(dX, *ref.matmul(dY, W, bounds, True, torch.zeros_like(dX)), (what, "input gradient"))


@pytest.mark.parametrize("sizes,out,red", [([2048], 512, 1024), ([1030, 0, 290], 136, 192),
                                           ([300, 301, 299, 400], 2048, 512), ([8192], 64, 1024),
                                           ([8000, 700], 256, 128), ([700], 72, 2048)])
def test_many_rows_of_a_small_grid(sizes, out, red):
    """Many rows per expert whose 256 x 256 tiles would be few: 128 x 64 or 128 x 128 tiles."""
    _both_ways(sizes, out, red, "small grid")


@pytest.mark.parametrize("sizes", [[600, 150, 0, 400], [3000], [1100, 1500]])
def test_longer_reductions_in_parts(sizes):
    """Reductions long enough that few 256 x 256 tiles are computed in parts and joined."""
    _both_ways(sizes, 384, 4096, "parts")


@pytest.mark.parametrize("rows,experts,out,red,kernel", [
    (2048, 1, 512, 1024, "grouped_ring_nt"),        # 16 large tiles, 128 small ones: 23 against 14 us
    (8192, 1, 64, 1024, "grouped_ring_nt"),         # three quarters of a large tile's columns unused
    (2048, 1, 512, 4096, "grouped_256_nt"),         # long enough to be cut: 30 against 37
    (2048, 16, 512, 1024, "grouped_256_nt"),        # large tiles for every block
])
def test_kernel_of_many_rows(rows, experts, out, red, kernel):
    """Many rows go to 256 x 256 tiles only where these occupy the chip."""
    W, X = _rand((experts, out, red), BF, 1), _rand((rows * experts, red), BF, 2)
    off = _offsets([rows * i for i in range(experts + 1)])
    mns.profile_begin()
    mns.grouped_matmul(X, W, off)
    torch.cuda.synchronize()
    assert [k["name"] for k in mns.profile_end()] == [kernel]


# sizes whose forward, input gradient and weight gradient take the 256 x 256 kernel (the forward in
# parts that are joined), and the ring kernel
MODES = {
    "large": ([600, 150, 0, 700], 512, 4096, ["grouped_256_nt", "grouped_256_nn", "grouped_256_tn"]),
    "ring": ([60, 100, 0, 31, 128, 77, 5, 90], 1024, 512,
             ["grouped_ring_nt", "grouped_ring_nn", "grouped_256_tn"]),
}


def _mode(mode, seed=0):
    sizes, n, k, names = MODES[mode]
    bounds = ref.bounds_of(sizes, 3)
    rows, e = bounds[-1] + 4, len(sizes)
    return (_rand((rows, k), BF, seed), _rand((e, n, k), BF, seed + 1, 0.3),
            _rand((rows, n), BF, seed + 2), bounds, names)


def _three(X, W, dY, off):
    return [mns.grouped_matmul(X, W, off), mns.grouped_matmul(dY, W, off, transpose_w=True),
            mns.grouped_weight_grad(dY, X, off)]


@pytest.mark.parametrize("mode", sorted(MODES))
def test_nothing_leaks_through_the_dma_kernels(mode):
    X, W, dY, bounds, names = _mode(mode)
    off = _offsets(bounds)
    mns.profile_begin()
    clean = _three(X, W, dY, off)
    torch.cuda.synchronize()
    assert [k["name"] for k in mns.profile_end()] == names
    rows, bad = X.shape[0], slice(bounds[1], bounds[2])
    for t in (X, dY):
        t[:bounds[0]] = float("nan")
        t[bad] = float("inf")
        t[bounds[-1]:] = float("nan")
    W[1] = float("nan")
    W[2] = float("inf")
    got = _three(X, W, dY, off)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[bad] = False
    for c, g in zip(clean[:2], got[:2]):
        assert torch.equal(g.cpu()[keep], c.cpu()[keep])
        assert not torch.isfinite(g.cpu()[~keep]).any()
    others = [i for i in range(W.shape[0]) if i != 1]
    assert torch.equal(got[2][others], clean[2][others])
    assert not torch.isfinite(got[2][1]).any()


@pytest.mark.parametrize("mode", sorted(MODES))
def test_dma_kernels_captured_and_replayed(mode):
    """Every replay against the eager call: other tokens, other routings (all rows to one expert, none
    to most), eager work and synchronisation in between."""
    X, W, dY, bounds, _ = _mode(mode)
    rows, e = X.shape[0], W.shape[0]
    off = _offsets(bounds)
    M = torch.zeros(W.shape, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _chain(X, W, dY, off, M)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, dX = _chain(X, W, dY, off, M)
    even = [i * rows // e for i in range(e + 1)]
    for i, b in enumerate([even, [0] * e + [rows], [0] + [rows] * e, bounds]):
        off.copy_(_offsets(b))
        X.copy_(_rand(X.shape, BF, 20 + i))
        M.copy_(_rand(M.shape, F32, 30 + i))
        M2 = M.clone()
        Y2, dX2 = _chain(X, W, dY, off, M2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Y2) and torch.equal(dX, dX2) and torch.equal(M, M2), (mode, i)


@pytest.mark.parametrize("mode", sorted(MODES))
def test_dma_kernels_on_two_streams_at_once(mode):
    sets = [_mode(mode, 10 * i)[:4] for i in range(2)]
    sets = [(X, W, dY, _offsets(b)) for X, W, dY, b in sets]
    alone = [_three(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for i, (s, args) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(_three(*args))
    torch.cuda.synchronize()
    for want, rounds in zip(alone, got):
        for outs in rounds:
            for a, b in zip(want, outs):
                assert torch.equal(a, b)
