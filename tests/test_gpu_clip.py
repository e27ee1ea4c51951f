"""The global norm and clipping of gradients against float64 on the CPU."""
import math

import pytest
import torch

import grouped_ref
import layer_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# the norm: sums of exact squares in float64 (2^-52 each way, n of them), one rounding to float32
NORM = 2.0 ** -24 + 1e-10


def _grads(shapes, seed=0, scale=1.0, dtypes=(BF, F32)):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda()
            for i, s in enumerate(shapes)]


LISTS = {
    "one_element": [(1,)],
    "one_piece": [(4096,)],
    "around_a_piece": [(4095,), (4097,), (8191,), (8193,), (8192,)],
    "mixed": [(256, 1024), (1024,), (333, 17), (257,), (1,), (0,), (3, 5, 7), ()],
    "large": [(2048, 2048), (1111, 3001), (5,)],
    "many": [((i * 131) % 5000 + 1,) for i in range(300)],
}


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_norm_and_clip(name, max_norm):
    grads = _grads(LISTS[name])
    norm, factor = ref.clip(grads, max_norm, 1e-6)
    assert abs(mns.grad_norm(grads).item() - norm) <= NORM * norm
    out = [torch.full_like(g, 3.0) for g in grads]
    got = mns.clip_grad_norm(grads, max_norm, out=out)
    assert got.dtype == F32 and got.dim() == 0 and abs(got.item() - norm) <= NORM * norm
    for i, (g, o) in enumerate(zip(grads, out)):
        grouped_ref.check(o, *ref.clipped(g, factor), (name, i))
    before = [g.clone() for g in grads]
    again = mns.clip_grad_norm(grads, max_norm)
    assert torch.equal(again, got)
    for g, o, b in zip(grads, out, before):
        assert torch.equal(g, o)
        if factor == 1.0:
            assert torch.equal(g, b)


@pytest.mark.parametrize("scale", [1e-24, 1e24, 1e-38])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_range(scale, dtype):
    """Squares beyond float32's range either way."""
    grads = _grads([(300, 100), (77,)], 3, scale, (dtype,))
    norm, factor = ref.clip(grads, scale, 0.0)
    got = mns.clip_grad_norm(grads, scale, eps=0.0, out=[torch.empty_like(g) for g in grads])
    assert abs(got.item() - norm) <= NORM * norm + 2.0 ** -149
    out = [torch.empty_like(g) for g in grads]
    mns.clip_grad_norm(grads, scale, eps=0.0, out=out)
    for g, o in zip(grads, out):
        want, err = ref.clipped(g, factor)
        # results below the normal numbers: half of the smallest step, or flushed whole
        small = 2.0 ** -126
        grouped_ref.check(o, want, err + small * (want.abs() < 2 * small), scale)


def test_zero_gradients_and_limits():
    zero = [torch.zeros(100, device="cuda"), torch.zeros(3, 3, dtype=BF, device="cuda")]
    assert mns.clip_grad_norm(zero, 1.0).item() == 0 and (zero[0] == 0).all()
    assert mns.clip_grad_norm(zero, 0.0, eps=0.0).item() == 0 and (zero[0] == 0).all()
    empty = [torch.empty(0, device="cuda")]
    assert mns.grad_norm(empty).item() == 0 and mns.clip_grad_norm(empty, 1.0).item() == 0
    g = _grads([(50,)])
    assert mns.clip_grad_norm(g, 0.0).item() > 0 and (g[0] == 0).all()
    g = _grads([(50,)])
    b = g[0].clone()
    mns.clip_grad_norm(g[0], float("inf"))
    assert torch.equal(g[0], b)


def test_nan_and_infinity():
    grads = _grads([(5000,), (70, 3)])
    grads[1][2, 1] = float("nan")
    assert mns.clip_grad_norm(grads, 1.0).isnan() and all(g.isnan().all() for g in grads)
    grads = _grads([(5000,), (70, 3)])
    grads[0][4321] = float("inf")
    assert mns.clip_grad_norm(grads, 1.0).item() == float("inf")
    assert grads[0][4321].isnan() and (grads[1] == 0).all() and (grads[0][:4000] == 0).all()


def test_no_limit_keeps_infinite_gradients():
    g = [torch.randn(300, device="cuda"), torch.randn(5, 7, device="cuda").bfloat16()]
    g[0][17] = float("inf")
    want, out = [t.clone() for t in g], [torch.empty_like(t) for t in g]
    assert mns.clip_grad_norm(g, float("inf"), out=out).item() == float("inf")
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_unaligned_pieces_and_neighbours():
    """Gradients that are slices of one buffer, at odd addresses: what lies between stays."""
    for dtype in (BF, F32):
        buf = _grads([(60000,)], 5, 1.0, (dtype,))[0]
        spans = [(1, 9000), (9003, 9004), (9011, 30000), (30000, 45001)]
        grads = [buf[a:b] for a, b in spans]
        before = buf.clone()
        norm, factor = ref.clip(grads, 2.0, 1e-6)
        mns.clip_grad_norm(grads, 2.0)
        at = 0
        for a, b in spans:
            assert torch.equal(buf[at:a], before[at:a])
            grouped_ref.check(buf[a:b], *ref.clipped(before[a:b], factor), (a, b))
            at = b
        assert torch.equal(buf[at:], before[at:])


def test_the_same_tensor_twice():
    g = _grads([(777,)])[0]
    norm = ref.clip([g, g], 1.0, 0.0)[0]
    assert abs(mns.grad_norm([g, g]).item() - norm) <= NORM * norm
    for grads, out in (([g, g], None), ([g, g[:5]], None), ([g[1:], g[:-1]], None),
                       ([g[:10], g[20:30]], [g[20:30], g[:10]]), ([g[:-1]], [g[1:]])):
        with pytest.raises(mns.MnsError):
            mns.clip_grad_norm(grads, 1.0, out=out)
    o = [torch.empty_like(g), torch.empty_like(g)]          # read twice, written apart
    mns.clip_grad_norm([g, g], 1.0, out=o)
    assert torch.equal(o[0], o[1])


@pytest.mark.parametrize("dtype,lead", [(BF, 1), (BF, 0), (F32, 3)])
def test_lists_beyond_the_caches(dtype, lead):
    """More than 256 MB, which is read and written past the caches, at odd addresses too."""
    n = 150_000_001 if dtype == BF else 80_000_001
    buf = torch.empty(n + 8, dtype=dtype, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    grads = [buf[lead:lead + n - 5000], buf[lead + n - 4999:lead + n]]
    norm = math.sqrt(sum(float((p.double() ** 2).sum()) for g in grads for p in g.split(1 << 24)))
    factor = min(1.0, 3.0 / (norm + 1e-6))
    out = [torch.empty_like(g) for g in grads]
    got = mns.clip_grad_norm(grads, 3.0, out=out)
    assert abs(got.item() - norm) <= NORM * norm
    for g, o in zip(grads, out):
        for a, b in zip(g.split(1 << 24), o.split(1 << 24)):
            want = a.double() * factor
            bound = want.abs() * (2.0 ** -23 + grouped_ref.HALF_STEP[dtype] * (1 + 2.0 ** -23)) + 1e-38
            assert ((b.double() - want).abs() <= bound).all()
    between = buf[lead + n - 5000].clone()
    mns.clip_grad_norm(grads, 3.0)
    assert all(torch.equal(g, o) for g, o in zip(grads, out)) and buf[lead + n - 5000] == between


def test_captured_replayed_and_on_two_streams():
    grads = _grads([(700, 300), (41,), (9000,)])
    out = [torch.empty_like(g) for g in grads]
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mns.clip_grad_norm(grads, 1.0, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mns.clip_grad_norm(grads, 1.0, out=out, workspace=ws)
    for seed in range(3):
        for g, n in zip(grads, _grads([(700, 300), (41,), (9000,)], seed + 5, 10.0 ** seed)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        mine = [torch.empty_like(g) for g in grads]
        assert torch.equal(mns.clip_grad_norm(grads, 1.0, out=mine), norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(g) for g in grads] for _ in range(8)]
    torch.cuda.synchronize()
    norms = [mns.clip_grad_norm(grads, 1.0, out=o, stream=streams[i % 2]) for i, o in enumerate(outs)]
    torch.cuda.synchronize()
    assert all(torch.equal(n, norm) for n in norms)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, mine))
