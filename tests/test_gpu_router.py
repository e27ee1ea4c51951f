"""A router's ordered assignments (exactly) and balance loss (element by element, derived bounds) against
plain forms on the CPU."""
import pytest
import torch

import grouped_ref
import layer_ref as ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _ids(tokens, top, experts, seed, kind="uniform"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((tokens, top), experts - 1, dtype=torch.int64)
    ids = torch.randint(0, experts, (tokens, top), generator=g)
    if kind == "holes":
        drop = torch.rand(tokens, top, generator=g) < 0.3
        bad = torch.tensor([-1, experts, 2 ** 40, -(2 ** 40)])
        ids = torch.where(drop, bad[torch.randint(0, 4, (tokens, top), generator=g)], ids)
    if kind == "none":
        ids[:] = -1
    return ids


@pytest.mark.parametrize("kind", ["uniform", "holes", "one", "none"])
@pytest.mark.parametrize("tokens,top,experts", [
    (1, 1, 1), (1, 8, 8), (63, 1, 3), (64, 2, 32), (65, 3, 33), (511, 4, 256), (2048, 1, 7),
    (2049, 1, 2048), (5000, 2, 100), (8193, 1, 2048), (16384, 2, 32), (32769, 1, 513), (70001, 1, 60),
    (140000, 5, 129)])
def test_order(tokens, top, experts, kind):
    ids = _ids(tokens, top, experts, tokens + experts, kind)
    got = mns.expert_order(ids.cuda(), experts)
    for name, g, w in zip(("counts", "offsets", "order"), got, ref.order(ids, experts)):
        assert g.dtype == torch.int64 and torch.equal(g.cpu(), w), name


def test_order_without_places_and_without_assignments():
    ids = _ids(900, 3, 17, 1, "holes")
    counts, offsets, places = mns.expert_order(ids.cuda(), 17, order=False)
    want = ref.order(ids, 17)
    assert places is None and torch.equal(counts.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])
    counts, offsets, places = mns.expert_order(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert counts.tolist() == [0] * 5 and offsets.tolist() == [0] * 6 and places.numel() == 0


def _balance(tokens, top, experts, dtype, kind, scale, seed=0, spread=2.0):
    ids = _ids(tokens, top, experts, seed + 1, kind)
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(tokens, experts, generator=g) * spread).to(dtype).cuda()
    counts, _, _ = mns.expert_order(ids.cuda(), experts, order=False)
    return ids.cuda(), logits, counts


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["uniform", "holes", "one", "none"])
@pytest.mark.parametrize("tokens,top,experts", [
    (1, 1, 1), (5, 2, 3), (64, 2, 32), (33, 4, 33), (200, 70, 64), (77, 8, 128), (61, 2, 130),
    (40, 3, 256), (29, 8, 511), (9, 2, 513), (13, 2, 2048), (3000, 2, 8)])
def test_balance(tokens, top, experts, dtype, kind):
    ids, logits, counts = _balance(tokens, top, experts, dtype, kind, 1.5)
    loss, grad = mns.balance_loss(logits, ids, counts, scale=1.5)
    want, el, wg, eg = ref.balance(logits, ids, counts, 1.5)
    assert abs(loss.item() - want.item()) <= el.item(), (loss.item(), want.item(), el.item())
    assert grad.dtype == dtype
    grouped_ref.check(grad, wg, eg, (tokens, experts))
    again, none = mns.balance_loss(logits, ids, counts, scale=1.5, grad=False)
    assert none is None and torch.equal(again, loss)


def test_balance_pitch_and_in_place():
    ids, logits, counts = _balance(70, 2, 37, F32, "holes", 1.0)
    loss, grad = mns.balance_loss(logits, ids, counts, scale=-0.25)
    buf = torch.full((70, 45), 9.0, device="cuda")
    wide = buf[:, 3:40]
    wide.copy_(logits)
    loss2, grad2 = mns.balance_loss(wide, ids, counts, scale=-0.25, out=wide)
    assert grad2 is wide and torch.equal(wide, grad) and torch.equal(loss, loss2)
    assert (buf[:, :3] == 9).all() and (buf[:, 40:] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_masked_experts_and_tokens(dtype):
    """-inf logits have no probability; a token whose logits are all -inf has none at all; a token
    without an assignment is not looked at; NaN and +inf reach the loss and their own row only."""
    ids, logits, counts = _balance(90, 2, 40, dtype, "uniform", 1.0)
    ids[7] = -1
    logits[:, 5] = float("-inf")
    logits[11] = float("-inf")
    logits[12, 1:] = torch.finfo(dtype).min
    counts, _, _ = mns.expert_order(ids, 40, order=False)
    loss, grad = mns.balance_loss(logits, ids, counts)
    want, el, wg, eg = ref.balance(logits, ids, counts, 1.0)
    assert abs(loss.item() - want.item()) <= el.item()
    grouped_ref.check(grad, wg, eg)
    assert (grad[:, 5] == 0).all() and (grad[11] == 0).all() and (grad[7] == 0).all()
    logits[7] = float("nan")
    loss2, grad2 = mns.balance_loss(logits, ids, counts)
    assert torch.equal(loss2, loss) and torch.equal(grad2, grad)
    for value in (float("nan"), float("inf")):
        bad = logits.clone()
        bad[20, 3] = value
        loss2, grad2 = mns.balance_loss(bad, ids, counts)
        assert loss2.isnan() and grad2[20].isnan().all()
        keep = [i for i in range(90) if i != 20]
        assert torch.equal(grad2[keep], grad[keep])


def test_gradient_against_differences():
    ids, logits, counts = _balance(50, 2, 24, F32, "holes", 1.0, spread=1.0)
    _, grad = mns.balance_loss(logits, ids, counts, scale=3.0)
    x, c = logits.cpu().double(), counts.cpu().double()
    a = ((ids >= 0) & (ids < 24)).sum(1).cpu().double()

    def loss(v):
        return float(3.0 * 24 / c.sum() ** 2 * (a * (torch.softmax(v, 1) * c).sum(1)).sum())

    g = torch.Generator().manual_seed(4)
    for _ in range(4):
        v = torch.randn(50, 24, generator=g, dtype=torch.float64)
        diff = (loss(x + 1e-5 * v) - loss(x - 1e-5 * v)) / 2e-5
        mine = float((grad.cpu().double() * v).sum())
        size = float((grad.cpu().double() * v).abs().sum())
        assert abs(mine - diff) <= 80 * 2.0 ** -23 * size + 1e-8, (mine, diff)


@pytest.mark.parametrize("tokens,experts", [(53, 8), (300, 256), (7, 1)])
def test_equal_counts_leave_no_gradient(tokens, experts):
    """Every token to every expert: c_e - sum_j c_j p_j is 0. c_e - s is exact for s near c_e, off from 0 by
    d <= (E + 8) 2^-23 c (a sum of E terms and a quotient), and what is left of d once sum_j p_j d, off by as much
    relative to it, is taken away is at most c ((E + 8) 2^-23)^2."""
    g = torch.Generator().manual_seed(tokens)
    ids = torch.arange(experts).repeat(tokens, 1).cuda()
    logits = (3 * torch.randn(tokens, experts, generator=g)).cuda()
    counts, _, _ = mns.expert_order(ids, experts)
    loss, grad = mns.balance_loss(logits, ids, counts)
    n = tokens * experts
    assert grad.abs().max().item() <= experts / n ** 2 * experts * tokens * ((experts + 8) * 2.0 ** -23) ** 2
    assert abs(loss.item() - 1.0) <= 2.0 ** -23


def test_captured_replayed_and_on_two_streams():
    ids, logits, counts = _balance(9000, 4, 100, BF, "holes", 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mns.balance_loss(logits, ids, mns.expert_order(ids, 100)[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = mns.expert_order(ids, 100)
        second = mns.balance_loss(logits, ids, first[0])
    for seed in range(3):
        new_ids, new_logits, _ = _balance(9000, 4, 100, BF, "uniform" if seed else "none", 1.0, seed)
        ids.copy_(new_ids)
        logits.copy_(new_logits)
        graph.replay()
        torch.cuda.synchronize()
        want = mns.expert_order(ids, 100)
        want = want + mns.balance_loss(logits, ids, want[0])
        for g, w in zip(first + second, want):
            assert torch.equal(g, w), seed
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            o = mns.expert_order(ids, 100, stream=s)
            outs.append(o + mns.balance_loss(logits, ids, o[0], stream=s))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(g, w) for g, w in zip(o, want))
