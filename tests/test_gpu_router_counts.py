"""Counts: the balance loss where an expert has more assignments than float32 counts one by one (2^24), and the
order where a wave's steps find the place that the step before left."""
import pytest
import torch

import grouped_ref
import layer_ref
import muon_newton_schulz_amd as mns

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -23


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_counts_beyond_float32(dtype):
    """Two experts of 2^24 + 1 and 2^24 + 4 assignments: c_e - s is +-3 times the other's probability. With what the
    counts exceed the least one by, 0 and 3, a row's s is off by at most (10 + 2 |x - max|) 2^-23 of 3 and the
    gradient by twice that, by as much of itself, and by its factor's roundings."""
    c0, c1 = (1 << 24) + 1, (1 << 24) + 4
    tokens = c0 + c1
    ids = torch.zeros(tokens, 1, dtype=torch.int64, device="cuda")
    ids[c0:] = 1
    logits = torch.empty(tokens, 2, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    logits = logits.to(dtype)
    counts, offsets, order = mns.expert_order(ids, 2)
    assert counts.tolist() == [c0, c1] and offsets.tolist() == [0, c0, tokens]
    assert torch.equal(order, torch.arange(tokens, device="cuda"))
    loss, grad = mns.balance_loss(logits, ids, counts, scale=float(tokens) * 1000)
    factor = 1000.0 * 2 / tokens
    total = 0.0
    for part, got in zip(logits.split(1 << 22), grad.split(1 << 22)):
        x = part.double()
        p = torch.softmax(x, 1)
        far = (x[:, 0] - x[:, 1]).abs()[:, None]
        diff = p.flip(1) * torch.tensor([float(c0 - c1), float(c1 - c0)], dtype=torch.float64, device="cuda")
        want = factor * p * diff
        err = factor * p * (2 * 3 * (10 + 2 * far) * ULP + diff.abs() * (16 + 2 * far) * ULP)
        over = ((got.double() - want).abs() - grouped_ref.stored(want, err, dtype)).max().item()
        assert over <= 0, over
        total += float((p[:, 0] * c0 + p[:, 1] * c1).sum())
    want = factor * total
    assert abs(loss.item() - want) <= 2.0 ** -23 * want


@pytest.mark.parametrize("experts", [3, 512, 513, 2048])
@pytest.mark.parametrize("run", [1, 2, 63, 64, 65, 200])
def test_order_of_runs(run, experts):
    """Runs of one expert, and of two in turn, across a wave's steps of 64: every step's first place is the one that
    another lane of the wave wrote a step before."""
    m = 20011
    i = torch.arange(m)
    for ids in ((i // run) % experts, ((i // run) + (i & 1)) % experts, (i // run) % (experts + 1) - 1):
        got = mns.expert_order(ids.cuda(), experts)
        for name, g, w in zip(("counts", "offsets", "order"), got, layer_ref.order(ids, experts)):
            assert torch.equal(g.cpu(), w), (name, run, experts)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts", [(300, 4), (5000, 100)])
def test_loss_of_probabilities_on_unassigned_experts(tokens, experts, dtype):
    """Every token's probability lies on an expert without assignments, all but e^-20 of it: the loss is what is left,
    and as exact as any (layer_ref's bound is relative to sum_e c_e p_te)."""
    g = torch.Generator().manual_seed(experts)
    logits = torch.randn(tokens, experts, generator=g)
    logits[:, 0] = 20
    logits = logits.to(dtype).cuda()
    ids = torch.randint(1, experts, (tokens, 2), generator=g).cuda()
    counts, _, _ = mns.expert_order(ids, experts)
    loss, grad = mns.balance_loss(logits, ids, counts)
    want, el, wg, eg = layer_ref.balance(logits, ids, counts, 1.0)
    assert abs(loss.item() - want.item()) <= el.item(), (loss.item(), want.item(), el.item())
    grouped_ref.check(grad, wg, eg, (tokens, experts))
