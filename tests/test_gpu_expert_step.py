"""The example that runs the operators around the exchange together: its
gradients against torch's own differentiation of the same model, its ranks'
weights alike to the bit, and its loss falling."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain_loss(rank, weights, ids, target):
    x = weights["table"][ids] * rank.scale
    top, chosen = (x @ weights["router"]).topk(rank.k, dim=1)
    gate = torch.softmax(top, dim=1)
    y = sum(gate[:, j, None] * torch.stack([x[t] @ weights["up"][e] for t, e in enumerate(chosen[:, j].tolist())])
            for j in range(rank.k))
    return (y - target).square().mean()


def test_gradients_of_a_step():
    import expert_step

    rank = expert_step.Rank(tokens=70, vocab=40, dim=24, experts=5, k=2, align=4, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    ids = torch.randint(0, rank.vocab, (rank.tokens,), generator=g, device="cuda")
    target = torch.randn((rank.tokens, rank.dim), generator=g, device="cuda")
    loss = rank.step(ids, target)
    weights = {n: w.detach().cpu().double().requires_grad_() for n, w in rank.weights.items()}
    want = plain_loss(rank, weights, ids.cpu(), target.cpu().double())
    want.backward()
    want = float(want.detach())
    # sums of at most 70 * 2 * 24 fp32 products through four products in turn
    tol = 4 * 70 * 2 * 24 * 2.0 ** -24
    assert abs(float(loss) - want) <= tol * want
    for name, w in weights.items():
        off = (rank.grads[name].double().cpu() - w.grad).norm() / w.grad.norm()
        assert float(off) <= tol, (name, float(off))


@pytest.mark.parametrize("ranks", [1, 3])
def test_loss_falls_and_ranks_agree(ranks):
    import expert_step

    world, losses = expert_step.train(ranks, 40, say=None)
    assert losses[-1] < 0.9 * losses[0], losses[::8]
    for r in world[1:]:
        assert all(torch.equal(r.weights[n], world[0].weights[n]) for n in r.weights)
