"""Training steps of a small model with experts on emulated data-parallel
ranks, to show the operators around the gradient exchange together.

Every rank looks its tokens up in the table (hc_embedding), routes each to k
experts (hc_route, hc_expert_sort, hc_expert_dispatch), brings the experts' rows
back with their weights (hc_expert_combine) and learns to predict a vector that
belongs to the token.  With a norm, the experts see the token's row after
hc_rms_norm and their sum is added to it.  The backward pass runs
hc_expert_combine_grad, the experts' products, hc_expert_combine without weights
(the gradient of dispatch), hc_route_grad, hc_rms_norm_grad and
hc_embedding_grad, all into one bucket of gradients per rank.  hc_allreduce
sums the buckets, and every rank takes the same step: hc_clip_grad_norm clips
the sum by its global norm before plain descent, or hc_adamw clips it by
hc_grad_norm's on the way, with states of 32 or 8 bits.

    python examples/expert_step.py --ranks 2 --steps 30
    python examples/expert_step.py --norm --adamw 8
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from collective_communication_amd import binding as hc  # noqa: E402


class Rank:
    """One rank's weights, gradients (views of one bucket) and workspaces."""

    def __init__(self, tokens=512, vocab=1000, dim=64, experts=8, k=2, align=16, seed=0, norm=False, adamw=0):
        self.tokens, self.vocab, self.dim, self.experts, self.k = tokens, vocab, dim, experts, k
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shapes = {"table": (vocab, dim), "router": (dim, experts), "up": (experts, dim, dim)}
        if norm:
            shapes["norm"] = (dim,)
        self.bucket = torch.zeros(sum(math.prod(s) for s in shapes.values()), device="cuda")
        self.weights, self.grads, at = {}, {}, 0
        for name, shape in shapes.items():
            n = math.prod(shape)
            self.weights[name] = torch.randn(shape, generator=g, device="cuda") / math.sqrt(dim)
            self.grads[name] = self.bucket[at:at + n].view(shape)
            at += n
        self.normed, self.adamw = norm, adamw
        if norm:
            self.weights["norm"].fill_(1.0)
        self.scale = math.sqrt(dim)
        self.plan = hc.ExpertPlan.for_sizes(tokens, k, experts, align)
        space = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.sort_ws = space(hc.hc_expert_sort_workspace_bytes(tokens * k, experts))
        self.embed_ws = space(hc.hc_embedding_grad_workspace_bytes(tokens, vocab, dim))
        self.clip_ws = space(hc.hc_grad_norm_workspace_bytes(len(shapes)))
        rows = lambda: torch.zeros((self.plan.rows, dim), device="cuda")  # noqa: E731
        toks = lambda: torch.zeros((tokens, dim), device="cuda")  # noqa: E731
        self.x, self.y, self.dx = toks(), toks(), toks()
        self.xs, self.ys, self.dys, self.dxs = rows(), rows(), rows(), rows()
        self.u, self.du = (toks(), toks()) if norm else (self.x, self.dx)
        self.norm_ws = space(hc.hc_rms_norm_grad_workspace_bytes(tokens, dim))
        self.chosen = torch.zeros((tokens, k), dtype=torch.int32, device="cuda")
        self.gate, self.dweight = torch.zeros((tokens, k), device="cuda"), torch.zeros((tokens, k), device="cuda")
        self.dlogits = torch.zeros((tokens, experts), device="cuda")
        self.norm = torch.zeros(1, device="cuda")
        self.steps = 0
        if adamw:
            # no decay of the norm's weight
            self.states = hc.AdamWPlan.for_params(self.weights.values(), self.grads.values(), state_bits=adamw,
                                                  decays=[float(n != "norm") for n in self.weights])

    def step(self, ids, target):
        """Loss and gradients of one batch; the gradients land in the bucket."""
        w, plan = self.weights, self.plan
        hc.hc_embedding(ids, w["table"], self.x, scale=self.scale)
        if self.normed:
            hc.hc_rms_norm(self.x, w["norm"], self.u)
        logits, chosen, gate = self.u @ w["router"], self.chosen, self.gate
        hc.hc_route(logits, chosen, gate)
        hc.hc_expert_sort(chosen, plan, self.sort_ws)
        hc.hc_expert_dispatch(self.u, plan, self.xs)
        ends = plan.expert_offsets.tolist()
        for e in range(self.experts):
            a, b = ends[e], ends[e + 1]
            torch.mm(self.xs[a:b], w["up"][e], out=self.ys[a:b])
        hc.hc_expert_combine(self.ys, plan, gate, self.y)

        off = self.x + self.y - target if self.normed else self.y - target
        loss = off.square().mean()
        dy = off * (2.0 / off.numel())
        hc.hc_expert_combine_grad(dy, self.ys, plan, gate, self.dys, self.dweight)
        for e in range(self.experts):
            a, b = ends[e], ends[e + 1]
            torch.mm(self.xs[a:b].t(), self.dys[a:b], out=self.grads["up"][e])
            torch.mm(self.dys[a:b], w["up"][e].t(), out=self.dxs[a:b])
        hc.hc_expert_combine(self.dxs, plan, None, self.du)
        hc.hc_route_grad(logits, chosen, self.dweight, self.dlogits)
        torch.mm(self.u.t(), self.dlogits, out=self.grads["router"])
        self.du.addmm_(self.dlogits, w["router"].t())
        if self.normed:
            hc.hc_rms_norm_grad(self.du, self.x, w["norm"], self.dx, self.grads["norm"], self.norm_ws, dsum=dy)
        hc.hc_embedding_grad(ids, self.dx, self.grads["table"], self.embed_ws, scale=self.scale)
        return loss

    def update(self, ranks, lr, max_norm):
        """Clips the summed gradients by the norm of their mean and steps."""
        if self.adamw:
            self.steps += 1
            hc.hc_grad_norm(list(self.grads.values()), self.norm, self.clip_ws)
            hc.hc_adamw(self.states, self.steps, lr=lr, grad_scale=1.0 / ranks, d_norm=self.norm, max_norm=max_norm,
                        seed=self.steps if self.adamw == 8 else 0)
            return
        hc.hc_clip_grad_norm(list(self.grads.values()), max_norm * ranks, self.norm, self.clip_ws)
        for name, weight in self.weights.items():
            weight.add_(self.grads[name], alpha=-lr / ranks)


def train(ranks=2, steps=30, lr=None, max_norm=0.05, seed=0, say=print, **sizes):
    """Trains and returns the ranks and the losses (of all ranks' tokens)."""
    if lr is None:
        lr = 0.01 if sizes.get("adamw") else 20.0
    world = [Rank(seed=seed, **sizes) for _ in range(ranks)]
    one = world[0]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    answers = torch.randn((one.vocab, one.dim), generator=g, device="cuda")
    losses = []
    for step in range(steps):
        total = torch.zeros((), device="cuda")
        for rank in world:
            ids = torch.randint(0, one.vocab, (one.tokens,), generator=g, device="cuda")
            total += rank.step(ids, answers[ids])
        hc.hc_allreduce([r.bucket for r in world], [r.bucket for r in world])
        for rank in world:
            rank.update(ranks, lr, max_norm)
        losses.append(float(total) / ranks)
        if say and (step % 10 == 0 or step == steps - 1):
            say(f"step {step:4d}  loss {losses[-1]:.5f}  gradient norm {float(one.norm) / ranks:.5f}")
    return world, losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--norm", action="store_true", help="the experts see normed rows, added to the token's")
    ap.add_argument("--adamw", type=int, choices=(0, 8, 32), default=0, help="AdamW with states of so many bits")
    a = ap.parse_args()
    world, losses = train(a.ranks, a.steps, norm=a.norm, adamw=a.adamw)
    for r in world[1:]:
        assert all(torch.equal(r.weights[n], world[0].weights[n]) for n in r.weights), "ranks differ"
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}; all {len(world)} ranks hold the same weights")


if __name__ == "__main__":
    main()
