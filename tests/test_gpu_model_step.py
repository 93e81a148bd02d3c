"""The norm of rows, routing and the AdamW step together with the operators they
stand beside: the example with a norm against torch's own differentiation, its
ranks alike to the bit whatever the optimizer, and rows of 8 bits sent to their
experts."""
import os
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from collective_communication_amd import binding as hc
from test_gpu_step_ops import B, U, close, gen, space

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain_loss(rank, weights, ids, target):
    x = weights["table"][ids] * rank.scale
    u = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * weights["norm"]
    top, chosen = (u @ weights["router"]).topk(rank.k, dim=1)
    gate = torch.softmax(top, dim=1)
    y = sum(gate[:, j, None] * torch.stack([u[t] @ weights["up"][e] for t, e in enumerate(chosen[:, j].tolist())])
            for j in range(rank.k))
    return (x + y - target).square().mean()


def test_gradients_of_a_step_with_a_norm():
    import expert_step

    rank = expert_step.Rank(tokens=70, vocab=40, dim=24, experts=5, k=2, align=4, seed=3, norm=True)
    g = gen(4)
    rank.weights["norm"].copy_(1.0 + 0.2 * torch.randn(24, generator=g, device="cuda"))
    ids = torch.randint(0, rank.vocab, (rank.tokens,), generator=g, device="cuda")
    target = torch.randn((rank.tokens, rank.dim), generator=g, device="cuda")
    loss = rank.step(ids, target)
    weights = {n: w.detach().cpu().double().requires_grad_() for n, w in rank.weights.items()}
    want = plain_loss(rank, weights, ids.cpu(), target.cpu().double())
    want.backward()
    want = float(want.detach())
    # sums of at most 70 * 2 * 24 fp32 products through five products in turn
    tol = 5 * 70 * 2 * 24 * 2.0 ** -24
    assert abs(float(loss) - want) <= tol * want
    for name, w in weights.items():
        off = (rank.grads[name].double().cpu() - w.grad).norm() / w.grad.norm()
        assert float(off) <= tol, (name, float(off))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("adamw", [0, 8, 32])
def test_ranks_agree(adamw, norm):
    import expert_step

    world, losses = expert_step.train(2, 5, say=None, adamw=adamw, norm=norm)
    assert all(torch.isfinite(torch.tensor(losses)))
    first = expert_step.Rank(adamw=adamw, norm=norm)
    for r in world:
        for n, w in r.weights.items():
            assert torch.equal(w, world[0].weights[n])
            assert not torch.equal(w, first.weights[n]), f"{n} did not move"


def test_one_adamw_step_of_the_example():
    """The example's update is the formula on the ranks' mean gradient."""
    import expert_step

    rank = expert_step.Rank(adamw=32)
    g = gen(1)
    rank.bucket.copy_(torch.randn(rank.bucket.shape, generator=g, device="cuda"))
    before = {n: w.double().cpu() for n, w in rank.weights.items()}
    mean = {n: x.double().cpu() / 3 for n, x in rank.grads.items()}
    norm = torch.cat([m.reshape(-1) for m in mean.values()]).norm()
    rank.update(3, 0.01, 0.5)
    for n, w in rank.weights.items():
        d = mean[n] * min(1.0, 0.5 / (float(norm) + 1e-6))
        # from zero states the step is lr * g / (|g| + eps)
        want = before[n] * (1 - 0.01 * 0.01) - 0.01 * d / (d.abs() + 1e-8)
        # 24 U of the quotient, and the clipped gradients' own 7 U near eps
        close(w, want, want.abs() * 4 * U + 0.01 * 40 * U, n)


def test_rows_of_8_bits_to_their_experts():
    """Norm to 8 bits with scales, route, sort, and the bytes and scales sent by
    the same plan: each expert's rows are the tokens', bit for bit."""
    g = gen(2)
    t, d, n, k = 300, 1024, 16, 4
    x, res = torch.randn((t, d), generator=g, device="cuda").bfloat16(), torch.randn((t, d), generator=g, device="cuda").bfloat16()
    w = torch.randn(d, generator=g, device="cuda").bfloat16()
    h, q = torch.empty_like(x), torch.empty((t, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((t, d // 128), device="cuda")
    hc.hc_rms_norm_8bit(x, w, q, scales, group=128, residual=res, sum_out=h)
    plan = hc.ExpertPlan.for_sizes(t, k, n, 16)
    experts, weights = torch.empty((t, k), dtype=torch.int32, device="cuda"), torch.empty((t, k), device="cuda")
    hc.hc_route(torch.randn((t, n), generator=g, device="cuda"), experts, weights, scores="sigmoid", scale=2.5)
    hc.hc_expert_sort(experts, plan, space(hc.hc_expert_sort_workspace_bytes(t * k, n)))
    rows = torch.full((plan.rows, d), 0x55, dtype=torch.uint8, device="cuda")
    row_scales = torch.full((plan.rows, d // 128), -1.0, device="cuda")
    hc.hc_expert_dispatch(q.view(torch.bfloat16), plan, rows.view(torch.bfloat16))
    hc.hc_expert_dispatch(scales, plan, row_scales)
    at = plan.row_of_slot.view(t, k).long()
    assert bool((at >= 0).all())
    for j in range(k):
        assert torch.equal(rows[at[:, j]], q.view(torch.uint8))
        assert torch.equal(row_scales[at[:, j]], scales)
    # and they stand for the norm's own rows, to half a step of a code
    y = torch.empty_like(x)
    hc.hc_rms_norm(h, w, y)
    value = q.float() * scales.repeat_interleave(128, 1)
    step = scales.repeat_interleave(128, 1) * 2.0 ** -10
    close(value, y.float(), (y.float().abs() * (2.0 ** -4 + 2.0 ** -7) + step * 1.01).cpu(), "rows")


def test_a_captured_step():
    """Norm, routing, sort, dispatch, back and the optimizer as one graph, replayed
    with other tokens, against the same calls one by one."""
    g = gen(6)
    t, d, n, k = 200, 256, 8, 2

    class Side:
        def __init__(self):
            h = gen(7)
            self.w = torch.ones(d, device="cuda")
            self.x, self.u = torch.zeros((t, d), device="cuda"), torch.zeros((t, d), device="cuda")
            self.logits = torch.zeros((t, n), device="cuda")
            self.e, self.c = torch.zeros((t, k), dtype=torch.int32, device="cuda"), torch.zeros((t, k), device="cuda")
            self.plan = hc.ExpertPlan.for_sizes(t, k, n, 4)
            self.rows, self.y = torch.zeros((self.plan.rows, d), device="cuda"), torch.zeros((t, d), device="cuda")
            self.dx, self.dw = torch.zeros((t, d), device="cuda"), torch.zeros(d, device="cuda")
            self.drows, self.dc, self.dl = torch.zeros_like(self.rows), torch.zeros_like(self.c), torch.zeros_like(self.logits)
            self.router = torch.randn((d, n), generator=h, device="cuda")
            self.norm, self.lr = torch.zeros(1, device="cuda"), torch.full((1,), 0.01, device="cuda")
            self.at = torch.ones(1, dtype=torch.int64, device="cuda")
            self.ws = space(hc.hc_rms_norm_grad_workspace_bytes(t, d))
            self.nws = space(hc.hc_grad_norm_workspace_bytes(1))
            self.opt = hc.AdamWPlan.for_params([self.w], [self.dw], state_bits=8)

        def step(self):
            hc.hc_rms_norm(self.x, self.w, self.u)
            hc.hc_route(self.logits, self.e, self.c)
            hc.hc_expert_sort(self.e, self.plan)
            hc.hc_expert_dispatch(self.u, self.plan, self.rows)
            hc.hc_expert_combine(self.rows, self.plan, self.c, self.y)
            hc.hc_expert_combine_grad(self.y, self.rows, self.plan, self.c, self.drows, self.dc)
            hc.hc_route_grad(self.logits, self.e, self.dc, self.dl)
            hc.hc_rms_norm_grad(self.y, self.x, self.w, self.dx, self.dw, self.ws)
            hc.hc_grad_norm([self.dw], self.norm, self.nws)
            hc.hc_adamw(self.opt, self.at, lr=self.lr, d_norm=self.norm, max_norm=1.0, seed=5)
            self.at.add_(1)

        def all(self):
            return (self.u, self.e, self.c, self.y, self.dl, self.dx, self.dw, self.w, self.norm,
                    self.opt.exp_avgs[0].view(torch.uint8), self.opt.m_scales[0])

    a, b = Side(), Side()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for i in range(4):
        x, logits = torch.randn((t, d), generator=g, device="cuda"), torch.randn((t, n), generator=g, device="cuda")
        for s in (a, b):
            s.x.copy_(x)
            s.logits.copy_(logits)
        graph.replay()
        torch.cuda.synchronize()
        b.step()
        assert all(torch.equal(p, q) for p, q in zip(a.all(), b.all())), i


def test_two_threads_at_once():
    """Two host threads, a stream, tensors and a plan each, in calls of all the
    operators at once: what each computes alone."""
    t, d, n, k = 300, 512, 48, 4

    def work(seed, stream):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, res = (torch.randn((t, d), generator=g, device="cuda").to(B) for _ in range(2))
        w, logits = torch.randn(d, generator=g, device="cuda"), torch.randn((t, n), generator=g, device="cuda")
        p = torch.randn(5000, generator=g, device="cuda").to(B)
        out, s, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        ws = torch.empty(hc.hc_rms_norm_grad_workspace_bytes(t, d), dtype=torch.uint8, device="cuda")
        e = torch.empty((t, k), dtype=torch.int32, device="cuda")
        c, dl = torch.empty((t, k), device="cuda"), torch.empty_like(logits)
        plan = hc.AdamWPlan.for_params([p], [torch.randn(5000, generator=g, device="cuda")], state_bits=8)
        torch.cuda.synchronize()
        for i in range(30):
            hc.hc_rms_norm(x, w, out, residual=res, sum_out=s, stream=stream)
            hc.hc_rms_norm_grad(out, s, w, dx, dw, ws, dsum=res, stream=stream)
            hc.hc_route(logits, e, c, scores="sigmoid", bias=w[:n], groups=4, top_groups=2, group_best=2, stream=stream)
            hc.hc_route_grad(logits, e, c, dl, scores="sigmoid", stream=stream)
            hc.hc_adamw(plan, i + 1, seed=seed, stream=stream)
            with pytest.raises(hc.HcError, match="step 0" if seed == 1 else "eps"):
                hc.hc_adamw(plan, 0) if seed == 1 else hc.hc_adamw(plan, 1, eps=-1.0)
        stream.synchronize()
        return [out, s, dx, dw, e, c, dl, p]

    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [work(i + 1, streams[i]) for i in range(2)]
    with ThreadPoolExecutor(2) as pool:
        got = list(pool.map(work, (1, 2), streams))
    assert all(torch.equal(a, b) for i in range(2) for a, b in zip(got[i], want[i]))
