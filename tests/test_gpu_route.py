"""Routing of tokens to experts on the GPU, and its gradient, against the
definition in 64 bits on the CPU.  Experts have to be the same; weights and
gradients are fp32.

U = 2^-24 is half a step of fp32.  A weight has an exponential (an argument
rounded once, of at most 40 here, and the function's own 4 U: 44 U) in its
numerator and its denominator, with at most 20 additions in turn, and the
quotient and scale: under 120 U of its value."""
import math

import pytest
import torch

from collective_communication_amd import binding as hc
from test_gpu_step_ops import B, F, GUARD, HALF, TINY, U, check_guards, close, gen, guarded

pytestmark = pytest.mark.gpu

NEVER = -math.inf


def scores64(x, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(top > NEVER, top, 0.0))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def choose64(x, k, scores="softmax", bias=None, groups=1, top_groups=1, group_best=1, **_):
    """(tokens, k) experts by plain loops over stable sorts."""
    x = x.double().cpu()
    s = scores64(x, scores)
    c = x if bias is None else torch.where(x > NEVER, s + bias.double().cpu(), NEVER)
    if groups > 1:
        t = x.shape[0]
        value = c if bias is not None or group_best == 1 else torch.where(x > NEVER, s, NEVER)
        value = value.view(t, groups, -1).sort(2, descending=True).values[..., :group_best]
        best = value[..., 0]
        total = torch.where(value > NEVER, value, 0.0).sum(2)
        value = torch.where(best > NEVER, total if group_best == 2 else best, NEVER)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros((t, groups), dtype=torch.bool).scatter_(1, order, True)
        c = torch.where(kept[..., None], c.view(t, groups, -1), NEVER).view_as(c)
    c, e = torch.sort(c, dim=1, descending=True, stable=True)
    return torch.where(c[:, :k] > NEVER, e[:, :k], -1).int()


def weigh64(x, e, scores="softmax", renormalise=True, scale=1.0, **_):
    x = x.double().cpu() if not x.requires_grad else x
    there = e >= 0
    s = torch.where(there, scores64(x, scores).gather(1, e.long().clamp(min=0)), 0.0)
    if renormalise:
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total > 0, total, 1.0)
    return s * scale


def route(x, k, **o):
    t = x.shape[0]
    ebuf = torch.full((t * k + 64,), 77, dtype=torch.int32, device="cuda")
    wbuf, w = guarded((t * k,), F)
    e = ebuf[:t * k].view(t, k)
    hc.hc_route(x, e, w.view(t, k), **o)
    got = e.clone(), w.view(t, k).clone()
    e.fill_(77)
    assert bool((ebuf == 77).all())
    check_guards(wbuf, w)
    return got


def check(x, k, **o):
    e, w = route(x, k, **o)
    want = choose64(x, k, **o)
    assert torch.equal(e.cpu(), want), f"{int((e.cpu() != want).any(1).sum())} tokens differ"
    ww = weigh64(x, want, **o)
    close(w, ww, ww.abs() * 120 * U + TINY[F], "weights")
    return e, w


def logits(g, t, n, dtype, stride=None, offset=0, spread=1.0):
    stride = stride or n
    buf = torch.randn(offset + t * stride, generator=g, device="cuda").mul_(spread).to(dtype)
    return buf[offset:].view(t, stride)[:, :n]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n,k", [(1, 1), (2, 1), (2, 2), (3, 2), (7, 7), (8, 2), (16, 4), (17, 3), (32, 8), (60, 4),
                                 (64, 6), (65, 64), (100, 10), (128, 8), (160, 6), (255, 16), (256, 8), (257, 5),
                                 (384, 8), (512, 2), (640, 12), (1000, 9), (1024, 64)])
def test_top_k(n, k, dtype, scores):
    g = gen(n)
    for t in (1, 3, 130):
        x = logits(g, t, n, dtype, n + 3, 1, 2.0)
        for renormalise in (True, False):
            check(x, k, scores=scores, renormalise=renormalise, scale=1.0 if renormalise else 2.5)
        bias = 0.05 * torch.randn(n, generator=g, device="cuda")
        check(x, k, scores=scores, bias=bias, scale=-0.5)
    # rows that are few different values: many ties, to the lowest expert
    x = torch.randint(-2, 3, (130, n), generator=g, device="cuda").to(dtype)
    check(x, k, scores=scores)
    check(x, k, scores=scores, bias=torch.zeros(n, device="cuda"))


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,top,k", [(8, 2, 1, 2), (12, 4, 2, 3), (64, 8, 3, 6), (64, 64, 5, 5), (160, 8, 3, 6),
                                            (256, 8, 4, 8), (255, 5, 2, 9), (99, 33, 11, 7), (1024, 16, 4, 10),
                                            (1020, 60, 7, 12), (1020, 5, 2, 16), (512, 2, 2, 8), (1023, 3, 1, 4)])
def test_groups(n, groups, top, k, scores, best):
    if n == groups and best == 2:
        best = 1            # one expert a group: its own value either way
    g = gen(n + groups)
    for dtype in (F, B):
        x = logits(g, 200, n, dtype)
        for bias in (None, 0.05 * torch.randn(n, generator=g, device="cuda")):
            check(x, k, scores=scores, bias=bias, groups=groups, top_groups=top, group_best=best)
    x = torch.randint(-1, 2, (100, n), generator=g, device="cuda").float()
    check(x, k, scores=scores, groups=groups, top_groups=top, group_best=best)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_values_next_to_one_another(scores, groups):
    """A bias that brings all values of an expert's row within fp32's rounding of
    one another: only 64 bits tell them apart."""
    g = gen(3)
    for n in (16, 64, 256):
        x = logits(g, 1, n, F).expand(50, n).contiguous()
        s = scores64(x[:1].double().cpu(), scores)[0]
        bias = (0.5 - s).float().cuda()
        assert float((s + bias.double().cpu()).std()) < 1e-7
        check(x, 8, scores=scores, bias=bias, groups=groups, top_groups=max(1, groups // 2), group_best=2)
        # without a bias: logits next to one another
        x = 1.0 + torch.randint(0, 40, (50, n), generator=g, device="cuda") * 2.0 ** -23
        check(x, 8, scores=scores, groups=groups, top_groups=max(1, groups // 2), group_best=1)


def test_masks():
    """Rows without an expert, with fewer than k, groups without one, a bias
    that forbids one; both zeroes as one value."""
    g = gen(11)
    for scores in ("softmax", "sigmoid"):
        for dtype in (F, B):
            x = logits(g, 300, 40, dtype)
            x[torch.rand(x.shape, generator=g, device="cuda") < 0.85] = NEVER
            x[::7] = NEVER
            for o in ({}, {"groups": 8, "top_groups": 3}, {"groups": 8, "top_groups": 3, "group_best": 2}):
                for bias in (None, 0.1 * torch.randn(40, generator=g, device="cuda")):
                    for renormalise in (True, False):
                        e, w = check(x, 6, scores=scores, bias=bias, renormalise=renormalise, **o)
                        assert bool((e[::7] == -1).all()) and bool((w[::7] == 0).all())
            bias = torch.zeros(40, device="cuda")
            bias[::2] = NEVER
            e, _ = check(logits(g, 50, 40, dtype), 20, scores=scores, bias=bias)
            assert bool((e % 2 == 1).all())
    x = torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda")
    assert route(x, 4)[0].tolist() == [[0, 1, 2, 3]]
    lowest = torch.finfo(F).min
    x = torch.full((2, 10), lowest, device="cuda")
    x[1, 3] = 0.0
    e, w = check(x, 2)
    assert e.tolist() == [[0, 1], [3, 0]] and w.tolist() == [[0.5, 0.5], [1.0, 0.0]]


def test_far_logits():
    """Weights of chosen experts that lie far below the row's largest, or far
    below zero: by their distance from one another."""
    x = torch.tensor([[100.0, -50.0, -50.5, -300.0, -301.0, -2000.0]], device="cuda")
    bias = torch.tensor([-10.0, 0.0, 0.0, 1.0, 1.0, 0.0], device="cuda")
    for scores in ("softmax", "sigmoid"):
        e, w = route(x, 2, scores=scores, bias=bias)
        assert e.tolist() == [[3, 4]]
        p = 1.0 / (1.0 + math.exp(-1.0))
        assert abs(float(w[0, 0]) - p) <= 8 * U and abs(float(w[0, 1]) - (1 - p)) <= 8 * U


def test_nan_and_infinity():
    for scores in ("softmax", "sigmoid"):
        x = torch.randn((5, 20), device="cuda")
        x[1, 7] = math.nan
        x[2, 3] = math.inf
        x[3] = math.nan
        for o in ({}, {"bias": torch.zeros(20, device="cuda")}, {"groups": 4, "top_groups": 2, "group_best": 2}):
            e, w = route(x, 4, scores=scores, **o)
            assert bool((e >= 0).all()) and bool((e < 20).all())
            assert all(len(set(row)) == 4 for row in e.tolist())
            assert bool(w[1].isnan().all()) and bool(w[3].isnan().all())
            assert not bool(w[0].isnan().any()) and not bool(w[4].isnan().any())
            if scores == "sigmoid":
                # an infinity's score is 1: its group's two may still be less than two others'
                assert int(e[1, 0]) == 7 and not bool(w[2].isnan().any())
                assert torch.equal(e[2:3].cpu(), choose64(x[2:3], 4, scores=scores, **o))


def grad64(x, e, dw, **o):
    x = x.double().cpu().requires_grad_()
    dw = torch.where(e.cpu() >= 0, dw.double().cpu(), 0.0)
    (weigh64(x, e.cpu(), **o) * dw).sum().backward()
    return torch.where(x.grad.isnan(), 0.0, x.grad)


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,k", [(1, 1), (2, 2), (3, 2), (8, 2), (17, 5), (60, 4), (64, 6), (100, 64), (128, 8),
                                 (129, 3), (256, 8), (300, 10), (512, 16), (513, 2), (1000, 9), (1024, 64)])
def test_gradient(n, k, scores, renormalise):
    g = gen(n + k)
    o = {"scores": scores, "renormalise": renormalise, "scale": 2.5}
    for dtype in (F, B):
        for t in (1, 67):
            x = logits(g, t, n, dtype, n + 3, 1, 1.5)
            e, _ = route(x, k, **o)
            e[t // 2, 0] = -1                                  # a slot of nobody's
            dw = torch.randn((t, k), generator=g, device="cuda")
            buf, dx = guarded((t, n), dtype, n + 5, 1)
            hc.hc_route_grad(x, e, dw, dx, **o)
            want = grad64(x, e, dw, **o)
            s = scores64(x.double().cpu(), scores)
            there = (e.cpu() >= 0)
            p = torch.where(there, s.gather(1, e.cpu().long().clamp(min=0)), 0.0)
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300) if renormalise else p
            # each term is a weight times dw, and the sum of them: 120 U as a weight's, k more for the sum, each twice
            size = (p * dw.double().cpu().abs()).sum(1, keepdim=True) * 2.5
            each = torch.zeros((t, n), dtype=torch.float64).scatter_add_(
                1, e.cpu().long().clamp(min=0), torch.where(there, p * (dw.double().cpu().abs() * 2.5 + size), 0.0))
            if scores == "softmax" and not renormalise:
                each = each + s * size
            # where nothing depends on a logit, 64 bits leave what does not cancel of sums of s * size / p's sum
            left = size / (torch.where(there, s.gather(1, e.cpu().long().clamp(min=0)), 0.0).sum(1, keepdim=True)
                           if renormalise else 1.0) * s * (k + 8) * 2.0 ** -53
            close(dx, want, each * 2 * (130 + k) * U + left + want.abs() * HALF[dtype] + TINY[dtype], f"{t} x {n}")
            check_guards(buf, dx)


def test_gradient_of_a_single_choice():
    """One renormalised weight is its scale, whatever the logits: no gradient at
    all, not even a rounding's."""
    g = gen(25)
    x, dw = logits(g, 500, 87, B, spread=3.0), torch.randn((500, 1), generator=g, device="cuda")
    for scores in ("softmax", "sigmoid"):
        e, w = route(x, 1, scores=scores, scale=2.5)
        assert bool((w == 2.5).all())
        dx = torch.full_like(x, GUARD)
        hc.hc_route_grad(x, e, dw, dx, scores=scores, scale=2.5)
        assert bool((dx == 0).all())


def test_gradient_against_differences():
    g = gen(21)
    x, dw = logits(g, 3, 12, F), torch.randn((3, 4), generator=g, device="cuda")
    for scores in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            o = {"scores": scores, "renormalise": renormalise, "scale": 1.5}
            e, _ = route(x, 4, **o)
            dx = torch.empty_like(x)
            hc.hc_route_grad(x, e, dw, dx, **o)
            for at in ((0, int(e[0, 0])), (1, int(e[1, 3])), (2, 5)):
                d = torch.zeros((3, 12), dtype=torch.float64)
                d[at] = 1e-5
                loss = lambda y: float((weigh64(y, e.cpu(), **o) * dw.double().cpu()).sum())  # noqa: E731
                diff = (loss(x.double().cpu() + d) - loss(x.double().cpu() - d)) / 2e-5
                assert abs(diff - float(dx[at])) <= 1e-5, (scores, renormalise, at)


def test_gradient_of_masked_and_repeated_slots():
    g = gen(23)
    x = logits(g, 20, 30, F)
    x[3] = NEVER
    x[4, 5] = NEVER
    e = torch.randint(0, 30, (20, 5), generator=g, device="cuda", dtype=torch.int32)
    e[3] = -1
    e[4, 0] = 5                      # an expert that cannot have been chosen
    e[5] = 7                         # one expert in every slot
    e[6] = torch.tensor([30, -7, 2 ** 31 - 1, -2 ** 31, 3])
    dw = torch.randn((20, 5), generator=g, device="cuda")
    dw[3] = math.nan                 # of slots that nobody has
    for scores in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            o = {"scores": scores, "renormalise": renormalise}
            dx = torch.empty_like(x)
            hc.hc_route_grad(x, e, dw, dx, **o)
            bad = (e < 0) | (e >= 30)
            bad[4, 0] = True
            known = torch.where(bad, -1, e)
            want = grad64(x, known, torch.where(bad, 0.0, dw), **o)
            close(dx, want, torch.full(want.shape, 60 * U) * float(dw[5:].abs().max()) * 5, (scores, renormalise))
            same = x.clone()
            hc.hc_route_grad(same, e, dw, same, **o)          # over the logits
            assert torch.equal(same, dx)


def test_into_the_sort_and_back():
    """Routing, the sort by expert, the rows there and back: masked tokens have
    no rows, and the weights' gradient comes back through the choice."""
    g = gen(31)
    t, n, k, d = 90, 16, 3, 40
    x = logits(g, t, n, F)
    x[10:20] = NEVER
    plan = hc.ExpertPlan.for_sizes(t, k, n, 4)
    e, w = torch.empty((t, k), dtype=torch.int32, device="cuda"), torch.empty((t, k), device="cuda")
    tok = torch.randn((t, d), generator=g, device="cuda")
    rows = torch.zeros((plan.rows, d), device="cuda")
    y, dy = torch.empty_like(tok), torch.randn((t, d), generator=g, device="cuda")
    drows, dw, dx = torch.empty_like(rows), torch.empty_like(w), torch.empty_like(x)
    hc.hc_route(x, e, w)
    hc.hc_expert_sort(e, plan)
    hc.hc_expert_dispatch(tok, plan, rows)
    hc.hc_expert_combine(rows, plan, w, y)
    hc.hc_expert_combine_grad(dy, rows, plan, w, drows, dw)
    hc.hc_route_grad(x, e, dw, dx)
    assert int(plan.expert_counts.sum()) == (t - 10) * k
    close(y[20:], tok[20:].cpu(), tok[20:].abs().cpu() * 140 * U, "weights sum to 1")
    assert bool((y[10:20] == 0).all()) and bool((dx[10:20] == 0).all()) and bool((dw[10:20] == 0).all())
    # every expert's row is the token: the loss does not depend on the weights' division
    close(dx, torch.zeros_like(dx), (dy * tok).abs().sum(1, keepdim=True).cpu().expand(t, n) * (d + 300) * U, "dlogits")


def test_captured_on_a_stream_and_many_tokens():
    g = gen(41)
    x = logits(g, 20_000, 64, B)
    bias = 0.1 * torch.randn(64, generator=g, device="cuda")
    o = {"scores": "sigmoid", "bias": bias, "groups": 8, "top_groups": 4, "group_best": 2, "scale": 2.5}
    go = {"scores": "sigmoid", "scale": 2.5}
    check(x, 6, **o)
    x = x[:100].clone()
    e, w = torch.empty((100, 6), dtype=torch.int32, device="cuda"), torch.empty((100, 6), device="cuda")
    dw, dx = torch.randn((100, 6), generator=g, device="cuda"), torch.empty_like(x)

    def step(**s):
        hc.hc_route(x, e, w, **o, **s)
        hc.hc_route_grad(x, e, dw, dx, **go, **s)

    step()
    want = (e.clone(), w.clone(), dx.clone())
    side = torch.cuda.Stream()
    for s in ({"stream": side}, {"stream": side.cuda_stream}):
        for o_ in (e, w, dx):
            o_.zero_()
        torch.cuda.synchronize()
        step(**s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((e, w, dx), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(logits(g, 100, 64, B))
        graph.replay()
        torch.cuda.synchronize()
        got = (e.clone(), w.clone(), dx.clone())
        step()
        assert all(torch.equal(a, b) for a, b in zip((e, w, dx), got)), i


def test_offsets_past_32_bits():
    t, n, stride = 3, 20, (1 << 31) + 11
    base = torch.zeros(2 * stride + n, dtype=B, device="cuda")
    x = torch.as_strided(base, (t, n), (stride, 1))
    x.copy_(torch.randn((t, n), device="cuda"))
    e, _ = check(x, 4)
    dw, dx = torch.randn((t, 4), device="cuda"), torch.empty((t, n), dtype=B, device="cuda")
    hc.hc_route_grad(x, e, dw, dx)
    hc.hc_route_grad(x, e, dw, x)
    assert torch.equal(x, dx)


def test_no_tokens():
    x = torch.empty((0, 16), device="cuda")
    hc.hc_route(x, torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda"))
    hc.hc_route_grad(x, torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda"), x)


@pytest.mark.parametrize("lanes,base", [(31, -0.6919994354248047), (31, -0.6913518905639648), (32, -0.6879949569702148),
                                        (33, -0.6879949569702148), (33, -0.692230224609375), (33, -0.6923713684082031)])
def test_values_nearer_than_a_sums_rounding(lanes, base):
    """Softmax scores with a bias, of which two differ by less than what the row's
    sum in fp32 is off by: 31 experts a lane, an exponential just above 1/2 that is
    rounded down, and thirty just below half a step of it, which the sum loses."""
    groups, each = 33, 31
    x = torch.full((groups, each), -17.33)
    x[:, 0] = base
    x[0, 0] = 0.0
    x[lanes:] = NEVER
    x = x.view(1, -1)
    s = scores64(x.double(), "softmax")[0]
    bias = torch.full((groups * each,), NEVER)
    bias[0] = -s[0]
    first = s[0] + bias[0].double()
    # the second value above the first by so many times 2^-24 of the largest score
    for more in (1e-5, 1e-3, 0.3, 1.0, 3.0, 10.0):
        bias[1] = first - s[1] + more * U * s[0]
        assert float(s[1] + bias[1].double()) > float(first)
        for k, want in ((1, [1]), (2, [1, 0])):
            e, _ = check(x.cuda(), k, bias=bias.cuda(), groups=groups, top_groups=groups, renormalise=False)
            assert e.tolist() == [want]
