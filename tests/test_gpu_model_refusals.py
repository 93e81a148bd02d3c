"""What the binding of the norm of rows, routing and AdamW refuses of device
tensors: wrong shapes, types, layouts and lists, each before anything is written."""
import types

import pytest
import torch

from collective_communication_amd import binding as hc
from test_gpu_step_ops import B, F

pytestmark = pytest.mark.gpu

T, D = 6, 24


def full(shape, dtype=B, value=1.0):
    return torch.full(shape, value, dtype=dtype, device="cuda")


def refused(kind, calls, outs):
    before = [o.clone() for o in outs]
    for i, call in enumerate(calls):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} went through")
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, outs))


def test_norm():
    x, r, w, o, s = full((T, D)), full((T, D)), full((D,), F), full((T, D)), full((T, D))
    u = dict(dtype=torch.uint8, device="cuda")
    q, c = torch.ones((T, D), **u), full((T, 1), F)
    ws = torch.ones(hc.hc_rms_norm_grad_workspace_bytes(T, D), **u)
    dw = full((D,), F)
    wide = full((T, 2 * D))
    norm, norm8, grad = hc.hc_rms_norm, hc.hc_rms_norm_8bit, hc.hc_rms_norm_grad
    refused(ValueError, [
        lambda: norm(x, w[:-1], o), lambda: norm(x, w, o[:-1]), lambda: norm(x, w, o[:, :-1]),
        lambda: norm(x, w, wide[:, ::2]), lambda: norm(x[:, 0].expand(D, T).t(), w, o), lambda: norm(x[0], w, o),
        lambda: norm(x, w, o, residual=r[:-1]), lambda: norm(x, w, o, residual=r[:, 1:]),
        lambda: norm(x, w, o, residual=r, sum_out=s[:, 1:]), lambda: norm(x, w.cpu(), o),
        lambda: norm(x, w, o, residual=r.cpu()),
        lambda: norm8(x, w, q[:, 1:], c), lambda: norm8(x, w, q[:-1], c), lambda: norm8(x, w, q, c, group=-1),
        lambda: norm8(x, w, q, full((T, 2), F)[:, ::2][:-1]), lambda: norm8(x, w, q.cpu(), c),
        lambda: grad(x[:-1], x, w, o), lambda: grad(x, x, w, o[:, 1:]), lambda: grad(x, x, w, o, dw[:-1], ws),
        lambda: grad(x, x, w, o, dw, ws, dsum=r[:-1]), lambda: grad(x, x, w, o, dw, ws.cpu()),
    ], [x, r, o, s, q, c, dw, ws, wide])
    refused(TypeError, [
        lambda: norm(x, w, o.float()), lambda: norm(x, w.half(), o), lambda: norm(x, w, o, residual=r.float()),
        lambda: norm(x, w, o, residual=r, sum_out=s.float()), lambda: norm(x, w, None), lambda: norm(None, w, o),
        lambda: norm8(x, w, o, c), lambda: norm8(x, w, q, full((T, 1))), lambda: grad(x, None, w, o),
        lambda: grad(x, x, w, None), lambda: grad(x.float(), x, w, o),
    ], [x, r, o, s, q, c, dw, ws])
    refused(hc.HcError, [
        lambda: norm(x, w, o, eps=-1.0), lambda: norm(x, w, o, eps=float("nan")), lambda: norm(x, w, o, sum_out=s),
        lambda: norm(x, w, s, residual=r, sum_out=s), lambda: norm8(x, w, q, c, group=48),
        lambda: grad(x, x, w, o, dw), lambda: grad(x, x, w, o, dw, ws[:16]),
        lambda: norm(wide[:, :D], w, wide.view(-1)[:T * D].view(T, D)),
    ], [x, r, o, s, q, c, dw, ws, wide])


def test_route():
    x, e, w = full((T, 16), F), torch.ones((T, 2), dtype=torch.int32, device="cuda"), full((T, 2), F)
    b, d = full((16,), F), full((T, 16), F)
    route, grad = hc.hc_route, hc.hc_route_grad
    refused(ValueError, [
        lambda: route(x, e[:-1], w), lambda: route(x, e, w[:, :1]), lambda: route(x, e.t().contiguous().t(), w),
        lambda: route(x, e, w, bias=b[:-1]), lambda: route(x, e, w.cpu()), lambda: route(x, e, w, bias=b.cpu()),
        lambda: route(x, e[:, 0], w), lambda: route(full((T, 2000), F), e, w), lambda: route(x, e, w, groups=1 << 40),
        lambda: grad(x, e, w, d[:-1]), lambda: grad(x, e, w, d[:, 1:]), lambda: grad(x, e[:-1], w, d),
        lambda: grad(x, e, w[:, :1], d),
    ], [x, e, w, b, d])
    refused(TypeError, [
        lambda: route(x, e.long(), w), lambda: route(x, e, w.bfloat16()), lambda: route(x, e, w, bias=b.bfloat16()),
        lambda: route(x.half(), e, w), lambda: grad(x, e, w, d.bfloat16()), lambda: grad(x, w, w, d),
    ], [x, e, w, b, d])
    refused(hc.HcError, [
        lambda: route(x, e, w, groups=3), lambda: route(x, e, w, groups=4, top_groups=5),
        lambda: route(x, e, w, groups=16, top_groups=1), lambda: route(x, e, w, group_best=3),
        lambda: route(x, e, w, scale=float("inf")), lambda: route(x, e[:, :0], w[:, :0]),
        lambda: grad(x, e, w, d, scale=float("nan")),
    ], [x, e, w, b, d])


def test_adamw():
    p, g, m, v = (full((4, 40), F, x) for x in (1.0, 2.0, 0.0, 0.0))
    codes = lambda: torch.zeros((4, 40), dtype=torch.uint8, device="cuda")  # noqa: E731
    mq, vq, ms, vs = codes(), codes(), full((2,), F, 0.0), full((2,), F, 0.0)
    eight = dict(m_scales=[ms], v_scales=[vs])
    table = torch.zeros(hc.hc_adamw_table_bytes(1), dtype=torch.uint8, device="cuda")
    make = lambda *a, **k: hc.AdamWPlan(*a, **{"table": table, **k})  # noqa: E731
    outs = [p, g, m, v, mq, vq, ms, vs, table]
    refused(ValueError, [
        lambda: make([p], [g[:-1]], [m], [v]), lambda: make([p], [g.t().contiguous().t()], [m], [v]),
        lambda: make([p], [g[:, :1].expand(4, 40)], [m], [v]), lambda: make([p[:, ::2]], [g[:, ::2]], [m], [v]),
        lambda: make([p], [g, g], [m], [v]), lambda: make([p], [g], [], [v]), lambda: make([p], [g.cpu()], [m], [v]),
        lambda: make([p], [g], [mq], [vq], m_scales=[ms]), lambda: make([p], [g], [mq], [vq], m_scales=[ms[:1]], v_scales=[vs]),
        lambda: make([p], [g], [mq], [vq], m_scales=[], v_scales=[]), lambda: make([p], [g], [m], [v], decays=[]),
        lambda: make([p], [g], [m], [v], copies=[]), lambda: make([p], [g], [m], [v], table=table.cpu()),
    ], outs)
    refused(TypeError, [
        lambda: make([p], [g.half()], [m], [v]), lambda: make([p], [g], [mq], [vq]),
        lambda: make([p], [g], [m], [v], **eight), lambda: make([p], [g], [m.bfloat16()], [v]),
        lambda: make([p], [g], [mq], [vq], m_scales=[ms.bfloat16()], v_scales=[vs]),
        lambda: make([p], [g], [m], [v], copies=[p.half()]), lambda: make([p], [None], [m], [v]),
    ], outs)
    refused(hc.HcError, [
        lambda: make([p], [g], [m], [m]), lambda: make([p, p], [g, g], [m, m], [v, v]), lambda: make([p], [p], [m], [v]),
        lambda: make([p], [g], [m], [v], table=table[:16]), lambda: make([p], [g], [m], [v], decays=[float("nan")]),
        lambda: make([p.bfloat16()], [g], [m], [v], copies=[torch.empty_like(p, dtype=B)]),
    ], outs)
    plan = hc.AdamWPlan([p], [g], [m], [v])
    step = lambda *a, **k: hc.hc_adamw(plan, *a, **k)  # noqa: E731
    refused(hc.HcError, [
        lambda: step(0), lambda: step(1, lr=float("nan")), lambda: step(1, betas=(1.0, 0.9)), lambda: step(1, eps=-1.0),
        lambda: step(1, d_norm=ms[:1], max_norm=-1.0), lambda: step(1, grad_scale=float("inf")),
    ], outs)
    refused(TypeError, [
        lambda: step(torch.ones(1, device="cuda")), lambda: step(1, lr=torch.ones(1, device="cuda", dtype=torch.float64)),
        lambda: step("1"), lambda: step(1, d_norm=1.0),
    ], outs)
    refused(ValueError, [
        lambda: step(torch.ones(1, dtype=torch.int64)), lambda: step(1, d_norm=torch.ones(1)),
        lambda: step(torch.ones(0, dtype=torch.int64, device="cuda")),
        lambda: hc.hc_adamw(types.SimpleNamespace(_at=plan._at, table=torch.zeros(16)), 1),
    ], outs)
    refused(OverflowError, [lambda: step(1, seed=-1), lambda: step(1, seed=1 << 64)], outs)


def test_a_step_below_one_and_a_v_past_fp32():
    p, g = full((300,), F), full((300,), F, 0.5)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    hc.hc_adamw(hc.AdamWPlan.for_params([p], [g]), step)
    assert bool(p.isnan().all())
    g[200] = 2.0 ** 70
    for bits in (8, 32):
        p = full((300,), F)
        plan = hc.AdamWPlan.for_params([p], [g], state_bits=bits)
        hc.hc_adamw(plan, 1, weight_decay=0.0)
        other = torch.arange(300, device="cuda") != 200
        assert bool(p[other].isfinite().all()) and bool(p[200].isnan() if bits == 8 else p[200] == 1.0)
        if bits == 8:
            assert bool(plan.v_scales[0][1].isnan()) and bool(plan.v_scales[0][[0, 2]].isfinite().all())
