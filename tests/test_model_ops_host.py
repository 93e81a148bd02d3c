"""Host-side checks of the norm of rows, routing and the AdamW step (no GPU
needed): sizes, and every refusal of the C ABI and of the binding.  No call here
reaches a launch (in a process without a GPU that would be HC_ERR_DEVICE)."""
import ctypes
import math

import pytest
import torch

from test_step_ops_host import P, Q, W, hc, ptrs, sizes, types  # noqa: F401

NAN, INF = math.nan, math.inf


# ------------------------------------------------------------------ norm of rows

def test_norm_refusals(hc):  # noqa: F811
    L, E = hc.load(), hc.HC_ERR_INVALID_ARGUMENT
    ok = dict(x=P, dt=1, n=4, d=64, xs=64, r=Q, rs=64, w=W, wt=0, eps=1e-6, s=P + 4096, ss=64, o=P + 8192, os=64)

    def call(**k):
        a = list({**ok, **k}.values())
        return L.hc_rms_norm(*a, None)

    for bad in (dict(x=None), dict(x=P + 1), dict(dt=2), dict(dt=-1), dict(n=1 << 31), dict(d=0), dict(d=32769),
                dict(xs=63), dict(xs=1 << 41), dict(r=Q + 1), dict(rs=63), dict(w=None), dict(w=W + 2), dict(wt=7),
                dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(s=P + 4097), dict(ss=1), dict(o=None),
                dict(o=P + 8193), dict(os=63), dict(r=None), dict(s=P + 8192),
                dict(o=P, os=65), dict(o=Q, rs=65), dict(s=P, ss=72), dict(s=Q, ss=72)):
        assert call(**bad) == E, bad
    assert call(r=None) == E and b"residual" in L.hc_last_error()
    assert call(n=0, x=None, r=None, s=None, o=None) == 0

    def call8(group=128, scales=W + 4096, cs=1, **k):
        a = list({**ok, **k}.values())
        return L.hc_rms_norm_8bit(*a, group, scales, cs, None)

    for bad in (dict(x=None), dict(eps=NAN), dict(o=None), dict(os=63), dict(os=1 << 41), dict(group=1), dict(group=-1),
                dict(group=96), dict(group=512), dict(scales=None), dict(scales=W + 2), dict(cs=0),
                dict(group=32), dict(d=32769), dict(o=P), dict(o=Q), dict(o=P + 4096)):
        assert call8(**bad) == E, bad
    assert call8(n=0, x=None, r=None, s=None, o=None, scales=None) == 0


def test_norm_gradient_refusals_and_workspace(hc):  # noqa: F811
    L, E, C = hc.load(), hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    f = hc.hc_rms_norm_grad_workspace_bytes
    assert f(1 << 31, 64) == 0 and f(4, 0) == 0 and f(4, 32769) == 0 and f(0, 64) == 0
    tokens = [1, 2, 1023, 1024, 1025, 5000, 1 << 20]
    for d in (1, 7, 64, 4096, 32768):
        v = [f(t, d) for t in tokens]
        assert v == sorted(v) and v[0] >= 4 * d
    for t in tokens:
        v = [f(t, d) for d in (1, 7, 64, 65, 4096, 4097, 32768)]
        assert v == sorted(v)
    need = f(4, 64)
    ok = dict(dy=P, dt=1, n=4, d=64, ds=64, h=Q, hs=64, w=W, wt=0, eps=1e-6, add=None, adds=64, dx=P + 8192, dxs=64,
              dw=W + 4096, dwt=0, acc=0, ws=W + 8192, room=need)

    def call(**k):
        return L.hc_rms_norm_grad(*{**ok, **k}.values(), None)

    for bad in (dict(dy=None), dict(dy=P + 1), dict(dt=5), dict(ds=1), dict(h=None), dict(hs=63), dict(w=None),
                dict(wt=9), dict(eps=-1.0), dict(add=Q + 1), dict(add=Q, adds=3), dict(dx=None), dict(dxs=2),
                dict(dx=P, dxs=65), dict(dx=Q, hs=65), dict(add=P + 8192, adds=65),
                dict(dw=W + 2), dict(dwt=4), dict(ws=None), dict(ws=W + 8), dict(d=0), dict(n=1 << 31)):
        assert call(**bad) == E, bad
    assert call(room=need - 1) == C
    assert call(n=0, dy=None, h=None, dx=None, dw=None, ws=None, room=0) == 0
    assert call(n=0, dy=None, h=None, dx=None, acc=1, ws=None, room=0) == 0


# ------------------------------------------------------------------ routing

def opts(hc, **k):  # noqa: F811
    return hc.hc_route_opts_t(*{**dict(k=2, scores=0, ngroups=4, top_groups=2, group_best=1, renormalise=1, scale=1.0,
                                       bias=None), **k}.values())


def test_route_refusals(hc):  # noqa: F811
    L, E = hc.load(), hc.HC_ERR_INVALID_ARGUMENT

    def call(x=P, dt=0, n=4, e=16, s=16, ids=Q, w=W, **k):
        return L.hc_route(x, dt, n, e, s, ctypes.byref(opts(hc, **k)), ids, w, None)

    def grad(x=P, dt=0, n=4, e=16, s=16, ids=Q, w=W, dx=P + 4096, ds=16, **k):
        return L.hc_route_grad(x, dt, n, e, s, ctypes.byref(opts(hc, **k)), ids, w, dx, ds, None)

    both = (dict(x=None), dict(x=P + 2), dict(dt=3), dict(e=0), dict(e=1025, s=1025, ds=1025), dict(s=15), dict(ids=None),
            dict(ids=Q + 2), dict(w=None), dict(w=W + 1), dict(k=0), dict(k=65), dict(n=1 << 31), dict(n=1 << 30),
            dict(scores=2), dict(scores=-1), dict(scale=NAN), dict(scale=INF))
    for bad in both:
        assert grad(**bad) == E, bad
        assert call(**{n: v for n, v in bad.items() if n != "ds"}) == E, bad
    for bad in (dict(ngroups=0), dict(ngroups=3), dict(ngroups=65, e=65 * 4, s=65 * 4), dict(top_groups=0),
                dict(top_groups=5), dict(group_best=0), dict(group_best=3), dict(k=9), dict(bias=W + 2)):
        assert call(**bad) == E, bad
    assert grad(dx=None) == E and grad(dx=P + 1) == E and grad(ds=15) == E and grad(dx=P, ds=17) == E
    assert L.hc_route(P, 0, 4, 16, 16, None, Q, W, None) == E
    assert L.hc_route_grad(P, 0, 4, 16, 16, None, Q, W, P, 16, None) == E
    assert call(n=0, x=None, ids=None, w=None) == 0 and grad(n=0, x=None, ids=None, w=None, dx=None) == 0


# ------------------------------------------------------------------ AdamW

def floats(*v):
    return (ctypes.c_float * len(v))(*v)


def test_adamw_plan_refusals(hc):  # noqa: F811
    L, E, C = hc.load(), hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    need = hc.hc_adamw_table_bytes(2)
    assert need > hc.hc_adamw_table_bytes(1) >= 16 and hc.hc_adamw_table_bytes(0) >= 16
    assert hc.hc_adamw_table_bytes((1 << 24) + 1) == 0
    plan = hc.hc_adamw_plan_t()
    ok = dict(p=ptrs(P, P + 4096), g=ptrs(Q, Q + 4096), m=ptrs(P + 0x10000, P + 0x20000), v=ptrs(P + 0x30000, P + 0x40000),
              ms=None, vs=None, c=None, d=None, n=sizes(16, 1000), pt=types(0, 1), gt=types(1, 0), k=2, t=W, room=need)

    def call(**k):
        return L.hc_adamw_plan(ctypes.byref(plan), *{**ok, **k}.values(), None)

    scales = dict(ms=ptrs(W + 0x1000, W + 0x2000), vs=ptrs(W + 0x3000, W + 0x4000))
    for bad in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(n=None), dict(pt=None), dict(gt=None),
                dict(p=ptrs(P, 0)), dict(p=ptrs(P + 2, P + 4096)), dict(p=ptrs(P, P + 4097)), dict(g=ptrs(0, Q)),
                dict(g=ptrs(Q + 1, Q + 4096)), dict(m=ptrs(P + 0x10002, P + 0x20000)), dict(v=ptrs(P + 0x30000, 0)),
                dict(pt=types(0, 2)), dict(gt=types(-1, 0)), dict(n=sizes(16, 1 << 44)), dict(k=1 << 25),
                dict(c=ptrs(0, P + 0x50000)),                              # a copy of a bf16 parameter
                dict(c=ptrs(P + 0x50001, 0)), dict(d=floats(1.0, NAN)), dict(ms=ptrs(W, W)),
                dict(t=None), dict(t=W + 8),
                {**scales, "ms": ptrs(W + 0x1000, 0)}, {**scales, "vs": ptrs(W + 0x1002, W + 0x4000)}):
        assert call(**bad) == E, bad
    for bad in (dict(p=ptrs(P, P + 60)), dict(p=ptrs(P, P)), dict(g=ptrs(P, Q)), dict(m=ptrs(P, P + 0x20000)),
                dict(m=ptrs(P + 0x10000, P + 0x10020)), dict(v=ptrs(P + 0x30000, P + 0x20000 + 3996)),
                dict(g=ptrs(Q, P + 0x40000)), dict(c=ptrs(Q, 0)),
                {**scales, "ms": ptrs(W + 0x1000, W + 0x1000)}, {**scales, "vs": ptrs(P + 8, W + 0x4000)}):
        assert call(**bad) == E and b"overlaps" in L.hc_last_error(), bad
    assert call(room=need - 1) == C
    assert L.hc_adamw_plan(None, *ok.values(), None) == E
    # nothing to do: no launch
    assert call(k=0) == 0 and plan.chunks == 0 and plan.ntensors == 0 and plan.d_table == W
    assert call(n=sizes(0, 0), p=ptrs(0, 0), g=ptrs(0, 0), m=ptrs(0, 0), v=ptrs(0, 0)) == 0 and plan.chunks == 0


def test_adamw_refusals(hc):  # noqa: F811
    L, E = hc.load(), hc.HC_ERR_INVALID_ARGUMENT
    good = dict(ntensors=0, chunks=0, state_bits=32, d_table=W)
    o = dict(step=1, lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.0, scale=1.0, max_norm=1.0, d_norm=None, d_lr=None,
             d_step=None, seed=0, skip=0)

    def call(plan=None, **k):
        p = hc.hc_adamw_plan_t(*{**good, **(plan or {})}.values())
        return L.hc_adamw(ctypes.byref(p), ctypes.byref(hc.hc_adamw_opts_t(*{**o, **k}.values())), None)

    assert call() == 0                                     # of no tensors
    for bad in (dict(step=0), dict(step=-5), dict(lr=NAN), dict(lr=INF), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=NAN), dict(eps=-1e-8), dict(eps=NAN), dict(eps=1e300), dict(wd=INF),
                dict(scale=NAN), dict(d_norm=P, max_norm=-1.0), dict(d_norm=P, max_norm=NAN), dict(d_norm=P + 2),
                dict(d_lr=P + 2), dict(d_step=P + 4)):
        assert call(**bad) == E, bad
    for bad in (dict(state_bits=16), dict(d_table=None), dict(d_table=W + 8), dict(chunks=1), dict(ntensors=1),
                dict(chunks=1 << 32, ntensors=1)):
        assert call(plan=bad) == E, bad
    assert call(step=0, d_step=P) == 0
    assert L.hc_adamw(None, ctypes.byref(hc.hc_adamw_opts_t(*o.values())), None) == E
    assert L.hc_adamw(ctypes.byref(hc.hc_adamw_plan_t(*good.values())), None, None) == E


# ------------------------------------------------------------------ binding

def test_binding_refuses_host_tensors_and_wrong_types(hc):  # noqa: F811
    x, w, e = torch.zeros(4, 8), torch.zeros(8), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: hc.hc_rms_norm(x, w, x), lambda: hc.hc_rms_norm_8bit(x, w, x.to(torch.uint8), x),
                 lambda: hc.hc_rms_norm_grad(x, x, w, x), lambda: hc.hc_route(x, e, x[:, :2].contiguous()),
                 lambda: hc.hc_route_grad(x, e, x[:, :2].contiguous(), x),
                 lambda: hc.AdamWPlan([x], [x], [x], [x])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: hc.hc_rms_norm(x.double(), w, x), lambda: hc.hc_rms_norm([1.0], w, x),
                 lambda: hc.hc_route(x.half(), e, x), lambda: hc.AdamWPlan([x.half()], [x], [x], [x]),
                 lambda: hc.AdamWPlan([1.0], [x], [x], [x], table=w), lambda: hc.AdamWPlan(7, [x], [x], [x])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="scores"):
        hc.hc_route(x, e, x, scores="relu")
    with pytest.raises(ValueError, match="scores"):
        hc.hc_route_grad(x, e, x, x, scores="relu")
    with pytest.raises(ValueError, match="state_bits"):
        hc.AdamWPlan.for_params([x], [x], state_bits=16)
    with pytest.raises(ValueError, match="gaps"):
        hc.AdamWPlan([x[:, ::2]], [x], [x], [x])


def test_plan_memory_and_streams(hc, monkeypatch):  # noqa: F811
    """What a plan allocates is memory of the stream that it is made on, and is
    recorded on torch's other streams that run it: the calls that torch gets."""
    import contextlib

    class Stream:
        def __init__(self, handle, own=True):
            self.cuda_stream, self.stream_id = handle, 3 if own else handle
            self.waits = []

        def wait_stream(self, other):
            self.waits.append(other)

    class Native:
        def __init__(self):
            self.streams = []

        def adamw_plan(self, *a):
            self.streams.append(a[-1])
            return 0

        def adamw(self, *a):
            self.streams.append(a[-1])
            return 0

    class Fake:
        def __init__(self, n):
            self.n, self.is_cuda, self.device = n, True, torch.device("cuda", 0)

        def numel(self):
            return self.n

    now, made, recorded = [Stream(0)], [], []

    class Memory:
        device = torch.device("cuda", 0)

        def __init__(self, *a, **k):
            made.append((self, now[-1]))

        def zero_(self):
            return self

        def record_stream(self, s):
            recorded.append((self, s))

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    native = Native()
    monkeypatch.setattr(hc, "_native", native)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, Memory)
    external = {}
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: external.setdefault(h, Stream(h, False)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(hc, "_current_stream_handle", lambda: now[-1].cuda_stream)
    side, other = Stream(0x100), Stream(0x200)
    x = [Fake(5)]
    # a table by itself, by an object and by a handle
    plan = hc.AdamWPlan(x, x, x, x, stream=side)
    assert [s for _, s in made] == [side] and native.streams == [0x100]
    hc.AdamWPlan(x, x, x, x, stream=0x300)
    assert made[-1][1] is external[0x300] and native.streams[-1] == 0x300
    hc.AdamWPlan(x, x, x, x)
    assert made[-1][1] is now[0]
    mine = Memory()
    given = hc.AdamWPlan(x, x, x, x, table=mine, stream=side)
    assert given.table is mine and made[-1][0] is mine
    # steps: each of torch's streams once, no other's, and not what the caller owns
    for _ in range(2):
        hc.hc_adamw(plan, 1, stream=side)
        hc.hc_adamw(plan, 1, stream=other)
        hc.hc_adamw(plan, 1)
        hc.hc_adamw(plan, 1, stream=0x300)
        hc.hc_adamw(plan, 1, stream=external[0x300])
        hc.hc_adamw(given, 1, stream=other)
    assert recorded == [(plan.table, side), (plan.table, other), (plan.table, now[0])]
    # for_params: its states, which both streams see
    for bits, n in ((32, 3), (8, 5)):
        made.clear(), recorded.clear(), now[0].waits.clear()
        plan = hc.AdamWPlan.for_params(x, x, state_bits=bits, stream=side)
        assert len(made) == n and all(s is side for _, s in made) and now[0].waits == [side] and side.waits[-1] is now[0]
        hc.hc_adamw(plan, 1, stream=other)
        assert {id(m) for m, _ in recorded} == {id(m) for m, _ in made} and all(s is other for _, s in recorded)
    now[0].waits.clear()
    hc.AdamWPlan.for_params(x, x)
    assert made[-1][1] is now[0] and not now[0].waits
