"""Host-side checks of the operators around the gradient exchange (no GPU
needed): sizes, and every refusal of the C ABI and of the binding.  No call
here reaches a launch: each must return its status before anything is
enqueued (a launch in a process without a GPU would be HC_ERR_DEVICE)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "collective_communication_amd", "libhc.so")
P, Q, W = 0x10000000, 0x20000000, 0x30000000     # addresses that no call touches


@pytest.fixture(scope="module")
def hc():
    if not os.path.exists(LIB):
        pytest.skip("libhc.so not built")
    from collective_communication_amd import binding
    return binding


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def sizes(*v):
    return (ctypes.c_size_t * len(v))(*v)


def types(*v):
    return (ctypes.c_int32 * len(v))(*v)


# ------------------------------------------------------------------ sizes

def test_rows_bound(hc):
    assert hc.hc_expert_rows_bound(10, 2, 4, 1) == 20
    assert hc.hc_expert_rows_bound(10, 2, 4, 16) == 20 + 4 * 15
    assert hc.hc_expert_rows_bound(1, 2, 64, 16) == 2 + 2 * 15      # at most two experts have tokens
    assert hc.hc_expert_rows_bound(0, 2, 64, 16) == 0
    for bad in ((10, 0, 4, 1), (10, 65, 4, 1), (10, 2, 0, 1), (10, 2, 1025, 1), (10, 2, 4, 0), (1 << 31, 2, 4, 1)):
        assert hc.hc_expert_rows_bound(*bad) == 0


def test_workspaces_grow_and_cover(hc):
    assert hc.hc_grad_norm_workspace_bytes(0) > 0
    assert hc.hc_grad_norm_workspace_bytes(1000) >= hc.hc_grad_norm_workspace_bytes(0) + 1000 * 28
    assert hc.hc_expert_sort_workspace_bytes(64, 128) == 0           # one launch, nothing kept
    assert hc.hc_expert_sort_workspace_bytes(1 << 20, 128) >= 64 * 128 * 4
    assert hc.hc_expert_sort_workspace_bytes(64, 0) == 0
    a, b = hc.hc_embedding_grad_workspace_bytes(100, 50, 64), hc.hc_embedding_grad_workspace_bytes(100_000, 50, 64)
    assert 0 < a < b and b >= 2 * 4 * 100_000                        # keys and places of every token


def test_expert_sort_workspaces_serve_fewer_slots_and_experts(hc):
    """A workspace for some sizes is enough for all that are none larger."""
    slots = sorted({max(0, n + d) for n in (0, 1, 1000, 4096, 10_000, 60_000, 65_536, 70_000, 131_072, 1 << 20,
                                            (1 << 31) - 2) for d in (-1, 0, 1)})
    for e in (1, 3, 128, 1023, 1024):
        size = [hc.hc_expert_sort_workspace_bytes(n, e) for n in slots]
        assert size == sorted(size), [(n, s) for n, s in zip(slots, size)]
        assert all(hc.hc_expert_sort_workspace_bytes(n, max(1, e - 1)) <= s for n, s in zip(slots, size))
    # the call itself: past the check of the size, the misaligned workspace is what it refuses
    L, room = hc.load(), hc.hc_expert_sort_workspace_bytes(70_000, 128)
    for n in (70_000, 65_536, 60_000, 33_000, 5000):
        plan = plan_of(hc, ntokens=n, k=1, nexperts=128, row_align=1, rows=n)
        assert L.hc_expert_sort(Q, 4, 0, ctypes.byref(plan), W + 8, room, None) == hc.HC_ERR_INVALID_ARGUMENT
        assert b"aligned" in L.hc_last_error(), (n, L.hc_last_error())


def test_embedding_grad_workspaces_serve_smaller_batches(hc):
    """The same for the gradient of a table: fewer tokens, rows or columns."""
    f = hc.hc_embedding_grad_workspace_bytes
    near = lambda *v: sorted({max(0, x + d) for x in v for d in (-1, 0, 1)})  # noqa: E731
    tokens = near(0, 7, 64, 1000, 4096, 8192, 16_384, 20_000, 24_576, 32_768, 65_536, 98_304, 393_216, 1 << 20,
                  (1 << 31) - 2)
    rows = near(1, 500, 1024, 100_003, (1 << 31) - 2)
    columns = near(1, 8, 255, 256, 512, 1024, 2048, 4096, 8192, 1 << 20, (1 << 31) - 2)
    for v in rows:
        for d in columns:
            size = [f(n, v, d) for n in tokens]
            assert size == sorted(size), (v, d)
    for n in tokens:
        for d in columns:
            size = [f(n, v, d) for v in rows]
            assert size == sorted(size), (n, d)
        for v in rows:
            size = [f(n, v, d) for d in columns]
            assert size == sorted(size), (n, v)
    # what the call lays out: keys and places, the long sort's histograms and pairs, two partials per chunk
    for n, v, d, chunk, scratch in ((8191, 100_003, 4096, 16, 0), (8192, 100_003, 4096, 32, 0), (100, 10, 300, 8, 0),
                                    (24_575, 100_003, 4096, 32, 1), (32_768, 100_003, 4096, 64, 1),
                                    (5000, 1024, 64, 8, 1)):
        need = 8 * n + scratch * (64 * 1024 * 4 + 8 * n) + -(-n // chunk) * 2 * 4 * d
        assert f(n, v, d) >= need, (n, v, d)
    # the call itself: past the check of the size, the misaligned workspace is what it refuses
    L, room = hc.load(), f(32_768, 100_003, 4096)
    for n, v, d in ((32_768, 100_003, 4096), (24_575, 100_003, 4096), (8191, 100_003, 4096), (8000, 1000, 4096),
                    (32_768, 100_003, 511), (1, 1, 1)):
        assert L.hc_embedding_grad(P, 4, n, Q, 1, d, v, d, 0, -1, 1.0, W, 0, d, 0, W + 8, room,
                                   None) == hc.HC_ERR_INVALID_ARGUMENT
        assert b"aligned" in L.hc_last_error(), (n, v, d, L.hc_last_error())


# ------------------------------------------------------------------ gradients

def test_norm_refusals(hc):
    L = hc.load()
    E, C = hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    need = hc.hc_grad_norm_workspace_bytes(2)
    ok = dict(g=ptrs(P, Q), c=sizes(8, 8), d=types(0, 1), n=2, kind=0, out=W, ws=W + 64, room=need)

    def call(**k):
        a = {**ok, **k}
        return L.hc_grad_norm(a["g"], a["c"], a["d"], a["n"], a["kind"], a["out"], a["ws"], a["room"], None)

    assert call(g=None) == E and call(c=None) == E and call(d=None) == E
    assert call(g=ptrs(P, 0)) == E and b"grads[1]" in L.hc_last_error()
    assert call(g=ptrs(P + 2, Q)) == E and b"aligned" in L.hc_last_error()     # fp32 at a 2-byte address
    assert call(g=ptrs(P, Q + 1)) == E
    assert call(d=types(0, 7)) == E and call(d=types(-1, 0)) == E
    assert call(kind=2) == E
    assert call(out=None) == E and call(out=W + 2) == E
    assert call(ws=None) == E and call(ws=W + 8) == E
    assert call(room=need - 1) == C
    assert call(c=sizes(8, 1 << 60)) == E
    assert call(n=1 << 30) == E


def test_clip_refusals(hc):
    L = hc.load()
    E, C = hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    need = hc.hc_grad_norm_workspace_bytes(2)
    ok = dict(g=ptrs(P, P + 64), o=ptrs(Q, Q + 64), c=sizes(16, 32), d=types(0, 1), n=2, max=1.0, out=W, ws=W + 64,
              room=need)

    def both(**k):
        a = {**ok, **k}
        s = L.hc_clip_grad_norm(a["g"], a["o"], a["c"], a["d"], a["n"], 0, a["max"], a["out"], a["ws"], a["room"], None)
        t = L.hc_clip_grads(a["g"], a["o"], a["c"], a["d"], a["n"], a["out"], a["max"], a["ws"], a["room"], None)
        assert s == t
        return s

    assert both(o=None) == E
    assert both(o=ptrs(Q, 0)) == E and both(o=ptrs(Q + 1, Q + 64)) == E
    assert both(o=ptrs(Q, Q + 60)) == E and b"overlaps" in L.hc_last_error()    # two outputs
    assert both(o=ptrs(P + 64, Q)) == E                                        # over another's gradient
    assert both(o=ptrs(P + 4, Q)) == E                                         # over a part of its own
    assert both(g=ptrs(P, P), o=ptrs(P, P)) == E                               # one gradient listed twice, in place
    assert both(g=ptrs(P, P + 60), o=ptrs(Q, P + 60)) == E                     # an in-place one over another's input
    for bad in (-1.0, float("nan")):
        assert both(max=bad) == E and b"max_norm" in L.hc_last_error()
    assert both(room=need - 1) == C
    assert both(out=None) == E


# ------------------------------------------------------------------ embedding

def test_embedding_refusals(hc):
    L = hc.load()
    E, C = hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    ok = dict(ids=P, ib=8, n=4, w=Q, dt=1, v=10, dim=16, ws=16, out=W, os=16)

    def look(**k):
        a = {**ok, **k}
        return L.hc_embedding(a["ids"], a["ib"], a["n"], a["w"], a["dt"], a["v"], a["dim"], a["ws"], 0, 1.0, a["out"],
                              a["os"], None)

    assert look(ids=None) == E and look(ids=P + 4) == E
    assert look(ib=2) == E and look(dt=5) == E
    assert look(w=None) == E and look(w=Q + 1) == E and look(out=None) == E and look(out=W + 1) == E
    assert look(ws=15) == E and look(os=15) == E and b"stride" in L.hc_last_error()
    assert look(n=1 << 31) == E and look(v=1 << 31) == E and look(dim=1 << 31) == E
    need = hc.hc_embedding_grad_workspace_bytes(4, 10, 16)
    okg = dict(ids=P, ib=4, n=4, d=Q, ddt=0, ds=16, v=10, dim=16, w=W, wdt=1, wst=16, space=W + (1 << 20), room=need)

    def grad(**k):
        a = {**okg, **k}
        return L.hc_embedding_grad(a["ids"], a["ib"], a["n"], a["d"], a["ddt"], a["ds"], a["v"], a["dim"], 0, -1, 1.0,
                                   a["w"], a["wdt"], a["wst"], 0, a["space"], a["room"], None)

    assert grad(ids=None) == E and grad(ids=P + 2) == E and grad(ib=0) == E
    assert grad(d=None) == E and grad(d=Q + 2) == E and grad(w=None) == E and grad(w=W + 1) == E
    assert grad(ddt=9) == E and grad(wdt=9) == E and grad(ds=1) == E and grad(wst=1) == E
    assert grad(space=None) == E and grad(space=W + 8) == E and grad(room=need - 1) == C
    assert grad(n=1 << 31) == E


# ------------------------------------------------------------------ experts

def plan_of(hc, **k):
    a = {**dict(ntokens=4, k=2, nexperts=8, row_align=4, rows=8 + 8 * 3, row_of_slot=P, slot_of_row=P + 4096,
                expert_offsets=P + 8192, expert_counts=P + 12288), **k}
    return hc.hc_expert_plan_t(*a.values())


def test_expert_refusals(hc):
    L = hc.load()
    E, C = hc.HC_ERR_INVALID_ARGUMENT, hc.HC_ERR_INSUFFICIENT_CAPACITY
    sort = lambda ids=Q, ib=4, ws=None, room=0, **k: L.hc_expert_sort(  # noqa: E731
        ids, ib, 0, ctypes.byref(plan_of(hc, **k)), ws, room, None)
    assert L.hc_expert_sort(Q, 4, 0, None, None, 0, None) == E
    for bad in (dict(k=0), dict(k=65, rows=10_000), dict(nexperts=0), dict(nexperts=1025), dict(row_align=0),
                dict(ntokens=1 << 31), dict(row_of_slot=None), dict(slot_of_row=None), dict(expert_offsets=None),
                dict(expert_counts=None), dict(row_of_slot=P + 2), dict(rows=1 << 31),
                dict(row_align=1 << 30, rows=(1 << 31) - 1)):
        assert sort(**bad) == E, bad
    assert sort(rows=31) == C and b"rows" in L.hc_last_error()
    assert sort(ids=None) == E and sort(ids=Q + 1) == E and sort(ib=1) == E
    assert sort(ntokens=100_000, rows=200_024) == C                       # it needs a workspace
    plan = plan_of(hc)
    ref = ctypes.byref(plan)
    assert L.hc_expert_dispatch(None, 1, 16, 16, ref, W, 16, None) == E
    assert L.hc_expert_dispatch(Q, 1, 16, 16, None, W, 16, None) == E
    assert L.hc_expert_dispatch(Q, 1, 16, 8, ref, W, 16, None) == E
    assert L.hc_expert_dispatch(Q, 3, 16, 16, ref, W, 16, None) == E
    assert L.hc_expert_dispatch(Q, 1, 16, 16, ref, W + 1, 16, None) == E
    assert L.hc_expert_combine(Q, 1, 16, 16, ref, W + 2, W, 16, None) == E          # weights' alignment
    assert L.hc_expert_combine(Q, 1, 16, 16, ref, None, None, 16, None) == E
    assert L.hc_expert_combine(Q, 1, 16, 15, ref, None, W, 16, None) == E
    good = [Q, 1, 16, 16, W, 16, ref, P, W + (1 << 20), 16, W + (1 << 24), None]
    for at, bad in ((0, None), (1, 4), (3, 3), (4, None), (5, 3), (6, None), (7, None), (8, None), (9, 3), (10, None),
                    (10, W + 1), (7, P + 2)):
        args = list(good)
        args[at] = bad
        assert L.hc_expert_combine_grad(*args) == E, (at, bad)


# ------------------------------------------------------------------ binding

def test_binding_refuses_host_tensors_and_wrong_types(hc):
    f, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        hc.hc_grad_norm([f], torch.zeros(1), torch.zeros(64))
    with pytest.raises(ValueError):
        hc.hc_embedding(i, f, f)
    with pytest.raises(TypeError):
        hc.hc_embedding(i.to(torch.int16), f, f)
    with pytest.raises(TypeError):
        hc.hc_embedding(i, f, f.double())
    with pytest.raises(ValueError):
        hc.ExpertPlan.for_sizes(4, 2, 8, device="cpu")
    with pytest.raises(ValueError, match="norm"):
        hc.hc_grad_norm([], torch.zeros(1), torch.zeros(64), norm="l1")
    with pytest.raises(TypeError):
        hc.hc_grad_norm([f.double()], torch.zeros(1), torch.zeros(64))
    with pytest.raises(TypeError):
        hc.hc_grad_norm([1.0], torch.zeros(1), torch.zeros(64))
    with pytest.raises(TypeError):
        hc.hc_clip_grad_norm(7, 1.0, torch.zeros(1), torch.zeros(64))


def test_dense_storage_rule(hc):
    x = torch.zeros(6, 4, 5)
    for t in (x, x.transpose(0, 1), x.permute(2, 0, 1), x[:1], torch.zeros(3, 1, 4).transpose(0, 1)):
        assert t.is_contiguous() or hc._dense(t)
    for t in (x[:, :2], x[..., ::2], x[:, :, :1].expand(6, 4, 5)):
        assert not t.is_contiguous() and not hc._dense(t)


def test_operators_refuse_tensors_with_gaps(hc):
    """The gap is what they refuse, before the place (these are host tensors);
    without one, in any order of dimensions, it is the place."""
    d, ws = torch.zeros(1), torch.zeros(64)
    x = torch.zeros(6, 4, 5)
    calls = (lambda t: hc.hc_grad_norm([t, x], d, ws), lambda t: hc.hc_clip_grads([t, x], d, 1.0, ws),
             lambda t: hc.hc_clip_grad_norm([t, x], 1.0, d, ws))
    gaps = (x[:, :2], x[..., ::2], x[:, :, :1].expand(6, 4, 5), x.permute(2, 0, 1)[::2], x[:, 1:3].transpose(0, 2),
            torch.zeros(1).expand(7))
    dense = (x, x.transpose(0, 1), x.permute(2, 0, 1), x[:1], torch.zeros(3, 1, 4).transpose(0, 1), x[2, 3])
    for call in calls:
        for t in gaps:
            with pytest.raises(ValueError, match=r"grads\[0\] is not dense"):
                call(t)
        for t in dense:
            assert hc._dense(t)
            with pytest.raises(ValueError, match=r"grads\[0\] is not a device tensor"):
                call(t)
