"""The operators around the gradient exchange on the GPU, against the plain
formulas in 64 bits on the CPU: gradient norm and clipping, embedding lookup
and gradient, tokens sorted by expert and back, with the gradient.

Tolerances count roundings: half a step is 2^-24 of the value in fp32 and 2^-8
in bf16, and a sum of m fp32 terms in any order is off by at most m * 2^-24 of
the sum of magnitudes (m - 1 additions, and one for a product's rounding).
Every output buffer stands between guard values, which must survive."""
import math

import pytest
import torch

from collective_communication_amd import binding as hc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}   # half a step among the smallest numbers
F, B = torch.float32, torch.bfloat16
GUARD = 77.0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def guarded(shape, dtype, stride=None, offset=0):
    """A matrix (or vector) of GUARD values inside a larger buffer of them, its
    rows `stride` apart and its first element `offset` elements in."""
    rows, dim = shape if len(shape) == 2 else (1, shape[0])
    stride = stride or dim
    buf = torch.full((offset + rows * stride + 64,), GUARD, dtype=dtype, device="cuda")
    m = buf[offset:offset + rows * stride].view(rows, stride)[:, :dim]
    return buf, (m if len(shape) == 2 else m[0])


def check_guards(buf, view):
    view.fill_(GUARD)
    assert bool((buf == GUARD).all()), "values outside the output changed"


def close(got, want, bound, what=""):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(got.isnan(), want.isnan()), what
    off = (got - want).abs() - bound.double().cpu()
    off = torch.where(want.isnan() | (got == want), -1.0, off)
    assert bool((off <= 0).all()), f"{what}: {int((off > 0).sum())} of {off.numel()} outside, worst by {float(off.max())}"


def space(n):
    return torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ norm and clipping

def norm64(xs, kind="l2"):
    v = torch.cat([x.double().reshape(-1).cpu() for x in xs]) if xs else torch.zeros(0, dtype=torch.float64)
    if v.isnan().any():
        return math.nan
    return float(v.square().sum().sqrt()) if kind == "l2" else float(v.abs().max()) if v.numel() else 0.0


def clip(xs, max_norm, **k):
    d = torch.full((1,), -1.0, device="cuda")
    outs = [torch.full_like(x, GUARD) for x in xs]
    hc.hc_clip_grad_norm(xs, max_norm, d, space(hc.hc_grad_norm_workspace_bytes(len(xs))), outs=outs, **k)
    return float(d), outs


SIZES = {
    "one value": [1],
    "none": [],
    "empty tensors": [0, 5, 0, 0, 7, 0],
    "a chunk's edges": [4095, 4096, 4097, 8191, 8192, 8193],
    "128 tensors": [1 + 37 * (i % 11) for i in range(128)],
    "129 tensors": [1 + 37 * (i % 11) for i in range(129)],
    "600 tensors": [(i * 7919) % 5000 for i in range(600)],
    "large": [3_000_001, 17, 5_000_000],
}


@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("name", SIZES)
def test_norm_and_clip(name, types, kind):
    g = gen(1)
    xs = []
    for i, n in enumerate(SIZES[name]):
        dt = {"f32": F, "bf16": B, "mixed": (F, B)[i % 2]}[types]
        # an odd offset: only element aligned
        xs.append(torch.randn(n + 3, generator=g, device="cuda").mul_(10.0 ** (i % 5 - 2)).to(dt)[3:])
    want = norm64(xs, kind)
    d = torch.full((3,), GUARD, device="cuda")
    hc.hc_grad_norm(xs, d[1:2], space(hc.hc_grad_norm_workspace_bytes(len(xs))), norm=kind)
    assert float(d[0]) == GUARD and float(d[2]) == GUARD
    assert abs(float(d[1]) - want) <= 1.01 * U * want
    for max_norm in (0.3 * want, 2.0 * want + 1.0):
        norm, outs = clip(xs, max_norm, norm=kind)
        assert norm == float(d[1]), "one norm, whichever call finds it"
        coef = min(1.0, max_norm / (want + 1e-6))
        for x, o in zip(xs, outs):
            w = x.double().cpu() * coef
            # the norm, its sum with 1e-6, the quotient, the argument and the product: 5 roundings in fp32
            close(o, w, w.abs() * (5.1 * U + HALF[x.dtype]) + TINY[x.dtype], name)
        again = [x.clone() for x in xs]
        hc.hc_clip_grad_norm(again, max_norm, d[1:2], space(hc.hc_grad_norm_workspace_bytes(len(xs))), norm=kind)
        assert all(torch.equal(a, o) for a, o in zip(again, outs)), "in place gives the same bits"
        hc.hc_clip_grads(xs, d[1:2], max_norm, space(hc.hc_grad_norm_workspace_bytes(len(xs))), outs=outs)
        assert all(torch.equal(a, o) for a, o in zip(again, outs))


@pytest.mark.parametrize("outs_flat", [True, False])
@pytest.mark.parametrize("gap", [0, 3])
def test_views_of_buckets(gap, outs_flat):
    """Views that follow one another in their buckets, fp32 and bf16 in turn,
    some left out and (gap) some values between: as if they were apart."""
    g = gen(6)
    flat = {dt: torch.randn(400_000, generator=g, device="cuda").to(dt) for dt in (F, B)}
    into = {dt: torch.full_like(flat[dt], GUARD) for dt in (F, B)}
    at, xs, os, spots = {F: 0, B: 1}, [], [], []
    for i in range(300):
        dt, n = (F, B)[i * 7 % 3 % 2], (i * 131) % 1500
        if i % 50 != 49:
            xs.append(flat[dt][at[dt]:at[dt] + n])
            os.append(into[dt][at[dt]:at[dt] + n] if outs_flat else torch.full((n,), GUARD, dtype=dt, device="cuda"))
            spots.append((dt, at[dt], n))
        at[dt] += n + gap
    want = norm64(xs)
    d = torch.zeros(1, device="cuda")
    ws = space(hc.hc_grad_norm_workspace_bytes(len(xs)))
    hc.hc_clip_grad_norm(xs, 1.0, d, ws, outs=os)
    assert abs(float(d) - want) <= 1.01 * U * want
    coef = min(1.0, 1.0 / (want + 1e-6))
    for x, o in zip(xs, os):
        w = x.double().cpu() * coef
        close(o, w, w.abs() * (5.1 * U + HALF[x.dtype]) + TINY[x.dtype])
    if outs_flat:
        for dt, a, n in spots:
            into[dt][a:a + n] = GUARD
        assert all(bool((into[dt] == GUARD).all()) for dt in (F, B))
    first = [o.clone() for o in os] if not outs_flat else None
    hc.hc_clip_grad_norm(xs, 1.0, d, ws)              # in place
    if first is not None:
        assert all(torch.equal(x, o) for x, o in zip(xs, first))


def test_clip_leaves_what_surrounds_it():
    g = gen(2)
    for dt in (F, B):
        for n in (1, 7, 8, 9, 4097, 16384 + 5):
            for off in (0, 1, 3):
                buf, x = guarded((n,), dt, offset=off)
                x.copy_(torch.randn(n, generator=g, device="cuda"))
                d = torch.zeros(1, device="cuda")
                hc.hc_clip_grad_norm([x], 1e-3, d, space(hc.hc_grad_norm_workspace_bytes(1)))
                assert float(x.double().norm()) < 1.1e-3
                check_guards(buf, x)


def test_norm_of_extreme_and_special_values():
    big = torch.tensor([3e38, -2e38, 1e30], device="cuda")
    small = torch.tensor([1e-38, 2e-42, -3e-40], device="cuda")
    # the norm of `big` itself is past fp32's range and rounds to infinity; halved, only its squares are
    for x in (big, big / 2, small):
        norm, outs = clip([x], 1.0)
        want = norm64([x])
        if want > torch.finfo(F).max:
            assert norm == math.inf and bool((outs[0] == 0).all())
            continue
        assert abs(norm - want) <= 1.01 * U * want + 2.0 ** -150
    inf = torch.tensor([1.0, math.inf, -2.0], device="cuda")
    norm, outs = clip([inf, torch.ones(2, device="cuda")], 1.0)
    assert norm == math.inf                                     # coefficient 0: 0 * inf is NaN
    assert outs[0].tolist()[0] == 0.0 and math.isnan(outs[0].tolist()[1]) and outs[1].tolist() == [0.0, 0.0]
    for kind in ("l2", "inf"):
        for dt in (F, B):
            x = torch.ones(20_000, device="cuda", dtype=dt)
            x[12_345] = math.nan
            norm, outs = clip([torch.ones(5, device="cuda"), x], 1.0, norm=kind)
            assert math.isnan(norm) and all(bool(o.isnan().all()) for o in outs)
    norm, outs = clip([torch.zeros(9, device="cuda")], 0.0)
    assert norm == 0.0 and outs[0].tolist() == [0.0] * 9


@pytest.mark.parametrize("dtype", [F, B])
def test_clipping_of_the_smallest_values(dtype):
    """Gradients among the smallest numbers are scaled, not flushed."""
    x = torch.tensor([1e-38, 2e-40, -3e-40, 9.2e-41, -9.2e-41, 0.0], device="cuda").to(dtype)
    assert int((x != 0).sum()) == 5
    norm, outs = clip([x], 1.0)
    assert norm > 0 and torch.equal(outs[0], x)                 # a coefficient of 1
    norm, outs = clip([x], 3e-7)
    want = x.double().cpu() * (3e-7 / (norm64([x]) + 1e-6))
    close(outs[0], want, want.abs() * (5.1 * U + HALF[dtype]) + TINY[dtype])
    assert bool((outs[0][:3] != 0).all())


def test_clip_by_a_norm_of_more_than_these_tensors():
    """Two ranks' shards: each clips by the norm of both."""
    a, b = (torch.randn(5000, generator=gen(s), device="cuda") for s in (3, 4))
    norms = torch.zeros(2, device="cuda")
    ws = space(hc.hc_grad_norm_workspace_bytes(1))
    for i, x in enumerate((a, b)):
        hc.hc_grad_norm([x], norms[i:i + 1], ws)
    total = norms.square().sum().sqrt().reshape(1)
    want = norm64([a, b])
    for x in (a, b):
        y = x.double() * min(1.0, 2.0 / (want + 1e-6))
        hc.hc_clip_grads([x], total, 2.0, ws)
        close(x, y, y.abs().cpu() * 10 * U)


def test_clip_takes_dense_tensors_in_any_order_and_refuses_gaps():
    x = torch.randn(30, 40, generator=gen(5), device="cuda")
    norm, _ = clip([x.t()], 1.0)
    assert abs(norm - norm64([x])) <= 1.01 * U * norm
    with pytest.raises(ValueError):
        clip([x[:, :20]], 1.0)
    with pytest.raises(hc.HcError) as e:
        hc.hc_clip_grad_norm([x, x], 1.0, torch.zeros(1, device="cuda"), space(4096 * 8))
    assert e.value.status == hc.HC_ERR_INVALID_ARGUMENT


def test_norm_of_more_than_2_to_32_values():
    n = (1 << 32) + 12345
    x = torch.zeros(n, dtype=B, device="cuda")
    x[0], x[(1 << 31) + 1], x[-1] = 3.0, 4.0, 12.0
    d = torch.zeros(1, device="cuda")
    hc.hc_clip_grad_norm([x], 6.5, d, space(hc.hc_grad_norm_workspace_bytes(1)))
    assert float(d) == 13.0
    assert float(x[0]) == 1.5 and float(x[(1 << 31) + 1]) == 2.0 and float(x[-1]) == 6.0
    assert int(x.count_nonzero()) == 3


@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("apart", [3, 150])
@pytest.mark.parametrize("values", [20_000_000, 90_000_000, 170_000_000])
def test_norm_and_clip_of_large_buckets(values, apart, kind):
    """fp32 and bf16 tensors, few and many, through the sizes where the passes
    take other loads and stores; checked on the device, in slices of fp64."""
    g = gen(7)
    flat = torch.randn(values, generator=g, device="cuda")
    n = values // apart
    xs = [flat[i * n:i * n + n - 1 - i % 3].to((F, B)[i % 4 == 3]) for i in range(apart)]
    parts = [(x.double().square().sum() if kind == "l2" else x.double().abs().max()) for x in xs]
    total = torch.stack(parts)
    want = float(total.sum().sqrt() if kind == "l2" else total.max())
    norm, outs = clip(xs, 0.4 * want, norm=kind)
    assert abs(norm - want) <= 1.01 * U * want
    coef = 0.4 * want / (want + 1e-6)
    for x, o in zip(xs, outs):
        w = x.double() * coef
        assert bool(((o.double() - w).abs() <= w.abs() * (5.1 * U + HALF[x.dtype]) + TINY[x.dtype]).all())


# ------------------------------------------------------------------ embedding

def make_ids(pattern, n, vocab, start, idt, g):
    if pattern == "one":
        k = torch.full((n,), vocab // 2, device="cuda")
    elif pattern == "falling":
        k = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab + 1)).exp().long() - 1
        k = k.clamp_(0, vocab - 1)
    elif pattern == "outside":       # below, inside, at both borders, far above
        k = torch.randint(-vocab, 2 * vocab, (n,), generator=g, device="cuda")
        k[::7], k[1::7], k[2::7], k[3::7] = vocab, vocab - 1, -1, 0
    elif pattern == "none":
        k = torch.full((n,), vocab + 1, device="cuda")
    else:
        k = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    return (k + start).to(idt)


LOOKUPS = [
    # tokens, vocab, dim, pattern, start, id type
    (1, 1, 1, "any", 0, torch.int64),
    (1, 300, 4096, "any", 0, torch.int32),
    (0, 10, 8, "any", 0, torch.int64),
    (5, 7, 3, "outside", 1 << 40, torch.int64),
    (130, 77, 64, "outside", 50, torch.int32),
    (257, 1000, 65, "falling", -500, torch.int64),
    (1000, 50, 513, "outside", 0, torch.int32),
    (3001, 5003, 1031, "falling", 0, torch.int64),
    (64, 11, 8200, "any", 0, torch.int64),
    (33, 5, 40, "none", 0, torch.int32),
]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("case", LOOKUPS, ids=lambda c: "-".join(map(str, c[:4])))
def test_embedding(case, dtype):
    n, vocab, dim, pattern, start, idt = case
    g = gen(11)
    ids = make_ids(pattern, n, vocab, start, idt, g)
    for pad, off, scale in ((0, 0, 1.0), (5, 1, 0.37)):
        _, weight = guarded((vocab, dim), dtype, dim + pad, off)
        weight.copy_(torch.randn((vocab, dim), generator=g, device="cuda"))
        buf, out = guarded((n, dim), dtype, dim + 2 * pad, off)
        hc.hc_embedding(ids, weight, out, vocab_start=start, scale=scale)
        k = ids.cpu().to(torch.int64) - start
        there = (k >= 0) & (k < vocab)
        want = torch.zeros((n, dim), dtype=torch.float64)
        want[there] = weight.double().cpu()[k[there]] * float(torch.tensor(scale, dtype=F))
        close(out, want, want.abs() * (U + HALF[dtype]) + TINY[dtype])
        if scale == 1.0:
            assert torch.equal(out.double().cpu(), want)
        check_guards(buf, out)


GRADS = [
    # tokens, vocab, dim, pattern, start, id type, padding
    (1, 1, 1, "any", 0, torch.int64, None),
    (1, 40, 260, "any", 0, torch.int32, None),
    (0, 10, 8, "any", 0, torch.int64, None),
    (64, 5, 16, "one", 0, torch.int64, None),
    (65, 100, 7, "outside", 1 << 35, torch.int64, (1 << 35) + 3),
    (500, 33, 1031, "falling", 100, torch.int32, 100),
    (4096, 300, 24, "falling", 0, torch.int64, None),
    (4097, 300, 24, "falling", 0, torch.int64, 1),
    (8192, 1025, 24, "falling", 0, torch.int64, None),
    (8193, 1025, 24, "outside", 5, torch.int32, None),
    (5000, 2, 72, "one", 0, torch.int32, None),
    (5000, 9, 520, "none", 0, torch.int32, None),
    (9001, 1500, 130, "outside", -700, torch.int64, None),
    (20_000, 70_001, 40, "falling", 0, torch.int64, 5),
    (70_000, 2_000_003, 3, "any", 0, torch.int32, None),
    (140_000, 600, 600, "falling", 0, torch.int32, None),
    # tables too large to be zeroed beside the sort; a sort whose tiles hold more than four items a lane
    (500, 40_000, 520, "falling", 0, torch.int64, None),
    (700, 110_000, 500, "falling", 0, torch.int32, None),
    (5000, 150_000, 400, "outside", 0, torch.int64, None),
    (300_001, 5000, 9, "falling", 0, torch.int32, None),
    (400_003, 100, 10, "one", 0, torch.int32, None),
]


@pytest.mark.parametrize("types", [(F, F), (B, F), (B, B), (F, B)], ids=["f32", "bf16-f32", "bf16", "f32-bf16"])
@pytest.mark.parametrize("case", GRADS, ids=lambda c: "-".join(map(str, c[:4])))
def test_embedding_grad(case, types):
    n, vocab, dim, pattern, start, idt, padding = case
    dt, wt = types
    g = gen(12)
    ids = make_ids(pattern, n, vocab, start, idt, g)
    pad = 3 if dim < 1000 else 0
    _, dout = guarded((n, dim), dt, dim + pad, 1)
    dout.copy_(torch.randn((n, dim), generator=g, device="cuda"))
    ws = space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim))
    scale = float(torch.tensor(0.7, dtype=F))
    k = ids.cpu().to(torch.int64) - start
    there = (k >= 0) & (k < vocab)
    if padding is not None:
        there &= ids.cpu().to(torch.int64) != padding
    k, d = k[there], dout.double().cpu()[there]
    total = torch.zeros((vocab, dim), dtype=torch.float64).index_add_(0, k, d)
    mags = torch.zeros((vocab, dim), dtype=torch.float64).index_add_(0, k, d.abs())
    terms = torch.zeros(vocab, dtype=torch.float64).index_add_(0, k, torch.ones(len(k), dtype=torch.float64))[:, None]
    for accumulate in (False, True):
        buf, dw = guarded((vocab, dim), wt, dim + pad, 1)
        before = torch.zeros((vocab, dim), dtype=torch.float64)
        if accumulate:
            dw.copy_(torch.randn((vocab, dim), generator=g, device="cuda"))
            before = dw.double().cpu()
        start_bits = dw.clone()
        hc.hc_embedding_grad(ids, dout, dw, ws, vocab_start=start, padding_id=padding, scale=scale,
                             accumulate=accumulate)
        want = before + scale * total
        # the terms' additions, the scale's product, the accumulation; then the stored value's rounding
        bound = scale * mags * (terms + 2) * U + want.abs() * (U + HALF[wt]) + TINY[wt]
        close(dw, want, bound, f"accumulate={accumulate}")
        touched = terms[:, 0] > 0
        if accumulate:
            assert torch.equal(dw.cpu()[~touched], start_bits.cpu()[~touched])
        else:
            assert not bool(dw.cpu()[~touched].any())
            first = dw.clone()
            hc.hc_embedding_grad(ids, dout, dw, ws, vocab_start=start, padding_id=padding, scale=scale)
            assert torch.equal(first, dw), "two runs differ"
        check_guards(buf, dw)


def test_one_gradient_workspace_for_all_batches():
    """The workspace of the largest batch serves smaller ones, narrower tables
    and fewer rows, and only the sizes asked for are needed."""
    g = gen(16)
    ws = space(hc.hc_embedding_grad_workspace_bytes(16_500, 3000, 1024))
    for n, vocab, dim in ((16_500, 3000, 1024), (16_300, 3000, 1024), (8192, 3000, 1024), (8191, 1000, 1024),
                          (5000, 1000, 1024), (16_500, 3000, 255), (3, 1, 1)):
        ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        dout = torch.randint(-4, 5, (n, dim), generator=g, device="cuda").float()     # sums are exact
        want = torch.zeros((vocab, dim), dtype=torch.float64).index_add_(0, ids.cpu(), dout.cpu().double())
        room = hc.hc_embedding_grad_workspace_bytes(n, vocab, dim)
        assert room <= ws.numel()
        own = torch.full((room + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        for w in (ws, own[:room]):
            dw = torch.full((vocab, dim), GUARD, device="cuda")
            hc.hc_embedding_grad(ids, dout, dw, w)
            assert torch.equal(dw.double().cpu(), want), (n, vocab, dim)
        assert bool((own[room:] == 0xA5).all()), "written past the workspace"


def test_embedding_grad_against_differences():
    """d/dW of <out, r> by differences of the lookup's own output (fp32; the
    lookup is linear, so a step of 1 is exact up to rounding)."""
    g = gen(13)
    n, vocab, dim = 40, 9, 5
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    w = torch.randn((vocab, dim), generator=g, device="cuda")
    r = torch.randn((n, dim), generator=g, device="cuda")
    dw, out = torch.empty_like(w), torch.empty_like(r)
    hc.hc_embedding_grad(ids, r, dw, space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim)), scale=2.0)

    def loss(x):
        hc.hc_embedding(ids, x, out, scale=2.0)
        return float((out.double() * r.double()).sum())

    base = loss(w)
    mag = 2.0 * float(r.abs().sum()) * (float(w.abs().max()) + 1)
    for v in range(vocab):
        for d in range(dim):
            x = w.clone()
            x[v, d] += 1.0
            assert abs(loss(x) - base - float(dw[v, d])) <= 4 * n * U * mag


@pytest.mark.parametrize("n", [90, 6000])
def test_masked_tokens_may_hold_anything(n):
    """Gradients of tokens outside the table or of the padding id are not read
    into any row, whatever they hold."""
    g = gen(15)
    vocab, dim = 50, 33
    ids = torch.randint(-20, vocab + 20, (n,), generator=g, device="cuda")
    dout = torch.randn((n, dim), generator=g, device="cuda")
    out = (ids < 0) | (ids >= vocab) | (ids == 7)
    ws = space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim))
    got = []
    for junk in (0.0, math.nan, math.inf):
        dout[out] = junk
        dw = torch.full((vocab, dim), GUARD, device="cuda")
        hc.hc_embedding_grad(ids, dout, dw, ws, padding_id=7)
        got.append(dw)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert not bool(got[0][7].any())


def test_embedding_offsets_past_2_to_32():
    g = gen(14)
    vocab, dim, stride = 20, 70, 1 << 28
    big = torch.empty(vocab * stride, dtype=B, device="cuda")
    weight = big.view(vocab, stride)[:, :dim]
    weight.copy_(torch.randn((vocab, dim), generator=g, device="cuda"))
    ids = torch.arange(vocab, device="cuda").flip(0)
    out = torch.empty((vocab, dim), dtype=B, device="cuda")
    hc.hc_embedding(ids, weight, out)
    assert torch.equal(out, weight.flip(0))
    ws = space(hc.hc_embedding_grad_workspace_bytes(vocab, vocab, dim))
    dout = torch.randn((vocab, dim), generator=g, device="cuda").to(B)
    hc.hc_embedding_grad(ids, dout, weight, ws)
    assert torch.equal(weight.flip(0), dout)
    hc.hc_embedding_grad(ids, weight, out, ws)          # rows far apart as the input
    assert torch.equal(out, dout)


# ------------------------------------------------------------------ experts

EXPERTS = [
    # tokens, k, experts, align, dim, all experts, first of ours
    (1, 1, 1, 1, 1, 1, 0),
    (0, 2, 4, 8, 16, 4, 0),
    (1, 8, 64, 16, 2048, 64, 0),
    (3, 2, 5, 1, 7, 5, 0),
    (100, 64, 64, 4, 33, 64, 0),
    (130, 3, 7, 16, 513, 28, 14),
    (511, 2, 1024, 2, 64, 1024, 0),
    (513, 2, 1000, 1, 65, 1000, 0),
    (2500, 6, 16, 1, 260, 64, 16),
    (5003, 2, 8, 32, 1031, 8, 0),
    (4096, 5, 3, 7, 72, 9, 3),
    (33_000, 4, 129, 1, 24, 129, 0),
    (90_001, 4, 300, 3, 5, 300, 0),
    (50, 2, 4, 1000, 40, 4, 0),
    (2100, 3, 70, 65, 9, 75, 2),
]


def expert_case(case, dtype, g, idt=torch.int32):
    n, k, e, align, dim, every, start = case
    ids = torch.rand((n, every), generator=g, device="cuda").topk(k, dim=1).indices if k <= every else \
        torch.randint(0, every, (n, k), generator=g, device="cuda")
    if n > 20:
        ids[3] = -1                       # a masked token
        ids[5, 0] = every + 1000          # a masked choice
    plan = hc.ExpertPlan.for_sizes(n, k, e, align)
    for t in (plan.row_of_slot, plan.slot_of_row, plan.expert_offsets, plan.expert_counts):
        t.fill_(-99)
    hc.hc_expert_sort(ids.to(idt), plan, space(hc.hc_expert_sort_workspace_bytes(n * k, e)), expert_start=start)
    return ids, plan


def plan_by_loops(ids, n, k, e, align, start, rows):
    slots = [[] for _ in range(e)]
    for s, x in enumerate((ids.reshape(-1).cpu() - start).tolist()):
        if 0 <= x < e:
            slots[x].append(s)
    row_of, slot_of, offsets, at = [-1] * (n * k), [-1] * rows, [0], 0
    for l in slots:
        for i, s in enumerate(l):
            row_of[s], slot_of[at + i] = at + i, s
        at += -(-len(l) // align) * align
        offsets.append(at)
    return row_of, slot_of, offsets, [len(l) for l in slots]


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_expert_sort(case, idt):
    n, k, e, align, _, _, start = case
    ids, plan = expert_case(case, F, gen(21), idt)
    want = plan_by_loops(ids, n, k, e, align, start, plan.rows)
    got = (plan.row_of_slot, plan.slot_of_row, plan.expert_offsets, plan.expert_counts)
    for name, a, b in zip(("row_of_slot", "slot_of_row", "offsets", "counts"), got, want):
        assert a.tolist() == b, name


def test_one_sort_workspace_for_all_batches():
    """The workspace of the largest batch serves the smaller ones."""
    g = gen(26)
    k, e = 2, 128
    ws = space(hc.hc_expert_sort_workspace_bytes(35_000 * k, e))
    for n in (35_000, 32_768, 30_000, 2500, 7):
        ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
        plan = hc.ExpertPlan.for_sizes(n, k, e)
        hc.hc_expert_sort(ids, plan, ws)
        want = torch.sort(ids.reshape(-1), stable=True).indices.int()
        assert torch.equal(plan.slot_of_row, want), n


@pytest.mark.parametrize("tokens", [700, 40_000])
def test_expert_sort_when_all_choose_one(tokens):
    for chosen in (0, 4):                 # an expert of ours, then none of ours
        plan = hc.ExpertPlan.for_sizes(tokens, 1, 3, 64)
        ids = torch.full((tokens, 1), chosen, dtype=torch.int32, device="cuda")
        hc.hc_expert_sort(ids, plan, space(hc.hc_expert_sort_workspace_bytes(tokens, 3)))
        if chosen == 0:
            assert torch.equal(plan.row_of_slot, torch.arange(tokens, device="cuda", dtype=torch.int32))
            assert plan.expert_counts.tolist() == [tokens, 0, 0]
        else:
            assert bool((plan.row_of_slot == -1).all()) and bool((plan.slot_of_row == -1).all())
            assert plan.expert_offsets.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: "-".join(map(str, c)))
def test_expert_rows(case, dtype):
    n, k, e, align, dim, every, start = case
    g = gen(22)
    ids, plan = expert_case(case, dtype, g)
    row = plan.row_of_slot.cpu().long().view(n, k)
    slot = plan.slot_of_row.cpu().long()
    used = int(plan.expert_offsets[-1])
    for pad, off in ((0, 0), (3, 1)):
        mat = lambda r, fill=True: (lambda b, m: (m.copy_(torch.randn(m.shape, generator=g, device="cuda")), (b, m))[1]  # noqa: E731
                                    if fill else (b, m))(*guarded((r, dim), dtype, dim + pad, off))
        # dispatch: copies, zero padding, nothing past the last expert
        x = mat(n)[1]
        buf, rows = mat(plan.rows, False)
        hc.hc_expert_dispatch(x, plan, rows)
        want = torch.full((plan.rows, dim), GUARD, dtype=dtype)
        want[:used] = 0
        want[slot >= 0] = x.cpu()[slot[slot >= 0] // k]
        assert torch.equal(rows.cpu(), want)
        check_guards(buf, rows)
        # combine; rows that no slot has hold NaN, which must not be read
        rows = mat(plan.rows)[1]
        rows[slot.cuda() < 0] = math.nan
        weights = torch.rand((n, k), generator=g, device="cuda")
        here = row >= 0
        picked = torch.where(here[..., None], rows.double().cpu()[row.clamp(min=0)] if plan.rows else
                             torch.zeros(n, k, dim, dtype=torch.float64), 0.0)
        for w in (weights, None):
            buf, out = mat(n, False)
            hc.hc_expert_combine(rows, plan, w, out)
            terms = picked * (w.double().cpu()[..., None] if w is not None else 1.0)
            want = terms.sum(1)
            close(out, want, terms.abs().sum(1) * k * U + want.abs() * HALF[dtype] + TINY[dtype], "combine")
            first = out.clone()
            hc.hc_expert_combine(rows, plan, w, out)
            assert torch.equal(first, out)
            check_guards(buf, out)
        # the gradient of combine
        dout = mat(n)[1]
        buf, drows = mat(plan.rows, False)
        wbuf, dweights = guarded((n * k,), F)
        hc.hc_expert_combine_grad(dout, rows, plan, weights, drows, dweights)
        want = torch.full((plan.rows, dim), GUARD, dtype=torch.float64)
        want[:used] = 0
        s = slot[slot >= 0]
        want[slot >= 0] = dout.double().cpu()[s // k] * weights.double().cpu().view(-1)[s][:, None]
        close(drows, want, want.abs() * (U + HALF[dtype]) + TINY[dtype], "drows")
        prod = picked * dout.double().cpu()[:, None, :]
        close(dweights.view(n, k), prod.sum(2), prod.abs().sum(2) * dim * U + TINY[F], "dweights")
        first = (drows.clone(), dweights.clone())
        hc.hc_expert_combine_grad(dout, rows, plan, weights, drows, dweights)
        assert torch.equal(first[0], drows) and torch.equal(first[1], dweights)
        check_guards(buf, drows)
        check_guards(wbuf, dweights)


def test_row_numbers_outside_the_plan_count_as_none():
    g = gen(25)
    n, k, dim = 40, 3, 50
    ids, plan = expert_case((n, k, 6, 4, dim, 6, 0), F, g)
    x = torch.randn((n, dim), generator=g, device="cuda")
    w = torch.rand((n, k), generator=g, device="cuda")
    got = []
    for none in (-1, plan.rows, (1 << 31) - 1, -(1 << 31)):
        plan.row_of_slot[::5] = none
        _, rows = guarded((plan.rows, dim), F)
        buf, drows = guarded((plan.rows, dim), F)
        out, dw = torch.empty_like(x), torch.empty_like(w)
        hc.hc_expert_dispatch(x, plan, rows)
        hc.hc_expert_combine(rows, plan, w, out)
        hc.hc_expert_combine_grad(x, rows, plan, w, drows, dw)
        got.append((rows.clone(), out, drows.clone(), dw))
        check_guards(buf, drows)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    plan.expert_offsets[-1] = 1 << 30          # padding ends with the rows' room
    buf, rows = guarded((plan.rows, dim), F)
    hc.hc_expert_dispatch(x, plan, rows)
    check_guards(buf, rows)


def test_combine_gradients_against_differences():
    """<combine(rows, w), r>: its derivatives by every weight and by every row
    value, from differences of hc_expert_combine itself (it is linear in both)."""
    g = gen(23)
    n, k, e, dim = 6, 2, 4, 5
    ids, plan = expert_case((n, k, e, 3, dim, e + 2, 1), F, g)
    rows = torch.randn((plan.rows, dim), generator=g, device="cuda")
    w = torch.rand((n, k), generator=g, device="cuda")
    r = torch.randn((n, dim), generator=g, device="cuda")
    drows, dw, out = torch.full_like(rows, 0.0), torch.empty_like(w), torch.empty_like(r)
    hc.hc_expert_combine_grad(r, rows, plan, w, drows, dw)

    def loss(a, b):
        hc.hc_expert_combine(a, plan, b, out)
        return float((out.double() * r.double()).sum())

    base = loss(rows, w)
    tol = 64 * U * float(r.abs().sum()) * (float(rows.abs().max()) + 1) * 2 * k
    for t in range(n):
        for j in range(k):
            b = w.clone()
            b[t, j] += 1.0
            assert abs(loss(rows, b) - base - float(dw[t, j])) <= tol
    used = int(plan.expert_offsets[-1])
    for i in range(used):
        for d in range(dim):
            a = rows.clone()
            a[i, d] += 1.0
            assert abs(loss(a, w) - base - float(drows[i, d])) <= tol


def test_expert_offsets_past_2_to_32():
    g = gen(24)
    n, k, dim, stride = 10, 2, 130, 1 << 28
    ids, plan = expert_case((n, k, 3, 1, dim, 3, 0), B, g)
    big = torch.empty(plan.rows * stride, dtype=B, device="cuda")
    rows = big.view(plan.rows, stride)[:, :dim]
    x = torch.randn((n, dim), generator=g, device="cuda").to(B)
    hc.hc_expert_dispatch(x, plan, rows)
    assert torch.equal(rows, x[plan.slot_of_row.long() // k])
    out = torch.empty_like(x)
    hc.hc_expert_combine(rows, plan, None, out)
    assert torch.equal(out, 2 * x)
    w = torch.full((n, k), 0.5, device="cuda")
    small, dw = torch.empty((plan.rows, dim), dtype=B, device="cuda"), torch.empty_like(w)
    hc.hc_expert_combine_grad(x, rows, plan, w, small, dw)
    assert torch.equal(small, (x * 0.5)[plan.slot_of_row.long() // k])
    sq = x.double().square().sum(1)
    close(dw, sq[:, None].expand(n, k), sq[:, None].expand(n, k).cpu() * dim * U)
    hc.hc_expert_combine_grad(x, small, plan, w, rows, dw)
    assert torch.equal(rows, small)


@pytest.mark.parametrize("start", [(1 << 63) - 3, -(1 << 63)])
def test_ids_at_the_ends_of_64_bits(start):
    """A range that begins near an end of the ids' type holds the ids from its
    start on, and none from the other end."""
    top, low, vocab, dim = (1 << 63) - 1, -(1 << 63), 10, 12
    ids = torch.tensor([low, low + 1, low + 6, top - 7, top - 2, top - 1, top, 0], device="cuda")
    keys = [i - start if start <= i < start + vocab else -1 for i in ids.tolist()]
    weight = torch.randn((vocab, dim), generator=gen(27), device="cuda")
    out, dw = torch.full((len(keys), dim), GUARD, device="cuda"), torch.full((vocab, dim), GUARD, device="cuda")
    hc.hc_embedding(ids, weight, out, vocab_start=start)
    want = torch.stack([weight[k] if k >= 0 else torch.zeros(dim, device="cuda") for k in keys])
    assert torch.equal(out, want), keys
    dout = torch.arange(1.0, len(keys) + 1, device="cuda")[:, None].expand(-1, dim).contiguous()
    hc.hc_embedding_grad(ids, dout, dw, space(hc.hc_embedding_grad_workspace_bytes(len(keys), vocab, dim)),
                         vocab_start=start)
    sums = [sum(t + 1.0 for t, k in enumerate(keys) if k == v) for v in range(vocab)]
    assert dw[:, 0].tolist() == sums, keys
    plan = hc.ExpertPlan.for_sizes(len(keys), 1, vocab)
    hc.hc_expert_sort(ids, plan, expert_start=start)
    assert plan.expert_counts.tolist() == [keys.count(v) for v in range(vocab)], keys


def test_what_fixes_the_order_of_sums():
    """The embedding gradient's bits follow the ids, the tokens and the width
    alone, wherever the rows lie; the norm's, the tensors' places to one another
    and in their lines."""
    g = gen(28)
    n, vocab, dim = 6000, 700, 200
    ids = make_ids("falling", n, vocab, 0, torch.int64, g)
    ws = space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim))
    values = torch.randn((n, dim), generator=g, device="cuda")
    got = []
    for pad, off, idt in ((0, 0, torch.int64), (5, 3, torch.int32), (128, 1, torch.int64)):
        _, dout = guarded((n, dim), F, dim + pad, off)
        dout.copy_(values)
        _, dw = guarded((vocab, dim), F, dim + pad, off)
        hc.hc_embedding_grad(ids.to(idt), dout, dw, ws.random_(0, 256, generator=g))
        got.append(dw.clone())
    assert all(torch.equal(x, got[0]) for x in got[1:])
    flat = torch.randn(2_000_000, generator=g, device="cuda")
    norms = []
    for buf in (flat, flat.clone()):
        xs = [buf[3 + i * 9973:3 + i * 9973 + 9973 - i % 2] for i in range(200)]
        d = torch.zeros(1, device="cuda")
        hc.hc_grad_norm(xs, d, space(hc.hc_grad_norm_workspace_bytes(len(xs))))
        norms.append(float(d))
    assert norms[0] == norms[1]


# ------------------------------------------------------------------ with the exchange

@pytest.mark.parametrize("dtype", [F, B])
def test_a_table_split_over_ranks(dtype):
    """Each rank looks up its part of the vocabulary and hc_allreduce adds the
    rows, which gives the whole table's; each rank's gradient is its part of
    the whole one."""
    g = gen(71)
    n, vocab, dim = 501, 1000, 136
    weight = torch.randn((vocab, dim), generator=g, device="cuda").to(dtype)
    dout = torch.randn((n, dim), generator=g, device="cuda").to(dtype)
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    ws = space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim))
    whole, dwhole = torch.empty_like(dout), torch.empty_like(weight)
    hc.hc_embedding(ids, weight, whole, scale=0.3)
    hc.hc_embedding_grad(ids, dout, dwhole, ws, scale=0.3)
    cuts, outs = (0, 334, 667, vocab), []
    for a, b in zip(cuts, cuts[1:]):
        outs.append(torch.full_like(dout, GUARD))
        hc.hc_embedding(ids, weight[a:b], outs[-1], vocab_start=a, scale=0.3)
        part = torch.full((b - a, dim), GUARD, dtype=dtype, device="cuda")
        hc.hc_embedding_grad(ids, dout, part, ws, vocab_start=a, scale=0.3)
        k = ids[(ids >= a) & (ids < b)] - a
        terms = torch.zeros(b - a, device="cuda").index_add_(0, k, torch.ones(len(k), device="cuda"))[:, None]
        mags = torch.zeros((b - a, dim), device="cuda").index_add_(0, k, dout[(ids >= a) & (ids < b)].float().abs())
        # the same terms in another order: twice the order's bound and the result's two roundings
        near(part, dwhole[a:b].double(), 2 * (0.3 * mags * (terms + 2) * U + dwhole[a:b].double().abs() *
                                              (U + HALF[dtype]) + TINY[dtype]), (a, b))
    hc.hc_allreduce(outs, outs)
    assert all(torch.equal(o, whole) for o in outs)             # a row and zeroes: exact


def test_experts_split_over_ranks():
    """Each rank lays out, runs and combines its experts' rows, and
    hc_allreduce adds the ranks' sums, which gives all experts'."""
    g = gen(72)
    n, k, every, dim, ranks = 300, 4, 12, 72, 3
    x = torch.randn((n, dim), generator=g, device="cuda")
    ids = torch.rand((n, every), generator=g, device="cuda").topk(k, dim=1).indices
    ids[5] = -1                                                 # a masked token
    w = torch.rand((n, k), generator=g, device="cuda")
    gain = torch.randn((every, dim), generator=g, device="cuda")    # expert e scales its rows
    parts = []
    for r in range(ranks):
        e = every // ranks
        plan = hc.ExpertPlan.for_sizes(n, k, e, 16)
        hc.hc_expert_sort(ids, plan, expert_start=r * e)
        rows = torch.zeros((plan.rows, dim), device="cuda")
        hc.hc_expert_dispatch(x, plan, rows)
        ends = plan.expert_offsets.tolist()
        for i in range(e):
            rows[ends[i]:ends[i + 1]] *= gain[r * e + i]
        parts.append(torch.full((n, dim), GUARD, device="cuda"))
        hc.hc_expert_combine(rows, plan, w, parts[-1])
    hc.hc_allreduce(parts, parts)
    terms = torch.where((ids >= 0)[..., None], x.double()[:, None] * gain.double()[ids.clamp(min=0)], 0.0) * w[..., None]
    # a product in the rows, k in the sums, one addition per rank
    near(parts[0], terms.sum(1), terms.abs().sum(1) * (1 + k + ranks) * U + TINY[F], "sum")
    assert all(torch.equal(p, parts[0]) for p in parts[1:]) and not bool(parts[0][5].any())


# ------------------------------------------------------------------ rows past the caches

def slices(n, per):
    """Ranges of [0, n) of some 8 million values, `per` each."""
    step = max(1, (1 << 23) // per)
    return [slice(i, min(n, i + step)) for i in range(0, n, step)]


def near(got, want, bound, what):
    assert bool(((got.double() - want).abs() <= bound).all()), what


LARGE_LOOKUPS = [
    # tokens, rows, dim, type: 128 MiB of output and more
    (33_000, 900, 1031, F),
    (33_000, 20_011, 2051, B),
    (540_000, 5000, 65, F),
    (11_300_000, 1000, 3, F),
    (13_500_000, 70_000, 5, B),
]


@pytest.mark.parametrize("case", LARGE_LOOKUPS, ids=lambda c: "-".join(map(str, c)))
def test_large_lookups(case):
    n, vocab, dim, dtype = case
    g = gen(61)
    ids = torch.randint(-vocab // 4, vocab + 5, (n,), generator=g, device="cuda", dtype=torch.int32)
    _, weight = guarded((vocab, dim), dtype, dim + 3, 1)
    weight.copy_(torch.randn((vocab, dim), generator=g, device="cuda"))
    buf, out = guarded((n, dim), dtype, dim + 1, 3)
    assert out.numel() * out.element_size() >= 128 << 20
    hc.hc_embedding(ids, weight, out, scale=2.0)
    for s in slices(n, dim):
        k = ids[s].long()
        there = (k >= 0) & (k < vocab)
        want = torch.where(there[:, None], weight[k.clamp(0, vocab - 1)] * 2.0, 0.0)
        assert torch.equal(out[s], want), s
    check_guards(buf, out)


LARGE_ROWS = [
    # tokens, k, dim, type: rows by slot of 128 to 256 MiB or more, a token's side below 128 MiB or above
    (33_000, 1, 1031, F),
    (17_000, 4, 1031, F),
    (33_000, 2, 2051, B),
    (140_000, 1, 513, B),
    (100_000, 3, 250, F),
    (6_000_000, 2, 3, F),
    (14_000_000, 2, 5, B),
]


@pytest.mark.parametrize("case", LARGE_ROWS, ids=lambda c: "-".join(map(str, c)))
def test_large_expert_rows(case):
    n, k, dim, dtype = case
    g = gen(62)
    e, every, start, align = 7, 9, 1, 4
    first = torch.randint(0, every, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    ids = (first + torch.arange(k, device="cuda", dtype=torch.int32) * 2) % every
    plan = hc.ExpertPlan.for_sizes(n, k, e, align)
    hc.hc_expert_sort(ids, plan, space(hc.hc_expert_sort_workspace_bytes(n * k, e)), expert_start=start)
    row, slot, used = plan.row_of_slot.view(n, k), plan.slot_of_row, int(plan.expert_offsets[-1])
    here = (ids >= start) & (ids < start + e)
    assert torch.equal(row >= 0, here) and int(here.sum()) == int((slot >= 0).sum())
    placed = torch.where(here, row, 0).view(-1).long()
    assert torch.equal(slot[placed[here.view(-1)]], here.view(-1).nonzero()[:, 0].int())
    assert n * k * dim * (4 if dtype == F else 2) >= 128 << 20
    x = guarded((n, dim), dtype, dim + 1, 1)[1]
    x.copy_(torch.randn((n, dim), generator=g, device="cuda", dtype=dtype))
    # dispatch
    buf, rows = guarded((plan.rows, dim), dtype, dim + 3, 3)
    hc.hc_expert_dispatch(x, plan, rows)
    for s in slices(used, dim):
        want = torch.where((slot[s] >= 0)[:, None], x[(slot[s].long() // k).clamp(min=0)], 0.0)
        assert torch.equal(rows[s], want), s
    assert bool((rows[used:] == GUARD).all())
    check_guards(buf, rows)
    # combine; what no slot has is NaN, which must not be read
    rows.copy_(torch.randn((plan.rows, dim), generator=g, device="cuda", dtype=dtype))
    rows[slot < 0] = math.nan
    weights = torch.rand((n, k), generator=g, device="cuda")
    buf, out = guarded((n, dim), dtype, dim + 1, 1)
    for w in (weights, None):
        hc.hc_expert_combine(rows, plan, w, out)
        for s in slices(n, k * dim):
            picked = torch.where(here[s][..., None], rows[row[s].long().clamp(min=0)].double(), 0.0)
            terms = picked * (w[s].double()[..., None] if w is not None else 1.0)
            want = terms.sum(1)
            near(out[s], want, terms.abs().sum(1) * k * U + want.abs() * HALF[dtype] + TINY[dtype], ("combine", s))
    check_guards(buf, out)
    del buf, out
    # the gradient of combine, of x as the output's
    buf, drows = guarded((plan.rows, dim), dtype, dim + 1, 1)
    wbuf, dweights = guarded((n * k,), F)
    hc.hc_expert_combine_grad(x, rows, plan, weights, drows, dweights)
    by_slot = weights.view(-1)
    for s in slices(used, dim):
        at = slot[s].long().clamp(min=0)
        want = torch.where((slot[s] >= 0)[:, None], x[at // k].double() * by_slot[at].double()[:, None], 0.0)
        near(drows[s], want, want.abs() * (U + HALF[dtype]) + TINY[dtype], ("drows", s))
    assert bool((drows[used:] == GUARD).all())
    for s in slices(n, k * dim):
        prod = torch.where(here[s][..., None], rows[row[s].long().clamp(min=0)].double(), 0.0) * x[s].double()[:, None]
        near(dweights.view(n, k)[s], prod.sum(2), prod.abs().sum(2) * dim * U + TINY[F], ("dweights", s))
    check_guards(buf, drows)
    check_guards(wbuf, dweights)


@pytest.mark.parametrize("types", [(F, F), (B, B)], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(700, 300, 9001), (9000, 1500, 8195), (300, 1500, 24_001), (200, 40, 70_003)],
                         ids=lambda c: "-".join(map(str, c)))
def test_gradient_of_wide_rows_that_lie_apart(case, types):
    """Tables of few wide rows with something between them, which the zeroing
    beside the sort takes row by row.  Sums of small integers are exact."""
    n, vocab, dim = case
    dt, wt = types
    g = gen(63)
    ids = make_ids("falling", n, vocab, 0, torch.int32, g)
    dout = torch.randint(-2, 3, (n, dim), generator=g, device="cuda").to(dt)
    want = torch.zeros((vocab, dim), device="cuda").index_add_(0, ids.long(), dout.float())
    buf, dw = guarded((vocab, dim), wt, dim + 5, 1)
    hc.hc_embedding_grad(ids, dout, dw, space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim)))
    assert torch.equal(dw, want.to(wt))
    check_guards(buf, dw)


# ------------------------------------------------------------------ streams and graphs

def step_calls(s):
    """One of each operator on the state's buffers."""
    hc.hc_embedding(s["ids"], s["table"], s["x"], scale=1.5)
    hc.hc_expert_sort(s["experts"], s["plan"], s["ws1"])
    hc.hc_expert_dispatch(s["x"], s["plan"], s["rows"])
    hc.hc_expert_combine(s["rows"], s["plan"], s["w"], s["y"])
    hc.hc_expert_combine_grad(s["y"], s["rows"], s["plan"], s["w"], s["drows"], s["dw"])
    hc.hc_expert_combine(s["drows"], s["plan"], None, s["dx"])
    hc.hc_embedding_grad(s["ids"], s["dx"], s["dtable"], s["ws2"], scale=1.5)
    hc.hc_clip_grad_norm([s["dtable"], s["dw"]], 0.5, s["norm"], s["ws3"], outs=[s["clipped"], s["dw2"]])


def step_state(n=4500, k=3, e=20, dim=192, vocab=3000):
    g = gen(31)
    plan = hc.ExpertPlan.for_sizes(n, k, e, 8)
    r = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"plan": plan, "table": r(vocab, dim).to(B), "w": torch.rand((n, k), generator=g, device="cuda"),
         "ws1": space(hc.hc_expert_sort_workspace_bytes(n * k, e)),
         "ws2": space(hc.hc_embedding_grad_workspace_bytes(n, vocab, dim)),
         "ws3": space(hc.hc_grad_norm_workspace_bytes(2)), "norm": torch.zeros(1, device="cuda"),
         "ids": torch.zeros(n, dtype=torch.int64, device="cuda"),
         "experts": torch.zeros((n, k), dtype=torch.int32, device="cuda")}
    for name, rows in (("x", n), ("y", n), ("dx", n), ("rows", plan.rows), ("drows", plan.rows)):
        s[name] = torch.zeros((rows, dim), dtype=B, device="cuda")
    s["dtable"], s["clipped"] = (torch.zeros((vocab, dim), device="cuda") for _ in range(2))
    s["dw"], s["dw2"] = (torch.zeros((n, k), device="cuda") for _ in range(2))
    return s


def new_inputs(s, seed):
    g = gen(seed)
    n, k = s["w"].shape
    s["ids"].copy_(make_ids("falling", n, s["table"].shape[0], 0, torch.int64, g))
    s["experts"].copy_(torch.rand((n, s["plan"].nexperts), generator=g, device="cuda").topk(k, dim=1).indices)


OUTPUTS = ("y", "drows", "dw", "dx", "dtable", "clipped", "dw2", "norm")


def test_graph_replays_equal_eager():
    s = step_state()
    new_inputs(s, 40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step_calls(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_calls(s)
    for seed in range(41, 46):
        new_inputs(s, seed)
        graph.replay()
        torch.cuda.synchronize()
        got = {o: s[o].clone() for o in OUTPUTS}
        for o in OUTPUTS:
            s[o].fill_(GUARD)
        step_calls(s)
        torch.cuda.synchronize()
        for o in ("y", "dw", "dx", "dtable", "clipped", "dw2", "norm"):
            assert torch.equal(got[o], s[o]), (seed, o)
        used = int(s["plan"].expert_offsets[-1])
        assert torch.equal(got["drows"][:used], s["drows"][:used]), seed


def test_calls_run_on_the_stream_they_are_given():
    s, want = step_state(), step_state()
    new_inputs(s, 50)
    new_inputs(want, 50)
    step_calls(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    slow = torch.zeros(1 << 27, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):               # the inputs arrive late, on the same stream
            slow.add_(1.0)
        new_inputs(s, 50)
        step_calls(s)
    side.synchronize()
    for o in OUTPUTS:
        assert torch.equal(s[o], want[o]), o


@pytest.mark.parametrize("handle", ["stream", "raw handle"])
def test_calls_on_a_stream_given_by_argument(handle):
    """Every call takes stream=, and runs there in order, whichever stream is current."""
    s, want = step_state(), step_state()
    new_inputs(s, 51)
    new_inputs(want, 52)
    step_calls(want)
    want["norm2"] = want["norm"].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = {n: want[n].clone() for n in ("ids", "experts")}
    slow = torch.zeros(1 << 27, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            slow.add_(1.0)
        for n, x in late.items():
            s[n].copy_(x)
    k = {"stream": side if handle == "stream" else side.cuda_stream}
    s["norm2"] = torch.zeros(1, device="cuda")
    torch.cuda.current_stream().synchronize()        # s["norm2"]; the side stream is still at work
    hc.hc_embedding(s["ids"], s["table"], s["x"], scale=1.5, **k)
    hc.hc_expert_sort(s["experts"], s["plan"], s["ws1"], **k)
    hc.hc_expert_dispatch(s["x"], s["plan"], s["rows"], **k)
    hc.hc_expert_combine(s["rows"], s["plan"], s["w"], s["y"], **k)
    hc.hc_expert_combine_grad(s["y"], s["rows"], s["plan"], s["w"], s["drows"], s["dw"], **k)
    hc.hc_expert_combine(s["drows"], s["plan"], None, s["dx"], **k)
    hc.hc_embedding_grad(s["ids"], s["dx"], s["dtable"], s["ws2"], scale=1.5, **k)
    hc.hc_clip_grad_norm([s["dtable"], s["dw"]], 0.5, s["norm"], s["ws3"], outs=[s["clipped"], s["dw2"]], **k)
    hc.hc_grad_norm([s["dtable"], s["dw"]], s["norm2"], s["ws3"], **k)
    side.synchronize()
    for o in OUTPUTS:
        assert torch.equal(s[o], want[o]), o
    assert abs(float(s["norm2"]) - float(want["norm2"])) <= 2 * U * float(want["norm2"])
    hc.hc_clip_grads([s["dtable"], s["dw"]], s["norm"], 0.5, s["ws3"], **k)      # in place
    side.synchronize()
    assert torch.equal(s["dtable"], want["clipped"]) and torch.equal(s["dw"], want["dw2"])


def test_calls_on_a_stream_of_few_compute_units():
    """No call waits for more workgroups than the stream's compute units hold."""
    s, want = step_state(), step_state()
    new_inputs(s, 60)
    new_inputs(want, 60)
    step_calls(want)
    torch.cuda.synchronize()
    handle = hc.hc_stream_create_cu_budget(8)
    try:
        with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
            step_calls(s)
        torch.cuda.synchronize()
        for o in OUTPUTS:
            assert torch.equal(s[o], want[o]), o
    finally:
        torch.cuda.synchronize()
        hc.hc_stream_destroy(handle)
