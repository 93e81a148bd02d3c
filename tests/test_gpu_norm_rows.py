"""The root-mean-square norm of rows on the GPU, its rows of 8 bits and its
gradient, against the formulas in 64 bits on the CPU.

Tolerances count roundings: half a step is U = 2^-24 of the value in fp32 and
2^-8 in bf16.  A row's sum of squares is added up by a lane over at most 32
terms, over 64 lanes in 6 steps and over 16 waves in 15, each term rounded once:
55 roundings, which the root halves; with the mean, eps, root and quotient the
factor r is off by at most 32 U."""
import math

import pytest
import torch

from collective_communication_amd import binding as hc
from test_gpu_step_ops import B, F, GUARD, HALF, TINY, U, check_guards, close, gen, guarded, space

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
R = 32 * U


def rows(g, t, d, dtype, scale=1.0, stride=None, offset=0):
    """Random rows, `stride` apart, the first `offset` elements into their buffer."""
    stride = stride or d
    buf = torch.randn(offset + t * stride, generator=g, device="cuda").mul_(scale).to(dtype)
    return buf[offset:].view(t, stride)[:, :d]


def norm64(x, residual, w, eps):
    """h as it is stored, and the norm in 64 bits, on the CPU."""
    h = x.cpu() if residual is None else (x.float() + residual.float()).to(x.dtype).cpu()
    d = h.double()
    r = 1.0 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    return h, d, r, d * r * w.double().cpu()


DIMS = [1, 2, 3, 4, 7, 8, 9, 31, 64, 65, 100, 255, 256, 257, 512, 513, 1000, 1024, 1031, 2048, 2049, 4096, 4100, 8192,
        8195, 16384, 20001, 32768]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("types", [(F, F), (B, B), (B, F), (F, B)])
@pytest.mark.parametrize("d", DIMS)
def test_norm(d, types, residual):
    dtype, wtype = types
    g = gen(d)
    for t in (1, 5, 67) if d < 5000 else (1, 3):
        pad, off = (0, 0) if t == 5 else (3, 1)
        x = rows(g, t, d, dtype, 1.0, d + pad, off)
        w = torch.randn(d, generator=g, device="cuda").to(wtype)
        res = rows(g, t, d, dtype, 3.0, d + 2 * pad, off) if residual else None
        buf, out = guarded((t, d), dtype, d + pad, off)
        sbuf, s = guarded((t, d), dtype, d + pad, off)
        hc.hc_rms_norm(x, w, out, residual=res, sum_out=s if residual else None, eps=1e-5)
        h, _, _, want = norm64(x, res, w, 1e-5)
        if residual:
            assert torch.equal(s.cpu(), h)
            again = torch.empty_like(out)
            hc.hc_rms_norm(x, w, again, residual=res, eps=1e-5)          # the sum is not kept
            assert torch.equal(again, out)
        close(out, want, want.abs() * (R + 3 * U + HALF[dtype]) + TINY[dtype], f"{t} x {d}")
        check_guards(buf, out)
        check_guards(sbuf, s)


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("types", [(F, F), (B, B), (B, F)])
@pytest.mark.parametrize("d", [1, 3, 8, 31, 32, 33, 100, 255, 256, 263, 1000, 1031, 2048, 4096, 4097, 8192, 16388, 32768])
def test_rows_of_8_bits(d, types, group):
    dtype, wtype = types
    g = gen(d + group)
    t = 9 if d < 5000 else 2
    x, res = rows(g, t, d, dtype, 1.0, d + 1, 1), rows(g, t, d, dtype, 0.5)
    x[t // 2] = 0.0
    res[t // 2] = 0.0
    x[0] *= torch.logspace(-3, 3, d, device="cuda").to(dtype)           # groups of very different sizes
    w = torch.randn(d, generator=g, device="cuda").to(wtype)
    n = -(-d // group) if group else 1
    buf = torch.full((t * (d + 5) + 70,), 0x55, dtype=torch.uint8, device="cuda")
    out = buf[3:3 + t * (d + 5)].view(t, d + 5)[:, :d]
    sbuf, scales = guarded((t, n), F, n + 2, 1)
    hbuf, s = guarded((t, d), dtype, d + 3, 1)
    hc.hc_rms_norm_8bit(x, w, out, scales, group=group, residual=res, sum_out=s, eps=1e-6)
    h, _, r, y = norm64(x, res, w, 1e-6)
    assert torch.equal(s.cpu(), h)
    full = group or d
    prod = torch.nn.functional.pad(h.float() * w.float().cpu(), (0, n * full - d)).view(t, n, full)
    a = prod.abs().amax(2, keepdim=True)
    # one quotient (a number over a tensor is a reciprocal and a product in torch)
    codes = (prod * (torch.full_like(a, 448.0) / torch.where(a > 0, a, 1.0))).view(t, -1)[:, :d].to(E4M3).view(torch.uint8)
    # -0 stands for 0
    same = (out.cpu() == codes) | (((out.cpu() | codes) & 0x7F) == 0)
    assert bool(same.all()), f"{int((~same).sum())} codes differ"
    want = a[..., 0].double() * r / 448.0
    close(scales, want, want * (R + 3 * U) + TINY[F], "scales")
    got = out.contiguous().view(E4M3).cpu().double() * scales.cpu().double().repeat_interleave(full, 1)[:, :d]
    step = want.repeat_interleave(full, 1)[:, :d] * 2.0 ** -10
    # half a step of a code, and the roundings of product, quotient and scale
    close(got, y, y.abs() * (2.0 ** -4 + R + 6 * U) + step * 1.01, "values")
    out.fill_(0x55)
    assert bool((buf == 0x55).all())
    check_guards(sbuf, scales)
    check_guards(hbuf, s)


def test_8_bits_as_float8():
    g = gen(1)
    x, w = rows(g, 6, 256, B), torch.ones(256, device="cuda")
    a, b = torch.empty((6, 256), dtype=E4M3, device="cuda"), torch.empty((6, 256), dtype=torch.uint8, device="cuda")
    s = torch.empty((6, 2), device="cuda")
    hc.hc_rms_norm_8bit(x, w, a, s, group=128)
    hc.hc_rms_norm_8bit(x, w, b, s.clone(), group=128)
    assert torch.equal(a.view(torch.uint8), b)


@pytest.mark.parametrize("dtype", [F, B])
def test_tiny_and_odd_values(dtype):
    """Rows of zeroes, of the smallest normal numbers, with a NaN, with an
    infinity; eps of 0."""
    d = 300
    x = torch.ones((6, d), device="cuda").to(dtype)
    x[1] = 0.0
    x[2] = 2.0 ** -40
    x[3, 17] = math.nan
    x[4, 299] = math.inf
    x[5] = 2.0 ** 60
    w = torch.ones(d, device="cuda")
    out, q, s = torch.empty_like(x), torch.empty((6, d), dtype=E4M3, device="cuda"), torch.empty((6, 3), device="cuda")
    hc.hc_rms_norm(x, w, out, eps=0.0)
    hc.hc_rms_norm_8bit(x, w, q, s, group=128, eps=0.0)
    value = q.float() * s.repeat_interleave(128, 1)[:, :d]
    for i in (0, 2, 5):
        assert bool((out[i] == 1.0).all()) and bool((value[i] - 1.0).abs().max() <= 4 * U), i
    assert bool(out[1].isnan().all())            # 0 / 0, as the formula has it
    hc.hc_rms_norm(x[1:2], w, out[1:2], eps=1e-6)
    hc.hc_rms_norm_8bit(x[1:2], w, q[1:2], s[1:2], group=128, eps=1e-6)
    assert bool((out[1] == 0).all()) and bool((s[1] == 0).all()) and bool((q[1].float() == 0).all())
    assert bool(out[3].isnan().all()) and bool(s[3].isnan().all())
    assert bool((out[4, :299] == 0).all()) and bool(out[4, 299].isnan()) and bool(s[4, 2].isnan())
    # a product that fp32 cannot hold, of finite values: its group is no number, the others are
    x, big = torch.ones((1, 256), device="cuda"), torch.ones(256, device="cuda")
    x[0, 7], big[7] = 2.0 ** 10, 2.0 ** 120
    q, s = torch.empty((1, 256), dtype=E4M3, device="cuda"), torch.empty((1, 2), device="cuda")
    hc.hc_rms_norm_8bit(x, big, q, s, group=128, eps=0.0)
    assert bool(s[0, 0].isnan()) and bool(s[0, 1].isfinite()) and bool((q[0, 128:].float() == 448).all())
    # a weight that is no number, or infinite: its group is none, the others and a moved-back vector's are
    for d, at in ((261, 7), (261, 254), (300, 255), (131, 127)):
        for bad in (math.nan, math.inf):
            x, big = torch.ones((1, d), device="cuda"), torch.ones(d, device="cuda")
            big[at] = bad
            for dtype in (F, B):
                q, s = torch.empty((1, d), dtype=E4M3, device="cuda"), torch.empty((1, -(-d // 128)), device="cuda")
                hc.hc_rms_norm_8bit(x.to(dtype), big, q, s, group=128, eps=0.0)
                assert s[0].isnan().nonzero().view(-1).tolist() == [at // 128], (d, at, bad, dtype)
                other = torch.arange(d, device="cuda") // 128 != at // 128
                assert bool((q[0].float()[other] == 448).all()), (d, at, bad, dtype)
    # values whose t is far below what 448 / t can hold
    x = (torch.arange(1, 257, device="cuda", dtype=F) * 2.0 ** -126).view(1, 256)
    q, s = torch.empty((1, 256), dtype=E4M3, device="cuda"), torch.empty((1, 1), device="cuda")
    hc.hc_rms_norm_8bit(x, torch.ones(256, device="cuda"), q, s, eps=1e-6)
    want = torch.arange(1, 257).double() * 448 / 256
    close(q.float(), want.view(1, -1), want.view(1, -1) * (2.0 ** -4 + 4 * U), "tiny")


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("d", [5, 63, 1031, 4096, 9001])
def test_in_place(d, dtype):
    g = gen(d)
    x, res, w = rows(g, 33, d, dtype), rows(g, 33, d, dtype), torch.randn(d, generator=g, device="cuda")
    out, s = torch.empty_like(x), torch.empty_like(x)
    hc.hc_rms_norm(x, w, out, residual=res, sum_out=s)
    for a, b in (("x", "residual"), ("residual", "x"), (None, "x"), ("x", None), ("residual", None)):
        v = {"x": x.clone(), "residual": res.clone(), None: torch.empty_like(x)}
        hc.hc_rms_norm(v["x"], w, v[a], residual=v["residual"], sum_out=v[b] if b != a else None)
        assert torch.equal(v[a], out), (a, b)
        assert torch.equal(v[b], s), (a, b)
    dy, ds = rows(g, 33, d, dtype), rows(g, 33, d, dtype)
    dx = torch.empty_like(x)
    hc.hc_rms_norm_grad(dy, s, w, dx, dsum=ds)
    for name in ("dout", "dsum"):
        v = {"dout": dy.clone(), "dsum": ds.clone()}
        hc.hc_rms_norm_grad(v["dout"], s, w, v[name], dsum=v["dsum"])
        assert torch.equal(v[name], dx), name


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("d", [1, 3, 65, 129, 257, 511, 513, 1025, 2049, 4097, 4353, 8193, 8707, 16385, 16901])
def test_gradient_onto_its_addend(d, dtype):
    """dx is dsum, dout or h where a row's last vector, moved back to its end, is
    another wave's than the one before it, and where it is the same's."""
    g = gen(d)
    dy, h, ds = (rows(g, 19, d, dtype) for _ in range(3))
    w, dx = torch.randn(d, generator=g, device="cuda"), torch.empty_like(dy)
    hc.hc_rms_norm_grad(dy, h, w, dx, dsum=ds)
    for i in range(3):
        v = [dy.clone(), h.clone(), ds.clone()]
        hc.hc_rms_norm_grad(v[0], v[1], w, v[i], dsum=v[2])
        assert torch.equal(v[i], dx), i


def grads64(dy, h, w, eps, ds):
    """By torch's differentiation of the formula in 64 bits, and the sums of
    magnitudes that the roundings are relative to."""
    h, w, dy = h.double().cpu().requires_grad_(), w.double().cpu().requires_grad_(), dy.double().cpu()
    r = 1.0 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    (h * r * w * dy).sum().backward()
    dx = h.grad if ds is None else h.grad + ds.double().cpu()
    h, w, r = h.detach(), w.detach(), r.detach()
    size = r * (dy * w).abs() + h.abs() * r ** 3 * (dy * w * h).abs().mean(1, keepdim=True)
    return dx, size, (dy * h * r).sum(0), (dy * h * r).abs().sum(0)


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("types", [(F, F, F), (B, B, B), (B, F, F), (F, B, F)])
@pytest.mark.parametrize("d", [1, 3, 8, 31, 64, 100, 256, 513, 1031, 2048, 4096, 4100, 8195, 20000, 32768])
def test_gradient(d, types, dsum):
    dtype, wtype, dwtype = types
    g = gen(d)
    for t in (1, 70) if d < 5000 else (3,):
        h, dy = rows(g, t, d, dtype, 1.0, d + 3, 1), rows(g, t, d, dtype, 0.1, d + 1, 0)
        ds = rows(g, t, d, dtype, 0.1) if dsum else None
        w = torch.randn(d, generator=g, device="cuda").to(wtype)
        buf, dx = guarded((t, d), dtype, d + 3, 1)
        wbuf, dw = guarded((d,), dwtype, offset=1)
        ws = space(hc.hc_rms_norm_grad_workspace_bytes(t, d))
        hc.hc_rms_norm_grad(dy, h, w, dx, dw, ws, dsum=ds, eps=1e-5)
        want, size, wdw, wsize = grads64(dy, h, w, 1e-5, ds)
        # the dot product as the sum of squares, 57 roundings, and three times r's: under 200
        add = 0 if ds is None else ds.double().cpu().abs() * 2 * U
        close(dx, want, size * 200 * U + add + want.abs() * HALF[dtype] + TINY[dtype], f"dx {t} x {d}")
        # t products with r, added in some order
        tol = wsize * (R + (t + 4) * U)
        close(dw, wdw, tol + wdw.abs() * HALF[dwtype] + TINY[dwtype], f"dw {t} x {d}")
        only = torch.empty_like(dx)
        hc.hc_rms_norm_grad(dy, h, w, only, dsum=ds, eps=1e-5)            # without the weight's
        assert torch.equal(only, dx)
        old = torch.randn(d, generator=g, device="cuda").to(dwtype)
        more = old.clone()
        hc.hc_rms_norm_grad(dy, h, w, only, more, ws, dsum=ds, eps=1e-5, accumulate=True)
        total = old.double().cpu() + wdw
        close(more, total, tol + total.abs() * (U + HALF[dwtype]) + TINY[dwtype], "accumulated")
        check_guards(buf, dx)
        check_guards(wbuf, dw)


def test_gradient_against_differences():
    """The formula that the other tests take their gradient from, by central
    differences of the norm in 64 bits."""
    g = gen(5)
    h, w = torch.randn((4, 37), generator=g, device="cuda"), torch.randn(37, generator=g, device="cuda")
    dy = torch.randn((4, 37), generator=g, device="cuda")
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    hc.hc_rms_norm_grad(dy, h, w, dx, dw, space(hc.hc_rms_norm_grad_workspace_bytes(4, 37)), eps=1e-3)

    def loss(h, w):
        return float((norm64(h, None, w, 1e-3)[3] * dy.double().cpu()).sum())

    for at in ((0, 0), (1, 36), (3, 17)):
        e = torch.zeros((4, 37), dtype=torch.float64, device="cuda")
        e[at] = 1e-5
        diff = (loss(h.double() + e, w) - loss(h.double() - e, w)) / 2e-5
        assert abs(diff - float(dx[at])) <= 1e-5
        diff = (loss(h, w.double() + e[at[0]]) - loss(h, w.double() - e[at[0]])) / 2e-5
        assert abs(diff - float(dw[at[1]])) <= 1e-5


def test_many_rows_and_the_same_bits_again():
    """More rows than workgroups that sum the weight's gradient, and twice the
    same bits; no rows at all."""
    g = gen(7)
    for t, d in ((5000, 64), (4099, 600), (3001, 2048)):
        h, dy, w = rows(g, t, d, B), rows(g, t, d, B), torch.randn(d, generator=g, device="cuda")
        dx, dw = torch.empty_like(h), torch.empty_like(w)
        ws = space(hc.hc_rms_norm_grad_workspace_bytes(t, d))
        hc.hc_rms_norm_grad(dy, h, w, dx, dw, ws)
        want, size, wdw, wsize = grads64(dy, h, w, 1e-6, None)
        close(dx, want, size * 200 * U + want.abs() * HALF[B] + TINY[B], "dx")
        close(dw, wdw, wsize * (R + 200 * U), "dw")       # at most 100 rows in a lane, 64 partials in a lane, 16 lanes
        first = (dx.clone(), dw.clone())
        ws.fill_(0x3C)
        hc.hc_rms_norm_grad(dy, h, w, dx, dw, ws)
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
    none = torch.empty((0, 64), device="cuda")
    dw = torch.full((64,), GUARD, device="cuda")
    hc.hc_rms_norm(none, dw, none)
    hc.hc_rms_norm_8bit(none, dw, none.to(E4M3), torch.empty((0, 1), device="cuda"))
    hc.hc_rms_norm_grad(none, none, dw.clone(), none, dw, accumulate=True)
    assert bool((dw == GUARD).all())
    hc.hc_rms_norm_grad(none, none, dw.clone(), none, dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("d", [1031, 2048, 5000])
@pytest.mark.parametrize("dtype", [F, B])
def test_large_batches_as_small_ones(d, dtype):
    """Past 128 MiB rows are streamed: the same bits as of the rows in parts."""
    g = gen(d)
    t = (160 << 20) // (d * (4 if dtype == F else 2))
    x, res = (torch.randn((t, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.randn(d, generator=g, device="cuda")
    out, s, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    q, scales = torch.empty((t, d), dtype=E4M3, device="cuda"), torch.empty((t, -(-d // 128)), device="cuda")
    s8 = torch.empty_like(x)
    hc.hc_rms_norm(x, w, out, residual=res, sum_out=s)
    hc.hc_rms_norm_8bit(x, w, q, scales, group=128, residual=res, sum_out=s8)
    hc.hc_rms_norm_grad(x, s, w, dx, dsum=res)
    assert torch.equal(s, s8)
    part = t // 7 + 1
    for a in range(0, t, part):
        b = slice(a, min(t, a + part))
        o, h, o8, c = torch.empty_like(x[b]), torch.empty_like(x[b]), torch.empty_like(q[b]), torch.empty_like(scales[b])
        hc.hc_rms_norm(x[b], w, o, residual=res[b], sum_out=h)
        assert torch.equal(o, out[b]) and torch.equal(h, s[b])
        hc.hc_rms_norm_8bit(x[b], w, o8, c, group=128, residual=res[b])
        assert torch.equal(o8.view(torch.uint8), q[b].view(torch.uint8)) and torch.equal(c, scales[b])
        hc.hc_rms_norm_grad(x[b], h, w, o, dsum=res[b])
        assert torch.equal(o, dx[b])


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes and elements in."""
    t, d, stride = 3, 100, (1 << 31) + 11
    base = torch.zeros(2 * stride + d, dtype=B, device="cuda")
    x = torch.as_strided(base, (t, d), (stride, 1))
    v = torch.randn((t, d), device="cuda").to(B)
    x.copy_(v)
    w, out, want = torch.ones(d, device="cuda"), torch.empty((t, d), dtype=B, device="cuda"), torch.empty_like(v)
    hc.hc_rms_norm(x, w, out)
    hc.hc_rms_norm(v, w, want)
    assert torch.equal(out, want)
    hc.hc_rms_norm(v, w, x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("q8", [False, True])
def test_captured_and_on_a_stream(q8):
    g = gen(9)
    x, res, w = rows(g, 40, 1000, B), rows(g, 40, 1000, B), torch.randn(1000, generator=g, device="cuda")
    s = torch.empty_like(x)
    out = torch.empty((40, 1000), dtype=E4M3 if q8 else B, device="cuda")
    scales = torch.empty((40, 8), device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = space(hc.hc_rms_norm_grad_workspace_bytes(40, 1000))

    def step(**k):
        if q8:
            hc.hc_rms_norm_8bit(x, w, out, scales, group=128, residual=res, sum_out=s, **k)
        else:
            hc.hc_rms_norm(x, w, out, residual=res, sum_out=s, **k)
        hc.hc_rms_norm_grad(x, s, w, dx, dw, ws, dsum=res, **k)

    outs = [out, s, dx, dw] + ([scales] if q8 else [])
    step()
    want = [o.clone() for o in outs]
    raw = lambda o: o.view(torch.uint8) if o.dtype == E4M3 else o  # noqa: E731
    side = torch.cuda.Stream()
    for k in ({"stream": side}, {"stream": side.cuda_stream}):
        for o in outs:
            raw(o).zero_()
        torch.cuda.synchronize()
        step(**k)
        side.synchronize()
        assert all(torch.equal(raw(a), raw(b)) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keep = x.clone()
    for i in range(3):
        x.copy_(keep * (1 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        assert all(torch.equal(raw(a), raw(b)) for a, b in zip(got, outs)), i


def test_8_bits_at_the_end_of_the_range():
    """Groups whose largest product lies within 2^4 of fp32's end, rows whose root
    mean square does, and a row of zeroes with an eps of 0."""
    g = gen(13)
    d = 384
    for dtype in (F, B):
        for e, we in ((126, 0), (124, 2), (60, 66), (117, 0), (121, 0), (100, 25), (100, -90), (-60, -62)):
            x = (torch.rand((5, d), generator=g, device="cuda") * 1.9 + 0.05).mul_(2.0 ** e).to(dtype)
            w = torch.ones(d, device="cuda").mul_(2.0 ** we)
            x[1, 128:256] *= 2.0 ** -20                       # a group of smaller values beside the others
            x[2] *= -1
            q, s = torch.empty((5, d), dtype=E4M3, device="cuda"), torch.empty((5, 3), device="cuda")
            hc.hc_rms_norm_8bit(x, w, q, s, group=128, eps=0.0)
            _, _, r, _ = norm64(x, None, w, 0.0)
            prod = (x.float() * w).cpu().view(5, 3, 128)
            a = prod.abs().amax(2, keepdim=True)
            # 448 / a of a below 2^-119 is past fp32: both 2^64 times as large
            up = torch.where(a < 2.0 ** -64, 2.0 ** 64, 1.0)
            codes = (prod * up * (torch.full_like(a, 448.0) / (a * up))).view(5, d).to(E4M3).float()
            assert bool((q.cpu().float() == codes).all()), (dtype, e, we)
            # r below 2^-126 is off by half a step of the smallest numbers more
            want = a[..., 0].double() * r / 448.0
            close(s, want, want * (R + 3 * U + 2.0 ** -150 / r) + TINY[F], (dtype, e, we))
        for d0 in (3, 300, 4096, 20001):
            n = -(-d0 // 128)
            x, w = torch.zeros((2, d0), device="cuda").to(dtype), torch.ones(d0, device="cuda")
            q = torch.full((2, d0), 0x55, dtype=torch.uint8, device="cuda")
            for group in (0, 128):
                s = torch.full((2, n if group else 1), GUARD, device="cuda")
                hc.hc_rms_norm_8bit(x, w, q, s, group=group, eps=0.0)
                assert bool((s == 0).all()) and bool((q & 0x7F == 0).all()), (dtype, d0, group)


@pytest.mark.parametrize("d", [2, 20, 64, 300, 1000, 2560, 4096, 9001, 20001])
@pytest.mark.parametrize("dtype", [F, B])
def test_gradient_of_large_rows(d, dtype):
    """Rows whose squares, and whose products with the gradient, pass what fp32
    holds, beside others, in the same wave too."""
    g = gen(d + 1)
    for e in (62, 70, 100, 118, 124):
        t = 7
        h = (torch.rand((t, d), generator=g, device="cuda") + 0.5).mul_(2.0 ** e).to(dtype)
        h[1::2] *= 2.0 ** -e
        dy = (torch.rand((t, d), generator=g, device="cuda") + 0.5).to(dtype)
        w = torch.rand(d, generator=g, device="cuda") + 0.5
        dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
        hc.hc_rms_norm_grad(dy, h, w, dx, dw, space(hc.hc_rms_norm_grad_workspace_bytes(t, d)), eps=1e-6)
        want, size, wdw, wsize = grads64(dy, h, w, 1e-6, None)
        # with the roundings of r and of the mean among the smallest numbers, and
        # the latter's product with h and r
        r = 1.0 / (h.double().cpu().square().mean(1, keepdim=True) + 1e-6).sqrt()
        tol = size * (200 * U + 2.0 ** -149 / r) + h.double().cpu().abs() * r * 2.0 ** -149
        close(dx, want, tol + want.abs() * HALF[dtype] + 4 * TINY[dtype], f"dx 2^{e}")
        close(dw, wdw, wsize * (R + (t + 4) * U + 2.0 ** -150 / float(r.min())), f"dw 2^{e}")


@pytest.mark.parametrize("d", [2, 20, 64, 300, 1000, 2560, 4096, 9001, 20001])
@pytest.mark.parametrize("dtype", [F, B])
def test_tiny_rows_and_a_tiny_eps(d, dtype):
    """Rows whose squares fall below fp32's smallest numbers, where eps is 0 or as
    small as they are: the norm, its 8 bits' scales and the gradient."""
    g = gen(d + 2)
    for e, eps in ((-45, 0.0), (-62, 0.0), (-72, 0.0), (-72, 2.0 ** -142), (-100, 0.0), (-100, 2.0 ** -149), (-120, 0.0)):
        t = 7
        h = torch.randn((t, d), generator=g, device="cuda").mul_(2.0 ** e).to(dtype)
        h[1::2] *= 2.0 ** -e
        h[::2, 0] = 2.0 ** e                                    # no row of zeroes
        w = torch.rand(d, generator=g, device="cuda") + 0.5
        out = torch.empty_like(h)
        hc.hc_rms_norm(h, w, out, eps=eps)
        _, _, r, y = norm64(h, None, w, eps)
        close(out, y, y.abs() * (R + 3 * U + HALF[dtype]) + TINY[dtype], f"2^{e}")
        q, s = torch.empty((t, d), dtype=E4M3, device="cuda"), torch.empty((t, 1), device="cuda")
        hc.hc_rms_norm_8bit(h, w, q, s, eps=eps)
        want = (h.float() * w).abs().amax(1, keepdim=True).double().cpu() * r / 448
        close(s, want, want * (R + 3 * U) + TINY[F], f"scales 2^{e}")
        assert bool((q.float().abs().amax(1) == 448).all())
        value = q.cpu().double() * s.cpu().double()
        close(value, y, y.abs() * (2.0 ** -4 + R + 6 * U) + s.cpu().double() * 2.0 ** -10 * 1.01, f"8 bits 2^{e}")
        dy = torch.randn((t, d), generator=g, device="cuda").mul_(2.0 ** -20).to(dtype)
        dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
        hc.hc_rms_norm_grad(dy, h, w, dx, dw, space(hc.hc_rms_norm_grad_workspace_bytes(t, d)), eps=eps)
        want, size, wdw, wsize = grads64(dy, h, w, eps, None)
        close(dx, want, size * 200 * U + want.abs() * HALF[dtype] + TINY[dtype], f"dx 2^{e}")
        close(dw, wdw, wsize * (R + (t + 4) * U), f"dw 2^{e}")


@pytest.mark.parametrize("d", [2, 20, 64, 120, 250, 500])
@pytest.mark.parametrize("dtype", [F, B])
def test_rows_beside_far_ones_keep_their_bits(d, dtype):
    """Rows of one wave, some of which are summed twice: the others are as they
    are alone."""
    g = gen(d + 3)
    x, dy, w = rows(g, 64, d, dtype), rows(g, 64, d, dtype), torch.rand(d, generator=g, device="cuda") + 0.5
    far = x.clone()
    far[1::4] *= 2.0 ** 100
    far[2::4] *= 2.0 ** -100
    out = []
    for h in (x, far):
        y, q = torch.empty_like(h), torch.empty((64, d), dtype=E4M3, device="cuda")
        s, dx = torch.empty((64, -(-d // 32)), device="cuda"), torch.empty_like(h)
        hc.hc_rms_norm(h, w, y, eps=0.0)
        hc.hc_rms_norm_8bit(h, w, q, s, group=32, eps=0.0)
        hc.hc_rms_norm_grad(dy, h, w, dx, eps=0.0)
        out.append([v.view(16, 4, -1)[:, ::3] for v in (y, q.view(torch.uint8), s, dx)])
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("t,d,dtype", [(600, 2560, F), (2100, 4096, B), (700, 8195, B), (300, 20001, F), (300, 20001, B),
                                       (1100, 6000, B), (1300, 520, F), (9000, 256, B)])
def test_more_rows_than_workgroups(t, d, dtype):
    """Every layout with more rows than workgroups: the weight's gradient over all
    of a workgroup's rows, and dx onto what the next row's loads run ahead of."""
    g = gen(t + d)
    dy, h, ds = (rows(g, t, d, dtype) for _ in range(3))
    w = torch.randn(d, generator=g, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(d, device="cuda")
    ws = space(hc.hc_rms_norm_grad_workspace_bytes(t, d))
    hc.hc_rms_norm_grad(dy, h, w, dx, dw, ws, dsum=ds)
    want, size, wdw, wsize = grads64(dy, h, w, 1e-6, ds)
    add = ds.double().cpu().abs() * 2 * U
    close(dx, want, size * 200 * U + add + want.abs() * HALF[dtype] + TINY[dtype], "dx")
    close(dw, wdw, wsize * (R + (t + 4) * U) + TINY[F], "dw")
    for i in range(3):
        v = [dy.clone(), h.clone(), ds.clone()]
        again = torch.empty_like(dw)
        hc.hc_rms_norm_grad(v[0], v[1], w, v[i], again, ws, dsum=v[2])
        assert torch.equal(v[i], dx) and torch.equal(again, dw), i
