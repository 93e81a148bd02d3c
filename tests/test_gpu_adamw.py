"""An AdamW step over many tensors on the GPU, states in 32 and in 8 bits,
against the formula in 64 bits on the CPU.

U = 2^-24 is half a step of fp32.  The step's own numbers (betas, rate, the
factor of the gradient) are fp32 of 64-bit values: U each.  g' has 2 roundings
before the factor's 5 (norm, sum, quotient, product, scale), m and v add 3 and 5
of their own, the quotient and its root 8: under 24 U of each term."""
import math

import pytest
import torch

from collective_communication_amd import binding as hc
from test_gpu_step_ops import B, F, GUARD, HALF, TINY, U, close, gen

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BLOCK = hc.HC_STATE_BLOCK
LOW = 0xFFFFFFFF


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0xB7E15163) & LOW
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & LOW
    return x ^ (x >> 16)


def random_bits(seed, step, tensor, n):
    key = mix(mix(mix(mix(seed & LOW) ^ (seed >> 32)) ^ (step & LOW)) ^ tensor)
    return mix((mix(key) + torch.arange(n) * 0x9E3779B9) & LOW)


class Case:
    """Tensors with guards around each, their states, and what the step makes of them."""

    def __init__(self, sizes, ptypes, gtypes, bits, seed=0, copies=False, offset=3):
        g = gen(seed)
        self.sizes, self.bits = sizes, bits
        self.buffers = []

        def make(n, dtype, fill):
            buf = torch.full((n + 8 + offset,), 0.0, device="cuda").to(dtype)
            raw = buf.view(torch.uint8) if dtype == E4M3 else buf
            raw.fill_(0x55 if dtype == E4M3 else GUARD)
            view = buf[offset:offset + n]
            (view.view(torch.uint8) if dtype == E4M3 else view).copy_(
                fill.to(dtype).view(torch.uint8) if dtype == E4M3 else fill.to(dtype))
            self.buffers.append((raw, offset, n))
            return view

        rand = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        types = [(ptypes[i % len(ptypes)], gtypes[i % len(gtypes)]) for i in range(len(sizes))]
        self.params = [make(n, p, rand(n)) for n, (p, _) in zip(sizes, types)]
        self.grads = [make(n, q, rand(n) * 0.01) for n, (_, q) in zip(sizes, types)]
        self.ms = self.vs = None
        if bits == 32:
            self.m = [make(n, F, rand(n) * 0.003) for n in sizes]
            self.v = [make(n, F, (rand(n) * 0.01).square()) for n in sizes]
        else:
            self.m = [make(n, E4M3, (rand(n) * 60).clamp(-448, 448)) for n in sizes]
            self.v = [make(n, E4M3, (rand(n).abs() * 60).clamp(0, 448)) for n in sizes]
            blocks = [-(-n // BLOCK) for n in sizes]
            self.ms = [make(b, F, torch.rand(b, generator=g, device="cuda") * 1e-4) for b in blocks]
            self.vs = [make(b, F, torch.rand(b, generator=g, device="cuda") * 1e-4) for b in blocks]
        self.copies = [make(n, B, rand(n)) if p.dtype == F and i % 3 else None
                       for i, (n, p) in enumerate(zip(sizes, self.params))] if copies else None
        self.decays = [float(i % 2) for i in range(len(sizes))]

    def plan(self, **k):
        scales = {} if self.bits == 32 else {"m_scales": self.ms, "v_scales": self.vs}
        return hc.AdamWPlan(self.params, self.grads, self.m, self.v, copies=self.copies, decays=self.decays, **scales, **k)

    def state64(self, i):
        m, v = self.m[i].cpu().float().double(), self.v[i].cpu().float().double()
        if self.bits == 8:
            at = torch.arange(m.numel()) // BLOCK
            m = m * self.ms[i].cpu().double()[at]
            v = (v * self.vs[i].cpu().double()[at]).square()
        return m, v

    def check_guards(self):
        for raw, at, n in self.buffers:
            mark = 0x55 if raw.dtype == torch.uint8 else GUARD
            assert bool((raw[:at] == mark).all()) and bool((raw[at + n:] == mark).all())


def want64(case, i, step, lr, betas, eps, wd, scale=1.0, norm=None, max_norm=1.0):
    c = scale if norm is None else scale * min(1.0, max_norm / (abs(scale) * norm + 1e-6))
    p, g = case.params[i].double().cpu(), case.grads[i].double().cpu() * c
    m0, v0 = case.state64(i)
    m = betas[0] * m0 + (1 - betas[0]) * g
    v = betas[1] * v0 + (1 - betas[1]) * g * g
    msize = betas[0] * m0.abs() + (1 - betas[0]) * g.abs()
    den = (v / (1 - betas[1] ** step)).sqrt() + eps
    rate = lr / (1 - betas[0] ** step)
    new = p * (1 - lr * wd * case.decays[i]) - rate * m / den
    return m, v, new, msize, p.abs(), rate * msize / den


SIZES = [1, 0, 5, 127, 128, 129, 1000, 4095, 4096, 4097, 8192, 12_345, 3, 64, 40_000]
HYPER = dict(lr=0.01, betas=(0.9, 0.99), eps=1e-6)


def check_params(case, i, w, seeded, what):
    m, v, new, msize, psize, ssize = w
    p = case.params[i]
    tol = psize * 4 * U + ssize * 24 * U
    half = HALF[p.dtype] * (2 if seeded and p.dtype == B else 1)
    close(p, new, tol + new.abs() * half * 1.01 + TINY[p.dtype], what)
    if case.copies and case.copies[i] is not None:
        assert torch.equal(case.copies[i], p.bfloat16()), what


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("types", [((F,), (F,)), ((B,), (B,)), ((B, F), (F, B, B)), ((F, B), (F,))])
@pytest.mark.parametrize("offset", [0, 3])
def test_states_of_32_bits(types, clip, offset):
    case = Case(SIZES, *types, 32, copies=True, offset=offset)
    more = dict(scale=0.25, norm=3.0, max_norm=0.5) if clip else {}
    want = [want64(case, i, 7, HYPER["lr"], HYPER["betas"], HYPER["eps"], 0.1, **more) for i in range(len(SIZES))]
    call = dict(grad_scale=0.25, d_norm=torch.full((1,), 3.0, device="cuda"), max_norm=0.5) if clip else {}
    grads = [x.clone() for x in case.grads]
    hc.hc_adamw(case.plan(), 7, weight_decay=0.1, **HYPER, **call)
    for i, w in enumerate(want):
        close(case.m[i], w[0], w[3] * 12 * U + TINY[F], f"m {i}")
        close(case.v[i], w[1], w[1] * 24 * U + TINY[F], f"v {i}")
        check_params(case, i, w, False, f"p {i}")
        assert torch.equal(case.grads[i], grads[i])
    case.check_guards()


@pytest.mark.parametrize("seed", [0, 0x123456789ABCDEF])
@pytest.mark.parametrize("types", [((F,), (F,)), ((B,), (B,)), ((B, F), (F, B, B))])
@pytest.mark.parametrize("offset", [0, 3])
def test_states_of_8_bits(types, seed, offset):
    case = Case(SIZES, *types, 8, copies=True, offset=offset)
    want = [want64(case, i, 3, HYPER["lr"], HYPER["betas"], HYPER["eps"], 0.1) for i in range(len(SIZES))]
    hc.hc_adamw(case.plan(), 3, weight_decay=0.1, seed=seed, **HYPER)
    for i, w in enumerate(want):
        n = SIZES[i]
        check_params(case, i, w, seed != 0, f"p {i}")
        bits = random_bits(seed, 3, i, n)
        # the cancellation in m makes its rounding relative to msize, the root's is relative
        for codes, scales, x, err, cut in ((case.m[i], case.ms[i], w[0], w[3] * 14 * U, 0),
                                           (case.v[i], case.vs[i], w[1].sqrt(), w[1].sqrt() * 16 * U, 16)):
            if not n:
                continue
            pad = lambda y: torch.nn.functional.pad(y, (0, -n % BLOCK)).view(-1, BLOCK)  # noqa: E731
            top = pad(x.abs()).amax(1)
            close(scales, top / 448, (pad(err).amax(1) + top * 2 * U) / 448, f"scales {i}")
            unit = (top / 448).repeat_interleave(BLOCK)[:n]
            q = codes.cpu().float().double()
            lo, hi = ((x + s * (err + x.abs() * 4 * U)) / unit for s in (-1, 1))
            if seed:
                u = (((bits >> cut) & 0xFFFF).double() + 0.5) / 65536

                def cut_at(y):
                    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
                    return torch.copysign(torch.floor(y.abs() / step + u) * step, y).clamp(-448, 448)

                lo, hi = cut_at(lo), cut_at(hi)
            else:
                lo, hi = (y.clamp(-448, 448).float().to(E4M3).double() for y in (lo, hi))
            if cut:
                lo, hi = lo.clamp(min=2.0 ** -9), hi.clamp(min=2.0 ** -9)
            # fp32 before fp8 in the bounds may round a value next to a border once more: by one part in 2^24
            bad = (q < torch.minimum(lo, hi)) | (q > torch.maximum(lo, hi))
            assert not bool(bad.any()), f"{i}: {int(bad.sum())} codes of {n}"
    case.check_guards()


@pytest.mark.parametrize("seed", [0, 77])
def test_states_by_single_operations(seed):
    """m, v and the 8-bit codes are those of the operations as they are written,
    each rounded once to fp32: numpy's, bit for bit."""
    import numpy as np

    f = np.float32
    n = 200_000
    for bits in (8, 32):
        case = Case([n], (F,), (B,), bits, seed=12, offset=0)
        g = case.grads[0].float().cpu().numpy() * f(0.25)
        m, v = case.m[0].float().cpu().numpy(), case.v[0].float().cpu().numpy()
        at = np.arange(n) // BLOCK
        if bits == 8:
            m = m * case.ms[0].cpu().numpy()[at]
            v = v * case.vs[0].cpu().numpy()[at]
            v = v * v
        b1, a1, b2, a2 = f(0.9), f(1 - 0.9), f(0.99), f(1 - 0.99)
        m = b1 * m + a1 * g
        v = b2 * v + a2 * (g * g)
        hc.hc_adamw(case.plan(), 4, lr=1e-3, betas=(0.9, 0.99), grad_scale=0.25, seed=seed)
        if bits == 32:
            assert np.array_equal(case.m[0].cpu().numpy(), m) and np.array_equal(case.v[0].cpu().numpy(), v)
            continue
        draw = random_bits(seed, 4, 0, n).numpy()
        for x, codes, scales, cut in ((m, case.m[0], case.ms[0], 0), (np.sqrt(v), case.v[0], case.vs[0], 16)):
            pad = np.zeros(-(-n // BLOCK) * BLOCK, f)
            pad[:n] = x
            unit = np.abs(pad).reshape(-1, BLOCK).max(1) * f(f(1) / f(448))
            assert np.array_equal(scales.cpu().numpy(), unit)
            y = np.clip(x / unit[at], f(-448), f(448))
            if seed:
                u = ((draw >> cut & 0xFFFF) + 0.5) / 65536
                a = np.abs(y).astype(np.float64)
                step = np.exp2(np.clip(np.frexp(a)[1] - 1, -6, None) - 3.0)
                y = np.copysign(np.minimum(np.floor(a / step + u) * step, 448), y)
            y = torch.from_numpy(np.asarray(y, f)).to(E4M3).float().numpy()
            if cut:
                y = np.where((x > 0) & (y == 0), f(2.0 ** -9), y)
            assert np.array_equal(codes.cpu().float().numpy(), y), int((codes.cpu().float().numpy() != y).sum())


def test_two_plans_of_the_same_tensors_and_two_streams():
    """Plans of one set of tensors may be used in turn, and two of disjoint
    tensors at once."""
    a, b = (Case([70_000, 333], (F, B), (F,), 8, seed=s) for s in (1, 2))
    c, d = (Case([70_000, 333], (F, B), (F,), 8, seed=s) for s in (1, 2))
    pa, pa2, pb, pc, pd = a.plan(), a.plan(), b.plan(), c.plan(), d.plan()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in range(1, 6):
        hc.hc_adamw(pa if t % 2 else pa2, t, seed=t, stream=one, **HYPER)
        hc.hc_adamw(pb, t, seed=t, stream=two, **HYPER)
    torch.cuda.synchronize()
    for t in range(1, 6):
        hc.hc_adamw(pc, t, seed=t, **HYPER)
        hc.hc_adamw(pd, t, seed=t, **HYPER)
    assert all(torch.equal(x[0], y[0]) for p, q in ((a, c), (b, d)) for x, y in zip(p.buffers, q.buffers))


def test_bf16_parameters_by_random_bits():
    """Rounded up with the probability of what is cut off, by the bits that the
    definition names; the mean stays."""
    n = 100_000
    case = Case([n], (B,), (F,), 32, offset=0)
    w = want64(case, 0, 2, 1e-4, (0.9, 0.99), 1e-6, 0.0)
    plan = case.plan()
    keep = [x.clone() for x in (case.params[0], case.m[0], case.v[0])]
    hc.hc_adamw(plan, 2, lr=1e-4, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.0, seed=99)
    got = case.params[0].double().cpu()
    bits = ((random_bits(99, 2, 0, n) * 0x9E3779B9) & LOW) >> 16
    down = torch.exp2(torch.floor(torch.log2(w[2].abs())) - 7)          # a bf16 step
    place = w[2].abs() / down
    frac = place - place.floor()
    up = frac + bits.double() / 65536 >= 1.0
    near = (frac + bits.double() / 65536 - 1.0).abs() < 1e-3           # fp32 has 16 bits of what is cut off
    want = torch.copysign((place.floor() + up) * down, w[2])
    assert bool(((got == want) | near).all())
    off = ((got - w[2]) / down)
    assert abs(float(off.mean())) < 5 * 0.5 / math.sqrt(n), "unbiased, within 5 deviations"
    for seed, step, same in ((99, 2, True), (98, 2, False), (99, 3, False)):
        for a, b in zip((case.params[0], case.m[0], case.v[0]), keep):
            a.copy_(b)
        hc.hc_adamw(plan, step, lr=1e-4, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.0, seed=seed)
        assert (int((case.params[0].double().cpu() != got).sum()) == 0) == same


def test_random_bits_keep_small_changes():
    """v of a constant gradient, from another size, over 400 steps: nearest
    rounding keeps it where it was, random bits follow in the mean."""
    n = 64 * BLOCK
    def run(seed):
        p, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
        g[::BLOCK] = 1.0                                   # each block's largest
        plan = hc.AdamWPlan.for_params([p], [g], state_bits=8)
        plan.exp_avg_sqs[0].copy_(torch.where(g == 1.0, 448.0, 112.0).to(E4M3))     # roots of 1 and 0.25
        plan.v_scales[0].fill_(1.0 / 448)
        for step in range(1, 401):
            hc.hc_adamw(plan, step, lr=0.0, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, seed=seed)
        root = plan.exp_avg_sqs[0].float() * plan.v_scales[0].repeat_interleave(BLOCK)
        return float(root[g == 0.5].square().mean().sqrt())

    assert run(0) == 0.25
    # 1 - 0.99^400 of the way in the square; a block's noise is a twelfth of a step, of 8128 values
    assert abs(run(7) - 0.5) < 0.02


def test_two_hundred_steps_like_the_formula():
    """Many steps in a row from zero states, 32 bits against 64, and the first
    step of 8 bits as of 32."""
    n = 5000
    g = gen(4)
    p = torch.randn(n, generator=g, device="cuda")
    first, grad = p.clone(), torch.empty(n, device="cuda")
    plan = hc.AdamWPlan.for_params([p], [grad])
    q, m, v = p.double().cpu(), torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    for t in range(1, 201):
        grad.copy_(torch.randn(n, generator=g, device="cuda"))
        hc.hc_adamw(plan, t, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
        d = grad.double().cpu()
        m, v = 0.9 * m + 0.1 * d, 0.95 * v + 0.05 * d * d
        q = q * (1 - 1e-4) - 1e-3 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.95 ** t)).sqrt() + 1e-8)
        if t == 1:
            other = first.clone()
            hc.hc_adamw(hc.AdamWPlan.for_params([other], [grad], state_bits=8), 1, lr=1e-3, betas=(0.9, 0.95), eps=1e-8,
                        weight_decay=0.1)
            close(other, q, q.abs() * 8 * U + 1e-3 * 30 * U, "8 bits")
    # 200 steps of at most 24 U of 3e-3 (a step's largest) and 4 U of a value below 5, each
    close(p, q, torch.full((n,), 200 * (24 * U * 3e-3 + 4 * U * 5.0), dtype=torch.float64), "200 steps")


def test_zero_odd_and_infinite_values():
    for bits in (8, 32):
        p = torch.ones(1000, device="cuda")
        g = torch.zeros(1000, device="cuda")
        g[500] = math.nan
        g[900] = 1e-30
        plan = hc.AdamWPlan.for_params([p], [g], state_bits=bits)
        hc.hc_adamw(plan, 1, lr=0.1, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0)
        assert math.isnan(float(p[500])) and bool((p[:384] == 1.0).all())
        assert bool((plan.exp_avgs[0][:384].float() == 0).all()) and bool((plan.exp_avg_sqs[0][:384].float() == 0).all())
        if bits == 32:
            assert bool((p[501:900] == 1.0).all())
        else:
            assert bool((plan.m_scales[0][:3] == 0).all()) and bool(plan.m_scales[0][3].isnan())
    # a root that is not 0 stays so beside one 2^30 times as large
    p, g = torch.zeros(128, device="cuda"), torch.full((128,), 2.0 ** -30, device="cuda")
    g[0] = 1.0
    for seed in (0, 5):
        plan = hc.AdamWPlan.for_params([p], [g], state_bits=8)
        hc.hc_adamw(plan, 1, lr=0.0, seed=seed)
        assert bool((plan.exp_avg_sqs[0].float() > 0).all())


def test_norm_that_is_no_number():
    for bits in (8, 32):
        for value in (math.inf, math.nan):
            case = Case([300, 5000], (F, B), (F,), bits)
            before = [raw.clone() for raw, _, _ in case.buffers]
            norm = torch.tensor([value], device="cuda")
            hc.hc_adamw(case.plan(), 1, d_norm=norm, max_norm=1.0, skip_nonfinite=True)
            assert all(torch.equal(a, b) for a, (b, _, _) in zip(before, case.buffers))
            hc.hc_adamw(case.plan(), 1, d_norm=norm, max_norm=1.0)
            assert bool(case.params[0].isnan().all()) == math.isnan(value)


def test_views_of_buckets_and_dimensions_in_another_order():
    g = gen(8)
    flat, gflat = torch.randn(100_000, generator=g, device="cuda"), torch.randn(100_000, generator=g, device="cuda")
    shapes = [(33, 77), (5, 6, 7), (1,), (200, 300), (17,)]
    def views(b, at=1):
        out = []
        for s in shapes:
            n = math.prod(s)
            out.append(b[at:at + n].view(s))
            at += n
        return out
    def run(order, bits, **k):
        b, q = flat.clone(), gflat.clone()
        params, grads = ([order(x) for x in views(y)] for y in (b, q))
        plan = hc.AdamWPlan.for_params(params, grads, state_bits=bits)
        for t in (1, 2):
            hc.hc_adamw(plan, t, lr=0.01, **k)
        return b
    for bits in (8, 32):
        a = run(lambda x: x, bits)
        assert torch.equal(a[:1], flat[:1]) and torch.equal(a[63_000:], flat[63_000:])
        assert torch.equal(run(lambda x: x.transpose(0, -1), bits), a)
    # a size-1 dimension's stride says nothing
    p, q = torch.randn((1, 8), device="cuda"), torch.randn((8, 1), device="cuda").t()
    hc.hc_adamw(hc.AdamWPlan.for_params([p], [q]), 1)


def test_many_tensors_and_the_same_bits_again():
    sizes = [(i * 7919) % 3000 for i in range(700)]
    for bits in (8, 32):
        a, b = (Case(sizes, (F, B), (B, F, F), bits, seed=2, copies=True) for _ in range(2))
        pa, pb = a.plan(), b.plan(table=torch.empty(hc.hc_adamw_table_bytes(700), dtype=torch.uint8, device="cuda"))
        for t in (1, 2):
            hc.hc_adamw(pa, t, seed=3, **HYPER)
            hc.hc_adamw(pb, t, seed=3, **HYPER)
        assert all(torch.equal(x[0], y[0]) for x, y in zip(a.buffers, b.buffers))
        a.check_guards()
    hc.hc_adamw(hc.AdamWPlan([], [], [], []), 1)
    empty = [torch.empty(0, device="cuda")]
    hc.hc_adamw(hc.AdamWPlan(empty, empty, empty, empty), 1)


def test_clipped_as_by_the_clipping_call():
    """hc_grad_norm and the step's own factor against hc_clip_grad_norm first."""
    for bits in (8, 32):
        a, b = (Case([3000, 500, 7], (F,), (F,), bits, seed=5) for _ in range(2))
        norm, ws = torch.empty(1, device="cuda"), torch.empty(hc.hc_grad_norm_workspace_bytes(3), dtype=torch.uint8,
                                                              device="cuda")
        hc.hc_grad_norm(a.grads, norm, ws)
        hc.hc_adamw(a.plan(), 1, d_norm=norm, max_norm=0.1, **HYPER)
        hc.hc_clip_grad_norm(b.grads, 0.1, norm, ws)
        hc.hc_adamw(b.plan(), 1, **HYPER)
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_with_the_step_on_the_device(bits):
    """A captured launch follows the step, the rate, the norm and the gradients."""
    a, b = (Case([5000, 130], (F, B), (F,), bits, seed=6, offset=0) for _ in range(2))
    step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 0.1, device="cuda")
    norm = torch.full((1,), 2.0, device="cuda")
    plan, other = a.plan(), b.plan()
    k = dict(betas=(0.9, 0.999), eps=1e-8, d_norm=norm, max_norm=0.5, seed=77)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_adamw(plan, step, lr=lr, **k)
        step.add_(1)
    g = gen(6)
    for t in range(1, 6):
        rate = 0.1 / t
        lr.fill_(rate)
        norm.fill_(2.0 + t)
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        hc.hc_adamw(other, t, lr=float(lr), **k)
        assert all(torch.equal(x[0], y[0]) for x, y in zip(a.buffers, b.buffers)), t
    assert int(step) == 6


def test_on_a_stream_given():
    a, b = (Case([5000, 130], (F, B), (F,), 8, seed=9) for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    hc.hc_adamw(a.plan(stream=side), 1, stream=side, **HYPER)
    side.synchronize()
    hc.hc_adamw(b.plan(), 1, **HYPER)
    assert all(torch.equal(x[0], y[0]) for x, y in zip(a.buffers, b.buffers))


def test_large_tensor():
    """Values past 2^31 of one tensor: their states, parameters and random bits."""
    n = (1 << 31) + 5000
    p, g = torch.zeros(n, dtype=B, device="cuda"), torch.zeros(n, dtype=B, device="cuda")
    g[-5000:] = 1.0
    plan = hc.AdamWPlan.for_params([p], [g], state_bits=8)
    hc.hc_adamw(plan, 1, lr=0.37, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, seed=11)
    assert bool((p[:-5000] == 0).all())
    got = p[-5000:].double().cpu()
    i = torch.arange(n - 5000, n)
    key = mix(mix(mix(mix(11) ^ 0) ^ 1) ^ 0)
    bits = mix((mix(key) + i * 0x9E3779B9) & LOW)
    low = 0.3691406250                      # 0.37 between two bf16 values 2^-9 apart
    up = (0.37 - low) * 512 + (((bits * 0x9E3779B9) & LOW) >> 16).double() / 65536
    want = -(low + (up >= 1.0).double() / 512)
    assert bool(((got == want) | ((up - 1.0).abs() < 1e-3)).all())
    m = plan.exp_avgs[0][-5000:].float() * plan.m_scales[0][-40:].repeat_interleave(BLOCK)[-5000:]
    close(m, torch.full((5000,), 0.1), torch.full((5000,), 0.1 * 8 * U), "m")


@pytest.mark.parametrize("bits", [8, 32])
def test_plan_on_a_stream_of_its_own(bits):
    """for_params and its first step on a stream that nothing else orders after
    the states' zeroes, and under another default type."""
    n = 1 << 24
    p, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    want = p.clone()
    hc.hc_adamw(hc.AdamWPlan.for_params([want], [g], state_bits=bits), 1)
    got = p.clone()
    junk = [torch.full((n,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk                                             # memory that the states may get
    side = torch.cuda.Stream()
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.bfloat16)
    try:
        plan = hc.AdamWPlan.for_params([got], [g], state_bits=bits, stream=side)
    finally:
        torch.set_default_dtype(before)
    hc.hc_adamw(plan, 1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_plans_made_and_dropped_while_streams_are_busy():
    """A plan made on a stream while kernels of the current one still write to
    memory that was freed there, stepped and dropped at once, and another use of
    what it had."""
    sizes = [5000, 130, 40_000]
    n = hc.hc_adamw_table_bytes(len(sizes))
    side = torch.cuda.Stream()
    assert side.stream_id != side.cuda_stream
    outside = torch.cuda.ExternalStream(side.cuda_stream)
    assert outside.stream_id == outside.cuda_stream       # how the binding tells torch's streams from others
    for bits in (8, 32):
        want = Case(sizes, (F, B), (F,), bits, seed=21)
        hc.hc_adamw(want.plan(), 1, **HYPER)
        for made, run in ((side, side), (side.cuda_stream, side.cuda_stream), (None, side), (side, None), (None, None)):
            case = Case(sizes, (F, B), (F,), bits, seed=21)
            torch.cuda.synchronize()
            junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
            torch.cuda._sleep(2_000_000)
            for j in junk:
                j.fill_(0)
            del junk, j
            plan = case.plan(stream=made)
            if made is not run:                           # the step after the table's writing
                torch.cuda.synchronize()
            with torch.cuda.stream(side if run is not None else torch.cuda.current_stream()):
                torch.cuda._sleep(2_000_000)
            hc.hc_adamw(plan, 1, stream=run, **HYPER)
            del plan
            junk = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
            with torch.cuda.stream(side):
                more = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
            torch.cuda.synchronize()
            del junk, more
            assert all(torch.equal(x[0], y[0]) for x, y in zip(case.buffers, want.buffers)), (bits, made, run)
    # states of for_params, dropped with a step pending
    g = gen(22)
    p, grad = torch.randn(100_000, generator=g, device="cuda"), torch.randn(100_000, generator=g, device="cuda")
    want = p.clone()
    hc.hc_adamw(hc.AdamWPlan.for_params([want], [grad]), 1)
    for made, run in ((side, side), (None, side)):
        got = p.clone()
        plan = hc.AdamWPlan.for_params([got], [grad], stream=made)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        hc.hc_adamw(plan, 1, stream=run)
        del plan
        junk = [torch.full((100_000,), math.nan, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(got, want), (made, run)


@pytest.mark.parametrize("eps", [1e-30, 0.0])
@pytest.mark.parametrize("seed", [0, 77])
def test_roots_of_the_smallest_second_moments(seed, eps):
    """Gradients whose squares are among fp32's smallest numbers, zeroes and
    ordinary ones between them: codes and scales by single operations, and the
    step as with states of 32 bits (without an eps no number where v is 0)."""
    import numpy as np

    f = np.float32
    n = 40_000
    rng = np.random.RandomState(3)
    size = np.repeat(10.0 ** rng.uniform(-23.5, -14, n // 125), 125)       # blocks that two sizes share, too
    size[::17] *= 1e-3
    g = (rng.standard_normal(n) * size).astype(f)
    g[::11] = 0
    g[5000:5200] = 1e-3
    p = torch.zeros(n, device="cuda")
    other = p.clone()
    grad = torch.from_numpy(g).cuda()
    plan = hc.AdamWPlan.for_params([p], [grad], state_bits=8)
    k = dict(lr=1e-3, betas=(0.9, 0.99), weight_decay=0.0, eps=eps)
    hc.hc_adamw(plan, 1, seed=seed, **k)
    hc.hc_adamw(hc.AdamWPlan.for_params([other], [grad]), 1, seed=seed, **k)
    v = f(1 - 0.99) * (g * g)
    root = np.sqrt(v)
    assert ((v > 0) & (v < f(2.0 ** -126))).sum() > 5000
    at = np.arange(n) // BLOCK
    pad = np.zeros(-(-n // BLOCK) * BLOCK, f)
    pad[:n] = root
    unit = pad.reshape(-1, BLOCK).max(1) * f(f(1) / f(448))
    off = plan.v_scales[0].cpu().numpy() != unit
    assert not off.any(), int(off.sum())
    y = np.divide(root, unit[at], out=np.zeros(n, f), where=unit[at] > 0)
    if seed:
        u = ((random_bits(seed, 1, 0, n).numpy() >> 16) + 0.5) / 65536
        a = y.astype(np.float64)
        step = np.exp2(np.clip(np.frexp(a)[1] - 1, -6, None) - 3.0)
        y = np.minimum(np.floor(a / step + u) * step, 448)
    y = torch.from_numpy(np.asarray(np.minimum(y, 448), f)).to(E4M3).float().numpy()
    y = np.where((root > 0) & (y == 0), f(2.0 ** -9), y)
    off = plan.exp_avg_sqs[0].cpu().float().numpy() != y
    assert not off.any(), int(off.sum())
    # the same m and root on both sides, a product, reciprocal and quotient apart: 8 U
    close(p, other, torch.where(other.isfinite(), other.abs() * 8 * U, 0.0) + TINY[F], "step")
