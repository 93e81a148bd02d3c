"""Cases and plain forms of the operators on either side of the exchange: an
AdamW step over many tensors with states in 32 or 8 bits, routing of tokens to
experts and its gradient, and the root-mean-square norm with the residual's
addition, its 8-bit output and its gradient.

``run`` computes them in elementary torch operations (``own`` false) or with
this package's kernels (``own`` true); both take what ``prepare`` gives.
``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_E4M3 = torch.float8_e4m3fn
BLOCK = 128           # values of a tensor that share a scale of their 8-bit states


# ---------------------------------------------------------------------------- cases

def _adamw(tensors, total, dtype, states, grads, copies, flat, clip, seeded):
    return {"kind": "adamw", "tensors": tensors, "total": total, "dtype": dtype, "states": states, "grads": grads,
            "copies": copies, "flat": flat, "clip": clip, "seeded": seeded}


def _route(kind, tokens, experts, k, scores, dtype, groups, top_groups, group_best, bias, renormalise, masked):
    return {"kind": kind, "tokens": tokens, "experts": experts, "k": k, "scores": scores, "dtype": dtype,
            "groups": groups, "top_groups": top_groups, "group_best": group_best, "bias": bias,
            "renormalise": renormalise, "masked": masked}


def _norm(kind, tokens, dim, dtype, wtype, residual, group):
    return {"kind": kind, "tokens": tokens, "dim": dim, "dtype": dtype, "wtype": wtype, "residual": residual,
            "group": group}


def listed():
    return [
        # the weights of one small block: a dozen separate tensors in fp32, where the launch counts
        dict(_adamw(12, 300_001, "f32", 32, "same", False, False, False, False), name="adamw_small_f32"),
        # one bucket of 2^25 weights with their gradients clipped on the way: fp32 vectors beside bf16 matrices
        dict(_adamw(290, 1 << 25, "mixed", 32, "f32", False, True, True, False), name="adamw_bucket_mixed"),
        # a whole model: 2^28 bf16 weights in separate tensors, states in 8 bits, rounded by random bits
        dict(_adamw(450, 1 << 28, "bf16", 8, "same", False, False, True, True), name="adamw_model_8bit"),
        # one decoding step of 64 sequences: 8 of 128 experts
        dict(_route("route", 64, 128, 8, "softmax", "bf16", 1, 1, 1, False, True, 0.0), name="route_decode_bf16"),
        # a pretraining micro-batch: sigmoid scores, a bias for balance, 8 of 256 experts out of 4 of 8 groups
        dict(_route("route", 32_768, 256, 8, "sigmoid", "f32", 8, 4, 2, True, True, 0.0), name="route_batch_groups_f32"),
        # its backward pass
        dict(_route("route_grad", 32_768, 256, 8, "sigmoid", "f32", 8, 4, 2, True, True, 0.0),
             name="route_grad_batch_f32"),
        # a padded batch over an odd number of experts, weights left as the softmax gives them
        dict(_route("route_grad", 9_999, 60, 4, "softmax", "bf16", 1, 1, 1, False, False, 0.2),
             name="route_grad_padded_bf16"),
        # one decoding step of 64 sequences: the residual added, rows in 8 bits
        dict(_norm("norm8", 64, 4096, "bf16", "bf16", True, 0), name="norm8_decode_bf16"),
        # a micro-batch of prompts: rows in 8 bits with a scale for every 128 columns
        dict(_norm("norm8", 16_384, 4096, "bf16", "bf16", True, 128), name="norm8_batch_bf16"),
        # a small model in fp32, a width that is no multiple of anything
        dict(_norm("norm", 5_003, 1031, "f32", "f32", False, 0), name="norm_odd_f32"),
        # the backward pass of a fine-tuning step's few tokens
        dict(_norm("norm_grad", 500, 2560, "f32", "f32", False, 0), name="norm_grad_small_f32"),
        # and of a pretraining micro-batch, with the gradient that arrives by the residual
        dict(_norm("norm_grad", 16_384, 4096, "bf16", "f32", True, 0), name="norm_grad_batch_bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi, *multiples):
    return max(lo, _log(rng, lo, hi) // (m := rng.choice(multiples)) * m)


def draw(rng):
    kind = rng.choice(("adamw", "adamw", "route", "route_grad", "norm", "norm8", "norm_grad"))
    dtype = rng.choice(("bf16", "f32"))
    while True:
        if kind == "adamw":
            tensors = _log(rng, 1, 600)
            dtype = rng.choice(("bf16", "f32", "mixed"))
            c = _adamw(tensors, _log(rng, 1000 * tensors, 1 << 28), dtype, rng.choice((8, 32)),
                       rng.choice(("same", "f32")), dtype != "bf16" and rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.5, rng.random() < 0.5)
        elif kind in ("route", "route_grad"):
            groups = rng.choice((1, 1, 4, 8))
            each = _log(rng, 4, 1024 // groups)
            top = rng.randint(max(1, groups // 4), groups)
            c = _route(kind, _log(rng, 1, 60_000), groups * each, rng.randint(1, min(16, top * each)),
                       rng.choice(("softmax", "sigmoid")), dtype, groups, top, rng.choice((1, 2)), rng.random() < 0.5,
                       rng.random() < 0.7, rng.choice((0.0, 0.0, 0.3)))
        else:
            residual = rng.random() < 0.6
            group = rng.choice((0, 64, 128)) if kind == "norm8" else 0
            c = _norm(kind, _log(rng, 1, 60_000), _width(rng, 32, 12_000, 1, 8, 64), dtype, rng.choice((dtype, "f32")),
                      residual, group)
        if work(c)["bytes"] <= 2.0e9:
            return c


def work(case):
    if case["kind"] == "adamw":
        n, total = 0, 0.0
        for size, t in _tensors(case):
            n += size
            total += size * (2 * _SIZE[t] + (4 if case["grads"] == "f32" else _SIZE[t]))
            total += size * (16 if case["states"] == 32 else 4 + 16 / BLOCK)
            total += 2 * size if case["copies"] and t == "f32" else 0
        return {"bytes": total, "flops": 14 * n}
    if case["kind"] in ("route", "route_grad"):
        t, e, k, es = case["tokens"], case["experts"], case["k"], _SIZE[case["dtype"]]
        if case["kind"] == "route":
            return {"bytes": t * (e * es + k * 8), "flops": t * e * 4}
        dense = case["scores"] == "softmax" and not case["renormalise"]
        return {"bytes": t * (e * es + k * 8 + (e if dense else k) * es), "flops": t * (k * 8 + (5 * e if dense else 0))}
    n, es = case["tokens"] * case["dim"], _SIZE[case["dtype"]]
    if case["kind"] == "norm_grad":
        return {"bytes": n * es * (4 if case["residual"] else 3) + 2 * case["dim"] * _SIZE[case["wtype"]], "flops": 10 * n}
    rows = n * es * (3 if case["residual"] else 1) + case["dim"] * _SIZE[case["wtype"]]
    if case["kind"] == "norm":
        return {"bytes": rows + n * es, "flops": 5 * n}
    return {"bytes": rows + n + 4 * case["tokens"] * _scales(case), "flops": 8 * n}


def _scales(case):
    """Scales of a row of 8-bit values: one for each group of columns, or one."""
    return -(-case["dim"] // case["group"]) if case["group"] else 1


# ---------------------------------------------------------------------------- inputs

def _tensors(case):
    """(size, type) of each tensor: sizes over a factor of 4096, as matrices stand beside vectors."""
    r = random.Random(case["tensors"] * 1_000_003 + case["total"])
    w = [math.exp(r.uniform(0.0, math.log(4096.0))) for _ in range(case["tensors"])]
    sizes = [int(case["total"] * x / sum(w)) for x in w]
    sizes[-1] += case["total"] - sum(sizes)
    middle = sorted(sizes)[len(sizes) // 2]
    return [(s, case["dtype"] if case["dtype"] != "mixed" else "f32" if s < middle else "bf16") for s in sizes]


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _views(flat, sizes, flatly):
    """A tensor's values each out of one buffer: one behind the other, or from addresses as an allocator gives them."""
    at, views = 0, []
    for n in sizes:
        views.append(flat[at:at + n])
        at += n if flatly else -(-n // 512) * 512 + 512
    return views


def _room(sizes, flatly):
    return sum(n if flatly else -(-n // 512) * 512 + 512 for n in sizes)


def _weights(case, g):
    parts, flatly = _tensors(case), case["flat"]
    sizes = {t: [n for n, of in parts if of == t] for t in _TYPES}
    grad = {t: "f32" if case["grads"] == "f32" else t for t in _TYPES}
    s = {"flat": {t: _normal(g, _room(sizes[t], flatly), _TYPES[t], 0.02) for t in _TYPES}}
    gflat = {t: _normal(g, _room(sizes[t], flatly), _TYPES[grad[t]], 1e-3) for t in _TYPES}
    views = {t: iter(_views(s["flat"][t], sizes[t], flatly)) for t in _TYPES}
    gviews = {t: iter(_views(gflat[t], sizes[t], flatly)) for t in _TYPES}
    s["params"] = [next(views[t]) for _, t in parts]
    s["grads"] = [next(gviews[t]) for _, t in parts]
    every = [n for n, _ in parts]
    # the states after some steps: a mean gradient, and squares over some orders of magnitude
    m = _normal(g, _room(every, flatly), torch.float32, 4e-4)
    root = _normal(g, m.numel(), torch.float32, 1.0).abs_().add_(0.02).mul_(1e-3)
    if case["states"] == 32:
        s["m"], s["v"] = m, root.square_()
        s["ms"], s["vs"] = _views(s["m"], every, flatly), _views(s["v"], every, flatly)
    else:
        s["m"], s["v"] = (x.div_(x.abs().max() / 400.0).to(_E4M3) for x in (m, root))
        s["ms"], s["vs"] = _views(s["m"], every, flatly), _views(s["v"], every, flatly)
        blocks = [-(-n // BLOCK) for n in every]
        s["mscale"] = torch.rand(sum(blocks), generator=g, device="cuda").add_(0.5).mul_(4e-6)
        s["vscale"] = torch.rand(sum(blocks), generator=g, device="cuda").add_(0.5).mul_(1e-5)
        s["mscales"], s["vscales"] = _views(s["mscale"], blocks, True), _views(s["vscale"], blocks, True)
    s["copies"] = None
    if case["copies"]:
        s["copy"] = s["flat"]["f32"].bfloat16()
        cviews = iter(_views(s["copy"], sizes["f32"], flatly))
        s["copies"] = [next(cviews) if t == "f32" else None for _, t in parts]
    s["norm"] = torch.full((1,), 2.5, device="cuda") if case["clip"] else None
    s.update(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, decay=0.1, step=20, scale=0.125, max_norm=0.25,
             seed=0x5DEECE66D17 + case["total"] if case["seeded"] else 0)
    # vectors are not decayed, matrices are
    middle = sorted(every)[len(every) // 2]
    s["decays"] = [0.0 if n < middle else 1.0 for n in every]
    return s


def _logits(case, g):
    """Scores before the softmax, some experts liked more than others; masked: a share of padding tokens, all -inf."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn((t, e), generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
    if case["masked"]:
        x[torch.rand(t, generator=g, device="cuda") < case["masked"]] = -math.inf
    return x.to(_TYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "adamw":
        return {**s, **_weights(case, g)}
    if case["kind"] in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        s["logits"] = _logits(case, g)
        s["bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        s["scale"] = 2.5 if case["scores"] == "sigmoid" else 1.0
        s["experts"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((t, k), dtype=torch.float32, device="cuda")
        if case["kind"] == "route_grad":
            s["experts"], _ = _choose(s)
            s["dweights"] = _normal(g, (t, k), torch.float32, 1e-2)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    t, d, dtype, wtype = case["tokens"], case["dim"], _TYPES[case["dtype"]], _TYPES[case["wtype"]]
    s["eps"] = 1e-6
    s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(wtype)
    s["x"] = _normal(g, (t, d), dtype)
    s["residual"] = _normal(g, (t, d), dtype, 2.0) if case["residual"] else None
    if case["kind"] == "norm_grad":
        s["dout"] = _normal(g, (t, d), dtype, 1e-2)
        s["dx"] = torch.empty((t, d), dtype=dtype, device="cuda")
        s["dweight"] = torch.empty(d, dtype=wtype, device="cuda")
        s["residual"] = _normal(g, (t, d), dtype, 1e-2) if case["residual"] else None    # the gradient that arrives there
        return s
    s["sum"] = torch.empty((t, d), dtype=dtype, device="cuda") if case["residual"] else None
    if case["kind"] == "norm8":
        s["out"] = torch.empty((t, d), dtype=_E4M3, device="cuda")
        s["scales"] = torch.empty((t, _scales(case)), dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.empty((t, d), dtype=dtype, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

_LOW = 0xFFFFFFFF


def _mix(x):
    """32 bits mixed, as whole numbers (tensors of int64 or Python's)."""
    x = x ^ (x >> 16)
    x = (x * 0xB7E15163) & _LOW
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & _LOW
    return x ^ (x >> 16)


def _random(seed, step, tensor, n):
    """The 32 random bits of each of a tensor's values at a step."""
    key = _mix(_mix(_mix(_mix(seed & _LOW) ^ (seed >> 32)) ^ step) ^ tensor)
    i = torch.arange(n, device="cuda")
    return _mix((_mix(key) + i * 0x9E3779B9) & _LOW)        # of tensors below 2^32 values


def _uniform(bits):
    return (bits.float() + 0.5) / 65536.0


def _quantise(x, bits, positive):
    """Codes and scales of blocks of 128: to nearest, or (bits) up with the probability of what is cut off."""
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = x.abs().amax(1) / 448.0
    y = x / torch.where(scale > 0, scale, 1.0)[:, None]
    if bits is not None:
        u = _uniform(torch.nn.functional.pad(bits, (0, -n % BLOCK)).view(-1, BLOCK))
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
        y = torch.copysign(torch.floor(y.abs() / step + u) * step, y)
    q = y.clamp(-448.0, 448.0).to(_E4M3).float()
    if positive:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return q.view(-1)[:n].to(_E4M3), scale


def _step_of(s):
    """The factor of the gradients."""
    if s["norm"] is None:
        return s["scale"]
    return s["scale"] * (s["max_norm"] / (s["scale"] * s["norm"] + 1e-6)).clamp(max=1.0)


def _round_bf16(p, bits):
    """fp32 to bf16: to nearest, or (bits) up with the probability of what is cut off."""
    if bits is None:
        return p.bfloat16()
    return ((p.view(torch.int32) + bits.int()) & -65536).view(torch.float32).bfloat16()


def _one_tensor(s, j, factor):
    p, g = s["params"][j], s["grads"][j].float() * factor
    b1, b2, eight = s["beta1"], s["beta2"], s["case"]["states"] == 8
    if eight:
        spread = lambda x: x.repeat_interleave(BLOCK)[:p.numel()]  # noqa: E731
        m = s["ms"][j].float() * spread(s["mscales"][j])
        v = (s["vs"][j].float() * spread(s["vscales"][j])).square()
    else:
        m, v = s["ms"][j], s["vs"][j]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g.square()
    root = v.sqrt()
    new = p.float() * (1.0 - s["lr"] * s["decay"] * s["decays"][j])
    new = new - s["lr"] / (1.0 - b1 ** s["step"]) * m / (root / math.sqrt(1.0 - b2 ** s["step"]) + s["eps"])
    bits = _random(s["seed"], s["step"], j, p.numel()) if s["seed"] else None
    if p.dtype == torch.bfloat16:
        p.copy_(_round_bf16(new, None if bits is None else ((bits * 0x9E3779B9) & _LOW) >> 16))
    else:
        p.copy_(new)
        if s["copies"] and s["copies"][j] is not None:
            s["copies"][j].copy_(new)
    if eight:
        for x, codes, scales, cut in ((m, s["ms"][j], s["mscales"][j], 0), (root, s["vs"][j], s["vscales"][j], 16)):
            q, scale = _quantise(x, None if bits is None else (bits >> cut) & 0xFFFF, cut == 16)
            codes.view(torch.uint8).copy_(q.view(torch.uint8))
            scales.copy_(scale)
    else:
        s["ms"][j].copy_(m)
        s["vs"][j].copy_(v)


def _states(s):
    return {n: s[n] for n in ("m", "v", "mscale", "vscale", "copy") if n in s} | s["flat"]


def _scores(x, kind):
    """Scores of logits, and zeroes for a row without any."""
    s = torch.sigmoid(x) if kind == "sigmoid" else torch.softmax(x, 1)
    return torch.where((x > -math.inf).any(1, keepdim=True), s, 0.0)


def _choose(s):
    """The experts of each token and their logits. Values next to one another decide, so they are taken in 64 bits; where only the logits' order counts, from that."""
    case, x = s["case"], s["logits"].double()
    c = x
    scores = _scores(x, case["scores"])
    if s["bias"] is not None:
        c = torch.where(x > -math.inf, scores + s["bias"].double(), -math.inf)
    if case["groups"] > 1:
        by_group = c.view(case["tokens"], case["groups"], -1)
        if case["group_best"] == 2:
            value = c if s["bias"] is not None else torch.where(x > -math.inf, scores, -math.inf)
            two = value.view_as(by_group).topk(2, dim=2).values
            value = torch.where(two[..., 0] > -math.inf, two.clamp(min=-1e300).where(two > -math.inf, 0.0).sum(2), -math.inf)
        else:
            value = by_group.amax(2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(kept[..., None], by_group, -math.inf).view_as(c)
    c, experts = torch.sort(c, dim=1, descending=True, stable=True)
    c, experts = c[:, :case["k"]], experts[:, :case["k"]]
    return torch.where(c > -math.inf, experts, -1).int(), None


def _weigh(s):
    case, x = s["case"], s["logits"].float()
    there = s["experts"] >= 0
    scores = torch.where(there, _scores(x, case["scores"]).gather(1, s["experts"].long().clamp(min=0)), 0.0)
    if not case["renormalise"]:
        return there, scores, scores
    total = scores.sum(1, keepdim=True)
    return there, scores, scores / torch.where(total > 0, total, 1.0)


def _route_grad(s):
    case, scale = s["case"], s["scale"]
    there, scores, p = _weigh(s)
    dw = torch.where(there, s["dweights"], 0.0) * scale
    at = s["experts"].long().clamp(min=0)
    out = torch.zeros(s["logits"].shape, dtype=torch.float32, device="cuda")
    if case["renormalise"]:
        dx = p * (dw - (dw * p).sum(1, keepdim=True))
        if case["scores"] == "sigmoid":
            dx = dx * torch.sigmoid(-s["logits"].float()).gather(1, at)
    elif case["scores"] == "sigmoid":
        dx = dw * scores * torch.sigmoid(-s["logits"].float()).gather(1, at)
    else:
        dx = dw * scores
        out -= _scores(s["logits"].float(), "softmax") * dx.sum(1, keepdim=True)
    return out.scatter_add_(1, at, torch.where(there, dx, 0.0)).to(s["logits"].dtype)


def _normed(s):
    x = s["x"].float()
    h = x.to(s["x"].dtype) if s["residual"] is None else (x + s["residual"].float()).to(s["x"].dtype)
    return h, h.float(), s["weight"].float()


def _inverse(h, eps):
    return torch.rsqrt(h.square().mean(1, keepdim=True) + eps)


def _plain(s):
    case = s["case"]
    if case["kind"] == "adamw":
        factor = _step_of(s)
        [_one_tensor(s, j, factor) for j in range(case["tensors"])]
        return _states(s)
    if case["kind"] == "route":
        s["experts"].copy_(_choose(s)[0])
        s["weights"].copy_(_weigh(s)[2] * s["scale"])
        return [s["experts"], s["weights"]]
    if case["kind"] == "route_grad":
        return _route_grad(s)
    if case["kind"] == "norm_grad":
        h, w, dy = s["x"].float(), s["weight"].float(), s["dout"].float()
        r = _inverse(h, s["eps"])
        dx = r * (dy * w - h * r * r * (dy * w * h).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return [dx.to(s["x"].dtype), (dy * h * r).sum(0).to(s["weight"].dtype)]
    stored, h, w = _normed(s)
    r = _inverse(h, s["eps"])
    outs = [] if s["residual"] is None else [stored]
    if case["kind"] == "norm":
        return [(h * r * w).to(s["x"].dtype)] + outs
    n, group = case["dim"], case["group"] or case["dim"]
    y = torch.nn.functional.pad(h * w, (0, -n % group)).view(case["tokens"], -1, group)
    top = y.abs().amax(2, keepdim=True)
    q = (y * (448.0 / torch.where(top > 0, top, 1.0))).clamp(-448.0, 448.0)
    return [q.view(case["tokens"], -1)[:, :n].to(_E4M3), top[..., 0] * r / 448.0] + outs


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------- the package's kernels

def _own(s):
    from collective_communication_amd import binding as hc

    case = s["case"]
    if case["kind"] == "adamw":
        if "plan" not in s:     # a program makes it once, as its tensors stay where they are
            scales = {} if case["states"] == 32 else {"m_scales": s["mscales"], "v_scales": s["vscales"]}
            s["plan"] = hc.AdamWPlan(s["params"], s["grads"], s["ms"], s["vs"], copies=s["copies"], decays=s["decays"],
                                     **scales)
        hc.hc_adamw(s["plan"], s["step"], lr=s["lr"], betas=(s["beta1"], s["beta2"]), eps=s["eps"],
                    weight_decay=s["decay"], grad_scale=s["scale"], d_norm=s["norm"], max_norm=s["max_norm"],
                    seed=s["seed"])
        return _states(s)
    if case["kind"] == "route":
        hc.hc_route(s["logits"], s["experts"], s["weights"], scores=case["scores"], bias=s["bias"],
                    groups=case["groups"], top_groups=case["top_groups"], group_best=case["group_best"],
                    renormalise=case["renormalise"], scale=s["scale"])
        return [s["experts"], s["weights"]]
    if case["kind"] == "route_grad":
        hc.hc_route_grad(s["logits"], s["experts"], s["dweights"], s["dlogits"], scores=case["scores"],
                         renormalise=case["renormalise"], scale=s["scale"])
        return s["dlogits"]
    if case["kind"] == "norm_grad":
        ws = s.get("ws")
        if ws is None:
            need = hc.hc_rms_norm_grad_workspace_bytes(case["tokens"], case["dim"])
            ws = s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        hc.hc_rms_norm_grad(s["dout"], s["x"], s["weight"], s["dx"], s["dweight"], ws, dsum=s["residual"], eps=s["eps"])
        return [s["dx"], s["dweight"]]
    outs = [] if s["residual"] is None else [s["sum"]]
    if case["kind"] == "norm":
        hc.hc_rms_norm(s["x"], s["weight"], s["out"], residual=s["residual"], sum_out=s["sum"], eps=s["eps"])
        return [s["out"]] + outs
    hc.hc_rms_norm_8bit(s["x"], s["weight"], s["out"], s["scales"], group=case["group"], residual=s["residual"],
                        sum_out=s["sum"], eps=s["eps"])
    return [s["out"], s["scales"]] + outs


# ---------------------------------------------------------------------------- 64 bits

def _nearest(y):
    """The e4m3 value nearest to each fp64 value within +-448, ties to the even code."""
    step = torch.exp2(torch.frexp(y)[1].double().clamp(min=-5) - 4)
    return torch.round(y / step) * step


def _exact_codes(x, bits, positive):
    """Codes as numbers and scales, block by block."""
    full = torch.zeros(-(-x.numel() // BLOCK) * BLOCK, dtype=torch.float64, device="cuda")
    full[:x.numel()] = x
    rows = full.view(-1, BLOCK)
    scale = rows.abs().max(1).values / 448
    y = rows / scale.where(scale > 0, torch.ones_like(scale)).unsqueeze(1)
    if bits is None:
        q = _nearest(y)
    else:
        u = torch.zeros_like(full)
        u[:x.numel()] = (bits.double() + 0.5) / 2 ** 16
        step = torch.exp2(torch.frexp(y)[1].double().clamp(min=-5) - 4)
        q = (torch.floor(y.abs() / step + u.view_as(y)) * step).clamp(max=448) * y.sign()
    if positive:
        q = q.where((q != 0) | (rows == 0), torch.full_like(q, 2.0 ** -9))
    return q.view(-1)[:x.numel()], scale


def _exact_adamw(s):
    case = s["case"]
    c = s["scale"]
    if case["clip"]:
        c *= min(1.0, s["max_norm"] / (abs(c) * float(s["norm"]) + 1e-6))
    flat = {t: f.double() for t, f in s["flat"].items()}
    out = {n: s[n].double() for n in ("m", "v", "mscale", "vscale", "copy") if n in s}
    place = lambda view: slice(view.storage_offset(), view.storage_offset() + view.numel())  # noqa: E731
    for j in range(case["tensors"]):
        p, g = s["params"][j].double(), s["grads"][j].double() * c
        if case["states"] == 8:
            where = torch.arange(p.numel(), device="cuda") // BLOCK
            m = s["ms"][j].double() * s["mscales"][j].double()[where]
            v = (s["vs"][j].double() * s["vscales"][j].double()[where]) ** 2
        else:
            m, v = s["ms"][j].double(), s["vs"][j].double()
        m = m + (1 - s["beta1"]) * (g - m)
        v = v + (1 - s["beta2"]) * (g * g - v)
        mhat, vhat = m / (1 - s["beta1"] ** s["step"]), v / (1 - s["beta2"] ** s["step"])
        p = p - s["lr"] * (mhat / (vhat.sqrt() + s["eps"]) + s["decay"] * s["decays"][j] * p)
        t = "bf16" if s["params"][j].dtype == torch.bfloat16 else "f32"
        flat[t][place(s["params"][j])] = p
        if case["copies"] and t == "f32":
            out["copy"][place(s["copies"][j])] = p
        at = place(s["ms"][j])
        if case["states"] == 8:
            bits = _random(s["seed"], s["step"], j, p.numel()) if s["seed"] else None
            for x, name, cut in ((m, "m", 0), (v.sqrt(), "v", 16)):
                q, scale = _exact_codes(x, None if bits is None else (bits >> cut) % 65536, cut > 0)
                out[name][at] = q
                out[name + "scale"][place(s[name + "scales"][j])] = scale
        else:
            out["m"][at], out["v"][at] = m, v
    return out | flat


def _exact_route(s):
    case, x = s["case"], s["logits"].double()
    e = s["experts"].long() if case["kind"] == "route_grad" else _choose(s)[0].long()
    chosen = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        hit = (e[:, j] >= 0).nonzero()[:, 0]
        chosen[hit, e[hit, j]] = 1.0
    if case["scores"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        top = x.max(1, keepdim=True).values
        score = torch.exp(x - top.where(top > -math.inf, torch.zeros_like(top)))
        score = score / score.sum(1, keepdim=True).clamp(min=1e-300)
    total = (score * chosen).sum(1, keepdim=True).clamp(min=1e-300) if case["renormalise"] else 1.0
    w = score * chosen / total
    if case["kind"] == "route":
        picked = w.gather(1, e.clamp(min=0)) * (e >= 0)
        return [None, picked * s["scale"]]
    dw = torch.zeros_like(w)
    for j in range(case["k"]):
        hit = (e[:, j] >= 0).nonzero()[:, 0]
        dw[hit, e[hit, j]] = s["dweights"][hit, j].double() * s["scale"]
    # from weights to scores, then from scores to logits
    ds = chosen * (dw - (dw * w).sum(1, keepdim=True)) / total if case["renormalise"] else dw
    if case["scores"] == "sigmoid":
        return ds * score * (1 - score)
    return score * (ds - (ds * score).sum(1, keepdim=True))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "adamw":
        return _exact_adamw(s)
    if case["kind"] in ("route", "route_grad"):
        return _exact_route(s)
    x, w = s["x"].double(), s["weight"].double()
    if case["kind"] == "norm_grad":
        dy, n = s["dout"].double(), case["dim"]
        rms = ((x * x).sum(1, keepdim=True) / n + s["eps"]).sqrt()
        unit, dunit = x / rms, dy * w
        dx = (dunit - unit * (dunit * unit).sum(1, keepdim=True) / n) / rms
        return [dx if s["residual"] is None else dx + s["residual"].double(), (dy * unit).sum(0)]
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    rms = ((x * x).sum(1, keepdim=True) / case["dim"] + s["eps"]).sqrt()
    outs = [] if s["residual"] is None else [x]
    y = x / rms * w
    if case["kind"] == "norm":
        return [y] + outs
    group = case["group"] or case["dim"]
    q, scales = torch.empty_like(y), torch.empty(s["scales"].shape, dtype=torch.float64, device="cuda")
    for i in range(scales.shape[1]):
        part = y[:, i * group:(i + 1) * group]
        scales[:, i] = part.abs().max(1).values / 448
        unit = scales[:, i:i + 1]
        q[:, i * group:(i + 1) * group] = _nearest(part / unit.where(unit > 0, torch.ones_like(unit)))
    return [q, scales] + outs
