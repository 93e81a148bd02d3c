"""Cases and plain forms of the operators around the gradient exchange: the
global gradient norm with clipping, the embedding lookup and its gradient, and
the sorting of tokens by expert with the weighted way back and its gradient.

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


# ---------------------------------------------------------------------------- cases

def _clip(tensors, total, dtype, norm, flat):
    return {"kind": "clip", "tensors": tensors, "total": total, "dtype": dtype, "norm": norm, "flat": flat}


def _embed(tokens, vocab, dim, dtype, ids, shards, scaled):
    return {"kind": "embed", "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "ids": ids,
            "shards": shards, "scaled": scaled}


def _embed_grad(tokens, vocab, dim, dtype, dw, ids, shards, scaled):
    return {"kind": "embed_grad", "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "dw": dw, "ids": ids,
            "shards": shards, "scaled": scaled}


def _expert(kind, tokens, k, experts, shards, dim, dtype, align):
    return {"kind": kind, "tokens": tokens, "k": k, "experts": experts, "shards": shards, "dim": dim, "dtype": dtype,
            "align": align}


def listed():
    return [
        # the gradients of one small block: a dozen separate tensors, where the launches count
        dict(_clip(12, 300_001, "f32", 4.0, False), name="clip_small_f32"),
        # one bucket of 2^25 values, as the compressed exchange takes it, with fp32 vectors beside bf16 matrices
        dict(_clip(290, 1 << 25, "mixed", 2.5, True), name="clip_bucket_mixed"),
        # a whole model's gradients: 2^29 bf16 values in separate tensors
        dict(_clip(450, 1 << 29, "bf16", 8.0, False), name="clip_model_bf16"),
        # one decoding step of 64 sequences
        dict(_embed(64, 128_000, 4096, "bf16", 64, 1, False), name="embed_decode_bf16"),
        # a batch of prompts against one of four shards of the vocabulary, scaled by sqrt(dim)
        dict(_embed(30_011, 64_000, 4096, "bf16", 32, 4, True), name="embed_prompt_shard_bf16"),
        # a small fine-tuning step, gradients in fp32, a width that is no power of two
        dict(_embed_grad(2_000, 10_007, 1000, "f32", "f32", 64, 1, True), name="embed_grad_small_f32"),
        # a pretraining micro-batch into the fp32 gradient of a large vocabulary
        dict(_embed_grad(32_768, 100_003, 2048, "bf16", "f32", 64, 1, False), name="embed_grad_batch_bf16"),
        # a decoding step: 96 tokens to 8 of 128 experts each
        dict(_expert("dispatch", 96, 8, 128, 1, 2048, "bf16", 16), name="dispatch_decode_bf16"),
        # a pretraining micro-batch to 8 of 128 experts each, rows padded for tiles of 32
        dict(_expert("dispatch", 16_384, 8, 128, 1, 4096, "bf16", 32), name="dispatch_batch_bf16"),
        # a prompt back from 2 of 8 experts, an odd width, fp32
        dict(_expert("combine", 5_003, 2, 8, 1, 1031, "f32", 1), name="combine_prompt_odd_f32"),
        # a micro-batch on one of four ranks of experts: most tokens' slots lie elsewhere
        dict(_expert("combine_grad", 9_999, 6, 16, 4, 2560, "f32", 1), name="combine_grad_shard_f32"),
        # the backward pass of a pretraining micro-batch
        dict(_expert("combine_grad", 16_384, 8, 64, 1, 4096, "bf16", 32), name="combine_grad_batch_bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, hi):
    """A row width: any number, or a multiple of 8 or of 64 as most models have."""
    return max(1, _log(rng, 16, hi) // (m := rng.choice((1, 8, 64))) * m)


def draw(rng):
    kind = rng.choice(("clip", "embed", "embed_grad", "dispatch", "combine", "combine_grad"))
    dtype = rng.choice(("bf16", "f32"))
    while True:
        if kind == "clip":
            tensors = _log(rng, 1, 700)
            c = _clip(tensors, _log(rng, 1000 * tensors, 1 << 28), rng.choice(("bf16", "f32", "mixed")),
                      rng.choice((0.5, 2.5, 30.0)), rng.random() < 0.5)
        elif kind == "embed":
            c = _embed(_log(rng, 1, 60_000), _log(rng, 500, 200_000), _width(rng, 6000), dtype, rng.choice((32, 64)),
                       rng.choice((1, 1, 2, 8)), rng.random() < 0.5)
        elif kind == "embed_grad":
            c = _embed_grad(_log(rng, 1, 60_000), _log(rng, 500, 200_000), _width(rng, 6000), dtype,
                            rng.choice((dtype, "f32")), rng.choice((32, 64)), rng.choice((1, 1, 2, 8)),
                            rng.random() < 0.5)
        else:
            experts = _log(rng, 2, 256)
            c = _expert(kind, _log(rng, 1, 40_000), rng.randint(1, min(10, experts)), experts, rng.choice((1, 1, 2, 8)),
                        _width(rng, 6000), dtype, rng.choice((1, 1, 16, 64)))
        if work(c)["bytes"] <= 1.0e9:
            return c


def _rows(case):
    """Rows that hold every expert's slots, each expert's from a multiple of align on."""
    n = case["tokens"] * case["k"]
    return n + min(case["experts"], n) * (case["align"] - 1)


def work(case):
    if case["kind"] == "clip":
        small = sum(s for s, t in _tensors(case) if t == "f32")
        return {"bytes": 2 * (4 * small + 2 * (case["total"] - small)), "flops": 3 * case["total"]}
    t, d, es = case["tokens"], case["dim"], _SIZE[case["dtype"]]
    if case["kind"] == "embed":
        return {"bytes": t * (case["ids"] // 8 + d * es * (1 + 1 / case["shards"])), "flops": t * d / case["shards"]}
    if case["kind"] == "embed_grad":
        return {"bytes": t * (case["ids"] // 8 + d * es / case["shards"]) + case["vocab"] * d * _SIZE[case["dw"]],
                "flops": t * d / case["shards"]}
    n = t * case["k"]
    here = n / case["shards"]
    if case["kind"] == "dispatch":
        return {"bytes": n * 4 + t * d * es * (1 - (1 - 1 / case["shards"]) ** case["k"]) + here * d * es + 8 * n,
                "flops": 0}
    if case["kind"] == "combine":
        return {"bytes": n * 8 + here * d * es + t * d * es, "flops": 2 * here * d}
    return {"bytes": n * 12 + t * d * es * (1 - (1 - 1 / case["shards"]) ** case["k"]) + 2 * here * d * es,
            "flops": 3 * here * d}


# ---------------------------------------------------------------------------- inputs

def _tensors(case):
    """(size, type) of each gradient: sizes over a factor of 4096, as matrices stand beside vectors."""
    r = random.Random(case["tensors"] * 1_000_003 + case["total"])
    w = [math.exp(r.uniform(0.0, math.log(4096.0))) for _ in range(case["tensors"])]
    sizes = [int(case["total"] * x / sum(w)) for x in w]
    sizes[-1] += case["total"] - sum(sizes)
    middle = sorted(sizes)[len(sizes) // 2]
    return [(s, case["dtype"] if case["dtype"] != "mixed" else "f32" if s < middle else "bf16") for s in sizes]


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _ids(case, g):
    """Token ids with frequencies that fall as 1/rank, over all shards of the vocabulary."""
    every = case["vocab"] * case["shards"]
    rank = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64).mul_(math.log(every + 1)).exp_()
    place = torch.randperm(every, generator=g, device="cuda")
    ids = place[(rank.long() - 1).clamp_(0, every - 1)]
    return ids.to(torch.int32 if case["ids"] == 32 else torch.int64)


def _choice(case, g):
    """Each token's k distinct experts of all shards', some experts liked more than others, and their weights."""
    every = case["experts"] * case["shards"]
    likes = torch.randn(every, generator=g, device="cuda")
    logits = torch.randn((case["tokens"], every), generator=g, device="cuda") + 0.7 * likes
    top, experts = logits.topk(case["k"], dim=1)
    return experts.to(torch.int32), torch.softmax(top, dim=1)


def _start(case, name):
    """The first id of this rank's shard."""
    return case[name] * (case["shards"] // 2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "clip":
        parts = _tensors(case)
        std = case["norm"] / math.sqrt(case["total"])
        flat, outs = {}, {}
        for t in ("bf16", "f32"):
            n = sum(size for size, of in parts if of == t)
            flat[t] = _normal(g, n, _TYPES[t], std) if case["flat"] else None
            outs[t] = torch.empty(n, dtype=_TYPES[t], device="cuda")
        at, s["grads"], s["outs"] = {"bf16": 0, "f32": 0}, [], []
        for size, t in parts:
            s["grads"].append(flat[t][at[t]:at[t] + size] if case["flat"] else _normal(g, size, _TYPES[t], std))
            s["outs"].append(outs[t][at[t]:at[t] + size])
            at[t] += size
        s["flat"], s["max_norm"] = outs, 1.0
        s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        return s
    dtype, t, d = _TYPES[case["dtype"]], case["tokens"], case["dim"]
    if case["kind"] in ("embed", "embed_grad"):
        s["ids"], s["start"] = _ids(case, g), _start(case, "vocab")
        s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
        if case["kind"] == "embed":
            s["weight"] = _normal(g, (case["vocab"], d), dtype, 0.02)
            s["out"] = torch.empty((t, d), dtype=dtype, device="cuda")
        else:
            s["dout"] = _normal(g, (t, d), dtype, 1e-3)
            s["out"] = torch.empty((case["vocab"], d), dtype=_TYPES[case["dw"]], device="cuda")
        return s
    s["experts"], s["weights"] = _choice(case, g)
    s["start"], rows = _start(case, "experts"), _rows(case)
    # row_of_slot, slot_of_row, the experts' first rows and their counts
    s["plan"] = [torch.empty(n, dtype=torch.int32, device="cuda")
                 for n in (t * case["k"], rows, case["experts"] + 1, case["experts"])]
    if case["kind"] == "dispatch":
        s["x"] = _normal(g, (t, d), dtype)
        s["out"] = torch.zeros((rows, d), dtype=dtype, device="cuda")  # rows past the last expert's stay as they are
        return s
    s["plan"] = _sort(s)
    s["rows"] = _normal(g, (rows, d), dtype)
    if case["kind"] == "combine":
        s["out"] = torch.empty((t, d), dtype=dtype, device="cuda")
    else:
        s["dy"] = _normal(g, (t, d), dtype, 1e-2)
        s["out"] = torch.zeros((rows, d), dtype=dtype, device="cuda")
        s["dweights"] = torch.empty((t, case["k"]), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

def _sort(s):
    case = s["case"]
    key = s["experts"].reshape(-1).long() - s["start"]
    n, e, align = key.numel(), case["experts"], case["align"]
    key = torch.where((key >= 0) & (key < e), key, e)
    slots = torch.sort(key, stable=True).indices
    counts = torch.zeros(e + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = ((counts[:e] + align - 1) // align * align).cumsum(0)
    skip = counts.cumsum(0) - counts  # slots before the expert's own, without alignment
    sorted_key = key[slots]
    row = offsets[sorted_key] + torch.arange(n, device="cuda") - skip[sorted_key]
    rows = _rows(case)
    there = sorted_key < e
    row_of_slot = torch.empty(n, dtype=torch.int32, device="cuda")
    row_of_slot[slots] = torch.where(there, row, -1).int()
    slot_of_row = torch.full((rows + 1,), -1, dtype=torch.int32, device="cuda")
    slot_of_row[torch.where(there, row, rows)] = torch.where(there, slots, -1).int()
    return [row_of_slot, slot_of_row[:rows], offsets.int(), counts[:e].int()]


def _plain(s):
    case = s["case"]
    if case["kind"] == "clip":
        norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
        coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        scaled = [(x.float() * coef).to(x.dtype) for x in s["grads"]]
        return [norm] + [torch.cat(p) if (p := [x for x in scaled if x.dtype == t]) else s["flat"][n]
                         for n, t in _TYPES.items()]
    dtype = _TYPES[case["dtype"]]
    if case["kind"] in ("embed", "embed_grad"):
        at = s["ids"].long() - s["start"]
        there = (at >= 0) & (at < case["vocab"])
        if case["kind"] == "embed":
            rows = s["weight"][torch.where(there, at, 0)].float() * s["scale"]
            return torch.where(there[:, None], rows, 0.0).to(dtype)
        grad = torch.zeros((case["vocab"] + 1, case["dim"]), dtype=torch.float32, device="cuda")
        grad.index_add_(0, torch.where(there, at, case["vocab"]), s["dout"].float())
        return (grad[:-1] * s["scale"]).to(_TYPES[case["dw"]])
    if case["kind"] == "dispatch":
        plan = _sort(s)
        slot, rows = plan[1].long(), torch.zeros_like(s["out"])
        token = torch.where(slot >= 0, slot // case["k"], 0)
        return plan + [torch.where((slot >= 0)[:, None], s["x"][token], rows)]
    row = s["plan"][0].long().view(case["tokens"], case["k"])
    there = row >= 0
    if case["kind"] == "combine":
        rows = s["rows"][torch.where(there, row, 0)].float()
        return torch.where(there[..., None], rows * s["weights"][..., None], 0.0).sum(1).to(dtype)
    slot = s["plan"][1].long()
    token = torch.where(slot >= 0, slot // case["k"], 0)
    drows = s["dy"][token].float()
    dots = (drows * s["rows"].float()).sum(1)
    drows = drows * s["weights"].view(-1)[torch.where(slot >= 0, slot, 0)][:, None]
    dweights = torch.where(there, dots[torch.where(there, row, 0)], 0.0)
    return [torch.where((slot >= 0)[:, None], drows, 0.0).to(dtype), dweights]


def run(s):
    return _own(s) if own else _plain(s)


# ---------------------------------------------------------------------------- the package's kernels

def _space(s, need):
    """The workspace that a program keeps for the call."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    from collective_communication_amd import binding as hc

    case = s["case"]
    if case["kind"] == "clip":
        ws = _space(s, hc.hc_grad_norm_workspace_bytes(len(s["grads"])))
        hc.hc_clip_grad_norm(s["grads"], s["max_norm"], s["norm"], ws, outs=s["outs"])
        return [s["norm"][0], s["flat"]["bf16"], s["flat"]["f32"]]
    if case["kind"] == "embed":
        hc.hc_embedding(s["ids"], s["weight"], s["out"], vocab_start=s["start"], scale=s["scale"])
        return s["out"]
    if case["kind"] == "embed_grad":
        ws = s.get("ws")
        if ws is None:
            ws = _space(s, hc.hc_embedding_grad_workspace_bytes(case["tokens"], case["vocab"], case["dim"]))
        hc.hc_embedding_grad(s["ids"], s["dout"], s["out"], ws, vocab_start=s["start"], scale=s["scale"])
        return s["out"]
    if "kept" not in s:
        s["kept"] = hc.ExpertPlan(case["tokens"], case["k"], case["experts"], case["align"], *s["plan"])
    plan = s["kept"]
    if case["kind"] == "dispatch":
        ws = s.get("ws")
        if ws is None:
            ws = _space(s, hc.hc_expert_sort_workspace_bytes(case["tokens"] * case["k"], case["experts"]))
        hc.hc_expert_sort(s["experts"], plan, ws, expert_start=s["start"])
        hc.hc_expert_dispatch(s["x"], plan, s["out"])
        return s["plan"] + [s["out"]]
    if case["kind"] == "combine":
        hc.hc_expert_combine(s["rows"], plan, s["weights"], s["out"])
        return s["out"]
    hc.hc_expert_combine_grad(s["dy"], s["rows"], plan, s["weights"], s["out"], s["dweights"])
    return [s["out"], s["dweights"]]


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "clip":
        total = 0.0
        for x in s["grads"]:
            x = x.double()
            total += float(torch.dot(x, x))
        norm = math.sqrt(total)
        coef = min(1.0, s["max_norm"] / (norm + 1e-6))
        flat = {n: torch.empty_like(f, dtype=torch.float64) for n, f in s["flat"].items()}
        at = {"bf16": 0, "f32": 0}
        for (size, t), x in zip(_tensors(case), s["grads"]):
            flat[t][at[t]:at[t] + size] = x.double() * coef
            at[t] += size
        return [torch.tensor(norm, dtype=torch.float64), flat["bf16"], flat["f32"]]
    if case["kind"] in ("embed", "embed_grad"):
        ids = s["ids"].double() - s["start"]
        pick = ((ids >= 0) & (ids < case["vocab"])).nonzero()[:, 0]
        to = ids[pick].long()
        if case["kind"] == "embed":
            out = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device="cuda")
            out[pick] = s["weight"].index_select(0, to).double() * s["scale"]
            return out
        out = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        return out.index_put_((to,), s["dout"].double()[pick] * s["scale"], accumulate=True)
    e = s["experts"].long() - s["start"]
    here = (e >= 0) & (e < case["experts"])
    # a slot's row: its expert's aligned start, and how many slots before it chose the same expert
    one = torch.zeros((e.numel(), case["experts"] + 1), dtype=torch.int32, device="cuda")
    key = torch.where(here, e, case["experts"]).view(-1, 1)
    one.scatter_(1, key, 1)
    before = (one.cumsum(0).gather(1, key) - 1).view(-1)
    padded = torch.ceil(one.sum(0)[:case["experts"]].double() / case["align"]).long() * case["align"]
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), padded.cumsum(0)])
    row = (first[key.view(-1)] + before).view_as(e)
    del one
    if case["kind"] == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            h = here[:, j]
            out[row[h, j]] = s["x"][h].double()
        return [None, None, None, None, out]
    if case["kind"] == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            h = here[:, j]
            out[h] += s["weights"][h, j, None].double() * s["rows"][row[h, j]].double()
        return out
    drows = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(s["dweights"].shape, dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        h = here[:, j]
        drows[row[h, j]] = s["weights"][h, j, None].double() * s["dy"][h].double()
        dweights[h, j] = (s["dy"][h].double() * s["rows"][row[h, j]].double()).sum(1)
    return [drows, dweights]
