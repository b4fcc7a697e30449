"""What is measured of the routing to experts and of the low-rank adapters.

moe_topk    the experts of every token and their weights, from the router's
            logits: what moe_route (the ids) and moe_combine (the weights) take.
lora        y = base + scale * B (A x) with the adapter of each row's request,
            beside a shared projection (or, for routed pairs, beside the
            experts' products, where the adapter has weights for each expert).

A case is a dict of plain values; `draw` gives more of the same ranges.
"""
import math

import torch

own = False

HBM_LIMIT = 16384 * (4096 * 2 + 2560 * 8)  # activation bytes of the largest listed adapter case


# ------------------------------------------------------------------ the cases

def _topk(name, t, e, top_k, score, groups=1, group_keep=1, group_top=1, bias=False, renormalize=True,
          scale=1.0, masked=0.0):
    return {"name": name, "op": "topk", "t": t, "e": e, "top_k": top_k, "score": score, "groups": groups,
            "group_keep": group_keep, "group_top": group_top, "bias": bias, "renormalize": renormalize,
            "scale": scale, "masked": masked}


def _lora(name, t, k, n, rank, adapters, top_k=1, experts=0, n2=0, order="runs", none=0.0):
    return {"name": name, "op": "lora", "t": t, "k": k, "n": n, "rank": rank, "adapters": adapters,
            "top_k": top_k, "experts": experts, "n2": n2, "order": order, "none": none}


def listed():
    return [
        # one decoded token through a layer of 128 experts, top-8 by softmax: latency only
        _topk("topk-1x128", 1, 128, 8, "softmax"),
        # a decode batch over 256 experts in 8 groups, scored by sigmoid with a balance bias
        _topk("topk-64x256-groups", 64, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # an odd prompt over 60 experts, softmax weights as they are, some experts switched off per token
        _topk("topk-1009x60", 1009, 60, 4, "softmax", renormalize=False, masked=0.1),
        # the prefill of the repository's mixture-of-experts layer: 2048 tokens, 128 experts, top-8
        _topk("topk-2048x128", 2048, 128, 8, "softmax"),
        # several long prompts at once with sigmoid scores, bias and groups: bandwidth and arithmetic
        _topk("topk-32768x256-groups", 32768, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # one decoded token of one request: the smallest projection pair of the decode model
        _lora("lora-1x1024x2048", 1, 1024, 2048, 16, 8),
        # a decode batch of 64 requests with 32 adapters in any order, one in four without: q, k and v at once
        _lora("lora-64-qkv", 64, 2560, 4096, 16, 32, n2=1024, order="mixed", none=0.25),
        # a mid-sized batch with odd sizes: 333 rows, 1001 columns, rank 24
        _lora("lora-333x1088x1001", 333, 1088, 1001, 24, 7, order="mixed", none=0.1),
        # four prompts of one prefill step through the widest projection
        _lora("lora-2048x2560x9728", 2048, 2560, 9728, 16, 4),
        # the experts' down projection of a prefill, an adapter with weights for every expert
        _lora("lora-512-experts-down", 512, 768, 2048, 16, 4, top_k=8, experts=128, order="mixed"),
        # many prompts at once, rank 64: bandwidth of activations and outputs
        _lora("lora-16384x4096x2560", 16384, 4096, 2560, 64, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        e = groups * rng.randint(8, 64 if groups == 1 else 256 // groups) if groups > 1 else _log(rng, 8, 384)
        keep = rng.randint(2, groups) if groups > 1 else 1
        bias = rng.random() < 0.5
        t = _log(rng, 1, 32768)
        t = min(t, 32768 * 256 // max(e, 256))
        top_k = min(rng.randint(1, 10), keep * (e // groups))
        masked = 0.0 if bias or groups > 1 else rng.choice([0.0, 0.1])
        c = _topk("", t, e, top_k, score, groups, keep, rng.choice([1, 2]) if groups > 1 else 1, bias,
                  rng.random() < 0.7, rng.choice([1.0, 2.5]), masked)
    else:
        rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
        adapters = _log(rng, 1, 48)
        none = rng.choice([0.0, 0.25])
        order = rng.choice(["runs", "mixed"])
        if rng.random() < 0.3:
            t, top_k = _log(rng, 1, 2048), rng.randint(1, 8)
            experts = rng.randint(8, 128)
            adapters = min(adapters, 8)
            k, n = 64 * rng.randint(4, 32), rng.randint(100, 2560)
            rank = min(rank, 32)
            c = _lora("", t, k, n, rank, adapters, top_k, experts, order=order, none=none)
        else:
            k, n = 64 * _log(rng, 8, 152), _log(rng, 64, 9728)
            n2 = rng.choice([0, 0, _log(rng, 64, 2048)])
            t = _log(rng, 1, 16384)
            t = max(1, min(t, HBM_LIMIT // (k * 2 + (n + 2 * n2) * 8) // 2, 2 ** 34 // (adapters * rank * (k + n + 2 * n2))))
            c = _lora("", t, k, n, rank, adapters, n2=n2, order=order, none=none)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _adapter_ids(c, gen):
    """One id per token: every adapter in use where there are tokens enough,
    in runs (prompts one after the other) or mixed; -1 for no adapter."""
    t = c["t"]
    # the first adapters come once each, the other tokens draw theirs
    ids = torch.randint(0, c["adapters"], (t,), generator=gen, device="cuda", dtype=torch.int32)
    first = min(t, c["adapters"])
    ids[:first] = torch.arange(first, device="cuda", dtype=torch.int32)
    ids = ids[torch.randperm(t, generator=gen, device="cuda")]
    if c["order"] == "runs":
        ids = ids.sort().values
    if c["none"]:
        off = torch.rand(t, generator=gen, device="cuda") < c["none"]
        ids = torch.where(off, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    rand = lambda *shape, **kw: torch.randn(*shape, generator=gen, device="cuda", **kw)  # noqa: E731
    if c["op"] == "topk":
        logits = rand(c["t"], c["e"]) * 1.5
        if c["masked"]:
            off = torch.rand(c["t"], c["e"], generator=gen, device="cuda") < c["masked"]
            off[:, : c["top_k"]] = False
            logits.masked_fill_(off, -math.inf)
        return {"case": c, "logits": logits, "bias": rand(c["e"]) * 0.05 if c["bias"] else None,
                "ids": torch.empty(c["t"], c["top_k"], dtype=torch.int32, device="cuda"),
                "weights": torch.empty(c["t"], c["top_k"], dtype=torch.float32, device="cuda")}
    rows, slots = c["t"] * c["top_k"], c["adapters"] * max(1, c["experts"])
    s = {"case": c, "x": rand(rows if c["experts"] else c["t"], c["k"], dtype=torch.float16),
         "adapter_ids": _adapter_ids(c, gen), "expert_ids": None, "workspace": None,
         "scales": 0.5 + torch.rand(c["adapters"], generator=gen, device="cuda") * 1.5, "projections": []}
    if c["experts"]:
        picks = torch.rand(c["t"], c["experts"], generator=gen, device="cuda").sort(dim=1).indices
        s["expert_ids"] = picks[:, : c["top_k"]].to(torch.int32).contiguous()
    for n in _widths(c):
        a = rand(slots, c["rank"], c["k"], dtype=torch.float16) / math.sqrt(c["k"])
        b = rand(slots, n, c["rank"], dtype=torch.float16) * 0.1
        base = rand(rows, n)
        s["projections"].append((a, b, base, torch.empty_like(base)))
    return s


def _widths(c):
    """Output columns of the projections that share the input: one, or q with k and v."""
    return (c["n"], c["n2"], c["n2"]) if c["n2"] else (c["n"],)


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if c["op"] == "topk":
        return _run_topk(state, c) if own else _plain_topk(state, c)
    return _run_lora(state, c) if own else _plain_lora(state, c)


def _run_topk(s, c):
    import quantized_matmul_qgemv_amd as qmm
    return qmm.moe_topk(s["logits"], c["top_k"], bias=s["bias"], score=c["score"], groups=c["groups"],
                        group_keep=c["group_keep"], group_top=c["group_top"], renormalize=c["renormalize"],
                        scale=c["scale"], expert_ids=s["ids"], weights=s["weights"])


def _run_lora(s, c):
    import quantized_matmul_qgemv_amd as qmm
    problems = [(s["x"], a, b, base, y) for a, b, base, y in s["projections"]]
    kw = {"scales": s["scales"], "expert_ids": s["expert_ids"], "x_row_per_pair": c["experts"] > 0}
    if s["workspace"] is None:  # kept by the program, like any workspace of the library
        s["workspace"] = qmm.lora_workspace(problems, s["adapter_ids"], expert_ids=s["expert_ids"])
    if len(problems) == 1:
        x, a, b, base, y = problems[0]
        return qmm.lora(x, a, b, s["adapter_ids"], base=base, y=y, workspace=s["workspace"], **kw)
    return qmm.lora_batched(problems, s["adapter_ids"], workspace=s["workspace"], **kw)


def _plain_topk(s, c):
    # 64 bits: which of two near scores is larger decides whole numbers
    logits = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        grouped = choice.view(c["t"], c["groups"], -1)
        best = grouped.sort(dim=2, descending=True).values[:, :, : c["group_top"]].sum(dim=2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : c["group_keep"]]
        out = torch.ones(c["t"], c["groups"], dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        choice = grouped.masked_fill(out[:, :, None], -math.inf).view(c["t"], -1)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    weights = score.gather(1, ids)
    if c["renormalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (weights * c["scale"]).float()


def _plain_lora(s, c):
    """Few rows: each row's own matrices are gathered.  Many rows: one product
    with the matrices of all slots, the other slots' columns set to zero, and
    one back."""
    adapter = s["adapter_ids"].repeat_interleave(c["top_k"])
    slot = adapter if s["expert_ids"] is None else adapter * c["experts"] + s["expert_ids"].view(-1)
    active = adapter >= 0
    slot = torch.where(active, slot, torch.zeros_like(slot)).long()
    scale = torch.where(active, s["scales"][adapter.clamp(min=0).long()], torch.zeros_like(s["scales"][:1]))
    x, out = s["x"].float(), []
    if len(slot) <= 256:
        out = [base + scale[:, None] * torch.matmul(
            b[slot].float(), torch.matmul(a[slot].float(), x[:, :, None]))[:, :, 0]
            for a, b, base, _ in s["projections"]]
    else:
        slots, rank = c["adapters"] * max(1, c["experts"]), c["rank"]
        mine = torch.arange(slots, device="cuda")[None, :] == slot[:, None]
        gate = mine.float() * scale[:, None]
        for a, b, base, _ in s["projections"]:
            v = x @ a.float().view(slots * rank, -1).t()
            v = (v.view(-1, slots, rank) * gate[:, :, None]).view(-1, slots * rank)
            out.append(base + v @ b.float().transpose(1, 2).reshape(slots * rank, -1))
    return out[0] if len(out) == 1 else out


# ------------------------------------------------------- what cannot be avoided

def work(case):
    c = case
    if c["op"] == "topk":
        t, e, top_k = c["t"], c["e"], c["top_k"]
        # a compare per logit and chosen expert's rank; an exponential counted as one operation
        return {"bytes": 4 * t * e + (4 * e if c["bias"] else 0) + 8 * t * top_k, "flops": 2 * t * e}
    rows = c["t"] * c["top_k"]
    active = max(1, round(c["t"] * (1 - c["none"]))) * c["top_k"]
    slots = c["adapters"] * max(1, c["experts"])
    used = min(active, slots) if not c["experts"] else slots * (1 - (1 - 1 / slots) ** active)
    total = {"bytes": (rows if c["experts"] else c["t"]) * c["k"] * 2 + 4 * c["t"], "flops": 0}
    for n in _widths(c):
        total["bytes"] += int(used * c["rank"] * (c["k"] + n) * 2) + rows * n * 8
        total["flops"] += 2 * active * c["rank"] * (c["k"] + n)
    return total


# ------------------------------------------------------------ in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_topk(s, case) if case["op"] == "topk" else _exact_lora(s, case)


def _exact_topk(s, c):
    import numpy as np
    z = s["logits"].cpu().numpy().astype(np.float64)
    rows = np.arange(c["t"])[:, None]
    if c["score"] == "sigmoid":
        p = np.exp(-np.logaddexp(0.0, -z))
    else:
        p = np.exp(z - np.logaddexp.reduce(z, axis=1, keepdims=True))
    rank_by = p + (0.0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64))
    size = c["e"] // c["groups"]
    if c["groups"] > 1:
        parts = np.sort(rank_by.reshape(c["t"], c["groups"], size), axis=2)
        order = np.argsort(-parts[:, :, size - c["group_top"]:].sum(axis=2), axis=1, kind="stable")
        dropped = order[:, c["group_keep"]:]
        rank_by.reshape(c["t"], c["groups"], size)[rows, dropped] = -np.inf
    ids = np.argsort(-rank_by, axis=1, kind="stable")[:, : c["top_k"]]
    w = p[rows, ids]
    if c["renormalize"]:
        w /= w.sum(axis=1, keepdims=True)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w * c["scale"])


def _exact_lora(s, c):
    """Slot by slot: the rows of one slot through its two matrices."""
    outs = [base.double() for _, _, base, _ in s["projections"]]
    adapter = s["adapter_ids"].cpu().repeat_interleave(c["top_k"])
    slot = adapter.clone()
    if s["expert_ids"] is not None:
        slot = torch.where(adapter < 0, adapter, adapter * c["experts"] + s["expert_ids"].cpu().view(-1))
    order = slot.argsort()
    values, counts = slot[order].unique_consecutive(return_counts=True)
    for value, part in zip(values.tolist(), order.split(counts.tolist())):
        if value < 0:
            continue
        part = part.cuda()
        x = s["x"][part].double()
        scale = float(s["scales"][value // max(1, c["experts"])])
        for y, (a, b, _, _) in zip(outs, s["projections"]):
            y[part] += scale * ((x @ a[value].double().t()) @ b[value].double().t())
    return outs[0] if len(outs) == 1 else outs
