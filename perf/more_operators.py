"""What is measured of the products in 8-bit integers.

gemm        y = sx sw (codes of x) (codes of w)^T [+ bias]: a scale for each token
            and one for each output channel; x comes in 16 or 32 bits and is
            rounded to 8 in the call, or as codes with their scales.
grouped     the same for the experts' down projection of a routed layer: the
            rows of each expert, however many they are, with its own weights.
swiglu      the experts' gate and up products with silu(gate) * up behind them.

A case is a dict of plain values; `draw` gives more of the same ranges.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "codes": torch.int8}
MOST = 16384 * 9728 * 2560  # multiply-adds of the largest listed product
MOST_ROUTED = 16384 * 8 * 2 * 768 * 2048  # and of the largest listed routed one


# ------------------------------------------------------------------ the cases

def _gemm(name, m, k, n, x="fp16", y="fp32", n2=0, bias=False):
    return {"name": name, "op": "gemm", "m": m, "k": k, "n": n, "x": x, "y": y, "n2": n2, "bias": bias}


def _routed(name, op, t, top_k, experts, k, n, x="fp16", y="fp32"):
    return {"name": name, "op": op, "t": t, "top_k": top_k, "experts": experts, "k": k, "n": n, "x": x, "y": y}


def listed():
    return [
        # one decoded token through q, k and v: latency
        _gemm("gemm-1-qkv", 1, 2560, 4096, "fp16", "fp32", 1024),
        # one decoded token through the widest projection: the weights once from memory
        _gemm("gemm-1x2560x9728", 1, 2560, 9728, "bf16", "bf16"),
        # a decode batch of 64 requests through the same
        _gemm("gemm-64x2560x9728", 64, 2560, 9728, "fp16", "fp16"),
        # an odd prompt, odd widths, with a bias
        _gemm("gemm-333x1088x1001", 333, 1088, 1001, "fp32", "fp32", 0, True),
        # a prefill's attention output, rounded to 8 bits by the step before
        _gemm("gemm-512x4096x2560-codes", 512, 4096, 2560, "codes", "fp16"),
        # a prefill's widest projection
        _gemm("gemm-2048x2560x9728", 2048, 2560, 9728, "fp16", "fp16"),
        # many prompts at once through the FFN's way back: the matrix cores
        _gemm("gemm-16384x9728x2560", 16384, 9728, 2560, "bf16", "bf16"),
        # one decoded token through its eight experts
        _routed("swiglu-1-of-128", "swiglu", 1, 8, 128, 2048, 768, "fp16", "fp16"),
        # a decode batch through the experts' way back
        _routed("grouped-64-down", "grouped", 64, 8, 128, 768, 2048),
        # an odd prompt over 60 experts of odd width
        _routed("swiglu-333-of-60", "swiglu", 333, 4, 60, 1088, 517, "bf16", "bf16"),
        # the prefill of the repository's mixture-of-experts layer, way back
        _routed("grouped-2048-down", "grouped", 2048, 8, 128, 768, 2048, "fp16", "fp32"),
        # several long prompts at once through gate and up
        _routed("swiglu-16384-of-128", "swiglu", 16384, 8, 128, 2048, 768, "fp16", "fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    x, y = rng.choice(["fp16", "fp16", "bf16", "fp32", "codes"]), rng.choice(["fp32", "fp16", "bf16"])
    if rng.random() < 0.55:
        k, n = 16 * _log(rng, 4, 608), _log(rng, 1, 9728)
        n2 = rng.choice([0, 0, _log(rng, 1, 2048)])
        m = max(1, min(_log(rng, 1, 16384), MOST // (2 * k * (n + 2 * n2))))
        c = _gemm("", m, k, n, x, y, n2, rng.random() < 0.3)
    else:
        experts = _log(rng, 2, 128)
        top_k = min(experts, rng.randint(1, 8))
        op = rng.choice(["grouped", "swiglu"])
        k, n = 16 * _log(rng, 4, 128), _log(rng, 16, 2048 if op == "grouped" else 768)
        t = max(1, min(_log(rng, 1, 16384), MOST_ROUTED // (2 * top_k * k * n)))
        c = _routed("", op, t, top_k, experts, k, n, x, "fp16" if op == "swiglu" and y == "fp32" else y)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _widths(c):
    """Output columns of the products that share the input: one, or q with k and v."""
    return (c["n"], c["n2"], c["n2"]) if c.get("n2") else (c["n"],)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    unit = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731

    def codes(*shape):  # a channel's weights: normal, its largest of three or four deviations at 127
        return (rand(*shape) * 36).round_().clamp_(-127, 127).to(torch.int8)

    rows = c["m"] if c["op"] == "gemm" else c["t"] * (c["top_k"] if c["op"] == "grouped" else 1)
    s = {"case": c, "x_scales": None, "workspace": None, "plan": None}
    if c["x"] == "codes":
        s["x"], s["x_scales"] = codes(rows, c["k"]), (0.5 + unit(rows)) / 36
    else:  # tokens of different size, a few channels much larger than the others
        x = rand(rows, c["k"]) * torch.exp(0.5 * rand(rows, 1))
        x *= torch.where(unit(c["k"]) < 0.004, 12.0, 1.0)
        s["x"] = x.to(TYPES[c["x"]])
    if c["op"] == "gemm":
        s["products"] = [(codes(n, c["k"]), (0.5 + unit(n)) * (0.02 / 36), rand(n) * 0.1 if c["bias"] else None,
                          torch.empty(rows, n, dtype=TYPES[c["y"]], device="cuda")) for n in _widths(c)]
        return s
    experts, pairs = c["experts"], c["t"] * c["top_k"]
    s["weights"] = [(codes(experts, c["n"], c["k"]), (0.5 + unit(experts, c["n"])) * (0.02 / 36))
                    for _ in range(2 if c["op"] == "swiglu" else 1)]
    # some experts are chosen more often than others
    liked = unit(c["t"], experts) * torch.exp(0.3 * rand(experts))
    s["ids"] = liked.sort(dim=1, descending=True).indices[:, : c["top_k"]].to(torch.int32).contiguous()
    s["y"] = torch.empty(pairs, c["n"], dtype=TYPES[c["y"]], device="cuda")
    # the layer's routing, made once for its products: pairs by expert
    if own:
        import quantized_matmul_qgemv_amd as qmm
        s["plan"] = qmm.moe_route(s["ids"], experts)
    flat = s["ids"].view(-1).long()
    s["order"], s["counts"] = flat.argsort(stable=True), torch.bincount(flat, minlength=experts).tolist()
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if c["op"] == "gemm":
        return _run_gemm(state, c) if own else _plain_gemm(state, c)
    return _run_routed(state, c) if own else _plain_routed(state, c)


def _run_gemm(s, c):
    import quantized_matmul_qgemv_amd as qmm
    problems = [(w, ws, s["x"], s["x_scales"], b, y) for w, ws, b, y in s["products"]]
    if s["workspace"] is None:  # kept by the program, like any workspace of the library
        s["workspace"] = qmm.i8_gemm_workspace(problems)
    if len(problems) == 1:
        w, ws, x, xs, b, y = problems[0]
        return qmm.i8_gemm(w, ws, x, xs, bias=b, y=y, workspace=s["workspace"])
    return qmm.i8_gemm_batched(problems, workspace=s["workspace"])


def _run_routed(s, c):
    import quantized_matmul_qgemv_amd as qmm
    if s["workspace"] is None:
        s["workspace"] = qmm.i8_grouped_workspace(s["x"])
    if c["op"] == "swiglu":
        return qmm.i8_moe_gate_up_swiglu(*s["weights"], s["x"], s["ids"], s["plan"], x_scales=s["x_scales"], h=s["y"],
                                         workspace=s["workspace"])
    w, ws = s["weights"][0]
    return qmm.i8_gemm_grouped(w, ws, s["x"], s["ids"], s["plan"], a_row_per_pair=True, a_scales=s["x_scales"], y=s["y"],
                               workspace=s["workspace"])


def _plain_rows(s):
    """(codes as fp32, scales): each row's largest magnitude stands at 127."""
    if s["x_scales"] is not None:
        return s["x"].float(), s["x_scales"]
    # 64 bits: whether a quotient lies above or below a half decides a whole number
    x = s["x"].double()
    scale = (x.abs().amax(dim=1) / 127).float()
    q = (x / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]).round()
    return q.clamp(-127, 127).float(), scale


def _plain_gemm(s, c):
    q, scale = _plain_rows(s)
    out = []
    for w, ws, bias, y in s["products"]:
        v = (q @ w.float().t()) * scale[:, None] * ws
        out.append((v if bias is None else v + bias).to(y.dtype))
    return out[0] if len(out) == 1 else out


def _plain_routed(s, c):
    """Expert by expert: its rows through its matrix, or through its two."""
    q, scale = _plain_rows(s)
    y, at = torch.empty_like(s["y"]), 0
    for e, count in enumerate(s["counts"]):
        if count == 0:
            continue
        pairs = s["order"][at:at + count]
        at += count
        rows = pairs if c["op"] == "grouped" else pairs // c["top_k"]
        v = [(q[rows] @ w[e].float().t()) * scale[rows, None] * ws[e] for w, ws in s["weights"]]
        y[pairs] = (v[0] if len(v) == 1 else v[0] / (1.0 + torch.exp(-v[0])) * v[1]).to(y.dtype)
    return y


# ------------------------------------------------------- what cannot be avoided

def work(case):
    c = case
    size = lambda name: TYPES[name].itemsize  # noqa: E731
    if c["op"] == "gemm":
        m, k, n = c["m"], c["k"], sum(_widths(c))
        return {"bytes": m * k * size(c["x"]) + (4 * m if c["x"] == "codes" else 0)
                + n * (k + 4 + (4 if c["bias"] else 0)) + m * n * size(c["y"]), "flops": 2 * m * n * k}
    pairs, two = c["t"] * c["top_k"], 2 if c["op"] == "swiglu" else 1
    rows = pairs if c["op"] == "grouped" else c["t"]
    used = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["t"])
    return {"bytes": int(rows * c["k"] * size(c["x"]) + (4 * rows if c["x"] == "codes" else 0) + 4 * pairs
                         + used * two * c["n"] * (c["k"] + 4) + pairs * c["n"] * size(c["y"])),
            "flops": 2 * pairs * two * c["n"] * c["k"]}


# ------------------------------------------------------------ in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["x_scales"] is None:
        top = x.abs().max(dim=1, keepdim=True).values
        step = (top / 127).float().double()
        x = torch.where(step > 0, torch.round(x / step), torch.zeros_like(x)) * step
    else:
        x = x * s["x_scales"].double()[:, None]
    if case["op"] == "gemm":
        out = []
        for w, ws, bias, _ in s["products"]:
            v = x @ (w.double() * ws.double()[:, None]).t()
            out.append(v if bias is None else v + bias.double())
        return out[0] if len(out) == 1 else out
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    ids = s["ids"].view(-1)
    for e in range(case["experts"]):
        pairs = (ids == e).nonzero()[:, 0]
        rows = pairs if case["op"] == "grouped" else pairs.div(case["top_k"], rounding_mode="floor")
        v = [x[rows] @ (w[e].double() * ws[e].double()[:, None]).t() for w, ws in s["weights"]]
        y[pairs] = v[0] if case["op"] == "grouped" else v[0] * torch.sigmoid(v[0]) * v[1]
    return y
