"""The dense base product with its epilogue, and a feed-forward block of experts: what a
serving step calls around ``lora_add_linear`` where the base weights are not microscaled.

    linear   z = x W^T + bias + addend, y = act(z) + residual; gated: W holds the gate's rows, then
             the up projection's, and y = act(z_gate) * z_up + residual.  The adapters' delta comes in as the
             addend (ahead of the activation) or as the residual (behind it)
    experts  the same per slot: slot i of expert ids[i] takes row i // x_div of x through the expert's own
             W; slots without an expert (-1) keep what their row of y held
    route    the k largest logits of a token (ties: the lowest expert), as expert ids and weights: softmax over all
             experts or a sigmoid of each, then scaled to a sum of one where `renorm` says so, times `scale`.  Experts
             masked with -infinity are never chosen: -1 and weight 0 in their place
    sum      the way back: a token's rows, weighted, and the residual
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


# ------------------------------------------------------------------------ cases
def _linear(name, T, d, n, dtype="bf16", act="none", gated=False, bias=False, addend=False, residual=False):
    return {"name": name, "op": "linear", "T": T, "d": d, "n": n, "dtype": dtype, "act": act, "gated": gated,
            "bias": bias, "addend": addend, "residual": residual}


def _experts(name, T, k, E, d, n, x_div, dtype="bf16", act="none", gated=False, bias=False):
    return {"name": name, "op": "experts", "T": T, "k": k, "E": E, "d": d, "n": n, "x_div": x_div, "dtype": dtype,
            "act": act, "gated": gated, "bias": bias}


def listed():
    return [
        # one token through an output projection into the residual stream: latency, and the weight's bytes
        _linear("linear 1 x 4096 x 4096", 1, 4096, 4096, residual=True),
        # a decode batch through gate and up, the adapters' delta ahead of the activation: the weight's bytes
        _linear("linear 64 x 4096 x 2 x 14336", 64, 4096, 14336, act="silu", gated=True, addend=True),
        # a short prompt, an odd number of rows, the down projection's long sums
        _linear("linear 257 x 14336 x 4096", 257, 14336, 4096, residual=True),
        # many prompts through gate and up: the tensor cores' rate
        _linear("linear 8192 x 4096 x 2 x 14336", 8192, 4096, 14336, act="silu", gated=True),
        # fp32, sizes that suit no tile, every operand of the epilogue
        _linear("linear 333 x 1003 x 777 fp32", 333, 1003, 777, dtype="fp32", act="gelu", bias=True, addend=True,
                residual=True),
        # a decode batch, two of eight experts a token: the bytes of the experts that it reaches
        _experts("experts 8 tokens, 2 of 8, 4096 x 2 x 14336", 8, 2, 8, 4096, 14336, 2, act="silu", gated=True),
        # prompts over many small experts: ragged groups, rows gathered by token
        _experts("experts 8192 tokens, 4 of 64, 2048 x 2 x 1024", 8192, 4, 64, 2048, 1024, 4, act="silu", gated=True),
        # fp32, the way down (a row a slot), odd sizes, a bias of each expert
        _experts("experts 77 tokens, 3 of 5, 259 x 130 fp32", 77, 3, 5, 259, 130, 1, dtype="fp32", bias=True),
        # one token's choice: latency
        {"name": "route 1 x 64", "op": "route", "T": 1, "E": 64, "k": 8, "dtype": "fp32", "score": "softmax",
         "renorm": True, "scale": 1.0, "masked": 0.0},
        # a prompt batch's choice among many experts, part of them closed
        {"name": "route 8192 x 256", "op": "route", "T": 8192, "E": 256, "k": 8, "dtype": "bf16", "score": "sigmoid",
         "renorm": True, "scale": 2.5, "masked": 0.1},
        # an odd decode batch's rows back to their tokens
        {"name": "sum 33 x 8 x 2048", "op": "sum", "T": 33, "k": 8, "d": 2048, "dtype": "fp32", "residual": True},
        # a prompt batch's rows back to their tokens
        {"name": "sum 8192 x 4 x 4096", "op": "sum", "T": 8192, "k": 4, "d": 4096, "dtype": "bf16", "residual": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """A width: any integer one time in four, else a multiple of 8 or of 128."""
    n = _log_int(rng, lo, hi)
    step = rng.choice([1, 8, 8, 128])
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "experts", "route", "sum"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "route":
        E = _log_int(rng, 2, 1024)
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 16)), "dtype": dtype,
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.1, 0.9])}
    if op == "sum":
        d, k = _width(rng, 64, 8192), rng.randint(1, 8)
        return {"op": op, "T": _log_int(rng, 1, min(16384, 8192 * 4 * 4096 // (d * k))), "k": k, "d": d, "dtype": dtype,
                "residual": rng.random() < 0.7}
    gated = rng.random() < 0.4
    case = {"op": op, "dtype": dtype, "act": rng.choice(ACTS), "gated": gated, "bias": rng.random() < 0.3}
    most = 8192 * 4096 * 28672 // (8 if dtype == "fp32" else 1)   # products of the largest listed case
    if op == "linear":
        case["d"], case["n"] = _width(rng, 64, 14336), _width(rng, 64, 14336)
        case["T"] = _log_int(rng, 1, max(1, min(8192, most // (case["d"] * case["n"] * (2 if gated else 1)))))
        case["addend"], case["residual"] = rng.random() < 0.3, rng.random() < 0.4
        return case
    case["E"] = _log_int(rng, 2, 128)
    case["k"] = rng.randint(1, min(case["E"], 8))
    top = 7 * 4096 * 28672 // (4 if dtype == "fp32" else 1) // case["E"] // (2 if gated else 1)   # elements of one W
    case["d"] = _width(rng, 64, 4096)
    case["n"] = _width(rng, 64, min(14336, top // case["d"]))
    products = case["d"] * case["n"] * (2 if gated else 1) * case["k"]
    rows = (1 << 28) // (case["k"] * max(case["d"], case["n"]))
    case["T"] = _log_int(rng, 1, max(1, min(8192, most // products, rows)))
    case["x_div"] = rng.choice([1, case["k"]])
    return case


# ------------------------------------------------------------------------ inputs
def _activations(T, d, g):
    """Rows as a transformer has them: unit scale, channels of uneven size."""
    channel = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    return torch.randn(T, d, generator=g, device="cuda") * channel


def _weight(rows, d, dt, g):
    """[rows][d] of unit row norm, in pieces: the largest have a billion elements."""
    w = torch.empty(rows, d, dtype=dt, device="cuda")
    step = max(1, (1 << 26) // d)
    for lo in range(0, rows, step):
        w[lo:lo + step] = torch.randn(min(step, rows - lo), d, generator=g, device="cuda") / d ** 0.5
    return w


def _choices(T, k, E, g):
    """Expert ids [T, k] as a router gives them: some experts liked more than others, one slot in 50 left out
    (an expert that another device holds)."""
    liking = torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(torch.randn(T, E, generator=g, device="cuda") + liking, k, dim=1).indices.to(torch.int32)
    out = torch.rand(T, k, generator=g, device="cuda") < 0.02
    return torch.where(out, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, T = DTYPE[case["dtype"]], case["op"], case["T"]
    s = {"case": case, "op": op}

    def rows(m, n, scale=1.0):
        return (scale * torch.randn(m, n, generator=g, device="cuda")).to(dt)

    if op == "route":
        x = 2 * torch.randn(T, case["E"], generator=g, device="cuda")
        closed = torch.rand(T, case["E"], generator=g, device="cuda") < case["masked"]
        s["logits"] = torch.where(closed, torch.full_like(x, -math.inf), x).to(dt)
        s["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
        return s
    if op == "sum":
        k, d = case["k"], case["d"]
        s["x"] = rows(T * k, d)
        s["ids"] = _choices(T, k, 64, g)
        s["weights"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        s["residual"] = rows(T, d, 4.0) if case["residual"] else None
        s["y"] = torch.empty(T, d, dtype=dt, device="cuda")
        return s
    d, n = case["d"], case["n"]
    n_w = 2 * n if case["gated"] else n
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "linear":
        s["x"] = _activations(T, d, g).to(dt)
        s["W"] = _weight(n_w, d, dt, g)
        s["bias"] = rows(1, n_w)[0] if case["bias"] else None
        s["addend"] = rows(T, n_w, 0.5) if case["addend"] else None
        s["residual"] = rows(T, n, 4.0) if case["residual"] else None
        s["y"] = torch.empty(T, n, dtype=dt, device="cuda")
        return s
    E, k = case["E"], case["k"]
    slots = T * k
    s["x"] = _activations(-(-slots // case["x_div"]), d, g).to(dt)
    s["W"] = _weight(E * n_w, d, dt, g).view(E, n_w, d)
    s["bias"] = rows(E, n_w) if case["bias"] else None
    s["ids"] = _choices(T, k, E, g).view(-1)
    s["y"] = torch.zeros(slots, n, dtype=dt, device="cuda")
    if own:
        import lora_adapter_application_b200 as lora
        s["meta"] = lora.Meta(slots, E, min_run=0)
        lora.lora_build_segments(s["ids"], s["meta"], s["status"])
    else:
        s["groups"] = [torch.nonzero(s["ids"] == e)[:, 0] for e in range(E)]   # the slots of each expert
    return s


# ------------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import lora_adapter_application_b200 as lora
    c = s["case"]
    if s["op"] == "route":
        score = lora.SCORE_SOFTMAX if c["score"] == "softmax" else lora.SCORE_SIGMOID
        lora.lora_expert_route(s["ids"], s["weights"], s["logits"], score=score, renormalize=c["renorm"],
                               scale=c["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if s["op"] == "sum":
        lora.lora_expert_sum(s["y"], s["x"], s["ids"], s["weights"], 64, residual=s["residual"])
        return {"y": s["y"]}
    act = {"none": lora.ACT_NONE, "silu": lora.ACT_SILU, "gelu": lora.ACT_GELU, "gelu_tanh": lora.ACT_GELU_TANH,
           "relu": lora.ACT_RELU}[c["act"]]
    if s["op"] == "linear":
        lora.lora_linear(s["y"], s["x"], s["W"], s["status"], bias=s["bias"], addend=s["addend"],
                         residual=s["residual"], act=act, gated=c["gated"])
    else:
        lora.lora_expert_linear(s["y"], s["x"], s["W"], s["meta"], s["status"], x_div=c["x_div"], bias=s["bias"],
                                act=act, gated=c["gated"])
    return {"y": s["y"]}


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":   # (1 + tanh u) / 2 is 1 / (1 + exp(-2 u))
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def _finish(z, c):
    """Activation and gate of z (fp32)."""
    if not c["gated"]:
        return _act(z, c["act"])
    return _act(z[:, :c["n"]], c["act"]) * z[:, c["n"]:]


def _run_plain(s):
    c = s["case"]
    dt = DTYPE[c["dtype"]]
    if s["op"] == "route":
        x = s["logits"].float()
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        top, ids = top[:, :c["k"]], ids[:, :c["k"]].to(torch.int32)
        closed = top == -math.inf
        most = x.max(1, keepdim=True).values
        if c["score"] == "softmax":
            w = torch.exp(top - most) / torch.exp(x - most).sum(1, keepdim=True)
        else:
            w = 1 / (1 + torch.exp(-top))
        w = torch.where(closed, torch.zeros_like(w), w)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = torch.where(closed, torch.zeros_like(w), w * c["scale"])
        return {"ids": torch.where(closed, torch.full_like(ids, -1), ids), "weights": w}
    if s["op"] == "sum":
        x = s["x"].float().view(c["T"], c["k"], c["d"])
        there = (s["ids"] >= 0)[:, :, None]
        y = torch.where(there, x * s["weights"][:, :, None], torch.zeros_like(x)).sum(1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt)}
    if s["op"] == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        if s["addend"] is not None:
            z = z + s["addend"].float()
        y = _finish(z, c)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt)}
    y = torch.zeros_like(s["y"])
    for e, slots in enumerate(s["groups"]):
        if slots.numel() == 0:
            continue
        z = s["x"][slots // c["x_div"]].float() @ s["W"][e].float().t()
        if s["bias"] is not None:
            z = z + s["bias"][e].float()
        y[slots] = _finish(z, c).to(dt)
    return {"y": y}


# ------------------------------------------------------------------------ accounting
def work(case):
    """Each input read once, each output written once; a multiply and an add count two.  Of the experts, those
    that T tokens of k independent choices are expected to reach."""
    T, es = case["T"], DTYPE[case["dtype"]].itemsize
    if case["op"] == "route":
        return {"bytes": T * (case["E"] * es + 8 * case["k"]), "flops": 4.0 * T * case["E"]}
    if case["op"] == "sum":
        k, d = case["k"], case["d"]
        return {"bytes": T * ((k + 1 + case["residual"]) * d * es + 8 * k), "flops": 2.0 * T * k * d}
    d, n = case["d"], case["n"]
    n_w = 2 * n if case["gated"] else n
    if case["op"] == "linear":
        rows = d + n + n_w * case["addend"] + n * case["residual"]
        return {"bytes": es * (T * rows + n_w * (d + case["bias"])), "flops": 2.0 * T * d * n_w}
    E, slots = case["E"], T * case["k"]
    hit = E * (1 - (1 - case["k"] / E) ** T)
    return {"bytes": es * (slots / case["x_div"] * d + slots * n + hit * n_w * (d + case["bias"])) + 4 * slots,
            "flops": 2.0 * slots * d * n_w}


# ------------------------------------------------------------------- 64-bit values
def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return torch.clamp(z, min=0) if act == "relu" else z


def _exact_rows(x, w, bias, addend, case):
    """The operator's rows in 64 bits, some columns of y at a time."""
    n = case["n"]
    y = torch.empty(x.shape[0], n, dtype=torch.float64, device=x.device)
    x = x.double()

    def part(lo, hi):
        z = torch.einsum("td,nd->tn", x, w[lo:hi].double())
        if bias is not None:
            z += bias[lo:hi].double()
        if addend is not None:
            z += addend[:, lo:hi].double()
        return z

    step = 4096
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        v = _exact_act(part(lo, hi), case["act"])
        if case["gated"]:
            v *= part(n + lo, n + hi)
        y[:, lo:hi] = v
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x, k = s["logits"].double(), case["k"]
        order = torch.argsort(-x, dim=1, stable=True)
        ids = order[:, :k]
        top = torch.gather(x, 1, ids)
        if case["score"] == "softmax":
            w = torch.gather(torch.softmax(x, 1), 1, ids)
        else:
            w = torch.sigmoid(top)
        gone = torch.isneginf(top)
        w = w.masked_fill(gone, 0)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = (case["scale"] * w).masked_fill(gone, 0)
        return {"ids": ids.masked_fill(gone, -1).to(torch.int32), "weights": w}
    if case["op"] == "sum":
        y = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            y += s["residual"].double()
        for j in range(case["k"]):
            w = torch.where(s["ids"][:, j] >= 0, s["weights"][:, j].double(), 0.0)
            y += w[:, None] * s["x"][j::case["k"]].double()
        return {"y": y}
    if case["op"] == "linear":
        y = _exact_rows(s["x"], s["W"], s["bias"], s["addend"], case)
        if s["residual"] is not None:
            y += s["residual"].double()
        return {"y": y}
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    slot = torch.arange(s["ids"].numel(), device="cuda")
    for e in range(case["E"]):
        mine = slot[s["ids"] == e]
        if mine.numel():
            x = s["x"][torch.div(mine, case["x_div"], rounding_mode="floor")]
            y[mine] = _exact_rows(x, s["W"][e], None if s["bias"] is None else s["bias"][e], None, case)
    return {"y": y}
