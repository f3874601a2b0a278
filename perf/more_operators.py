"""The router, microscaled 4-bit floating point and the layer for a few tokens: their cases,
inputs and plain forms.

  route           top-k experts and their scores from each token's logits
  route_backward  the logits' gradient from the scores' gradient
  quantize        a matrix to 4-bit floating point with block scales, and back
  fp4_experts     tokens quantised on their way to the experts' receive rows, and the product
                  (or the gated feed-forward block) of these rows with 4-bit weights
  layer           a whole mixture-of-experts layer for a few tokens

A case names one operator and its sizes. ``own`` false: the plain forms, elementary torch
operations in 32 bits (64 next to a border of the 4-bit grid), rounded once at the end.
``own`` true: the package's entry points.
"""
import math

import torch

own = False

_BF16 = torch.bfloat16
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = {"mx": 32, "nv": 16}       # elements that share a scale


def listed():
    return [
        # The router of one decode batch: 64 tokens over 256 experts, scores from sigmoids.
        {"name": "route decode", "op": "route", "tokens": 64, "experts": 256, "topk": 8,
         "score": "sigmoid", "normalize": True, "masked": 0.0, "type": "f32"},
        # The 32k prefill workload's tokens; logits as a bf16 projection leaves them (many ties),
        # with padded tokens and experts that a token may not reach.
        {"name": "route prefill", "op": "route", "tokens": 32768, "experts": 256, "topk": 8,
         "score": "softmax", "normalize": True, "masked": 0.1, "type": "bf16"},
        # A micro-batch of a small model's training step, 16 experts.
        {"name": "route backward small", "op": "route_backward", "tokens": 331, "experts": 16,
         "topk": 4, "score": "softmax", "normalize": False, "masked": 0.0, "type": "f32"},
        # The training step of the 32k tokens.
        {"name": "route backward", "op": "route_backward", "tokens": 32768, "experts": 256,
         "topk": 8, "score": "sigmoid", "normalize": True, "masked": 0.0, "type": "f32"},
        # A step's activations, an odd number of rows.
        {"name": "quantize rows 333", "op": "quantize", "experts": 1, "rows": 333, "cols": 1024,
         "format": "mx", "tensor_scale": False},
        # The gate and up weights of the mixtral workload's 8 experts, each with its scale.
        {"name": "quantize weights", "op": "quantize", "experts": 8, "rows": 4096, "cols": 4096,
         "format": "nv", "tensor_scale": True},
        # A micro-batch of a small model, one projection, a tenth of the pairs dropped.
        {"name": "fp4 small", "op": "fp4_experts", "tokens": 331, "hidden": 1024, "inter": 512,
         "experts": 16, "topk": 4, "routing": "uniform", "drop": 0.1, "format": "mx",
         "block": False, "act": "silu"},
        # The experts' block on the mixtral workload's rows.
        {"name": "fp4 mixtral", "op": "fp4_experts", "tokens": 4096, "hidden": 4096,
         "inter": 2048, "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0,
         "format": "nv", "block": True, "act": "silu"},
        # The block on the deepseek workload's rows, skewed over 256 experts.
        {"name": "fp4 deepseek", "op": "fp4_experts", "tokens": 8192, "hidden": 7168,
         "inter": 2048, "experts": 256, "topk": 8, "routing": "zipf", "drop": 0.0,
         "format": "nv", "block": True, "act": "silu"},
        # One decoded token through 2 of the mixtral workload's 8 experts, bf16 weights.
        {"name": "layer 1 bf16", "op": "layer", "tokens": 1, "hidden": 4096, "inter": 2048,
         "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "weights": "bf16",
         "act": "silu"},
        # One decoded token through 8 of the deepseek workload's 256 experts, 4-bit weights.
        {"name": "layer 1 fp4", "op": "layer", "tokens": 1, "hidden": 7168, "inter": 2048,
         "experts": 256, "topk": 8, "routing": "uniform", "drop": 0.0, "weights": "nv",
         "act": "silu"},
        # A decode batch of 16 tokens on the same layer.
        {"name": "layer 16 fp4", "op": "layer", "tokens": 16, "hidden": 7168, "inter": 2048,
         "experts": 256, "topk": 8, "routing": "uniform", "drop": 0.0, "weights": "mx",
         "act": "gelu"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    largest = {}
    for c in listed():
        w = work(c)
        cost = largest.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in cost:
            cost[k] = max(cost[k], w[k])
    op = rng.choice(["route", "route_backward", "quantize", "fp4_experts", "fp4_experts", "layer",
                     "layer"])
    while True:
        case = {"op": op}
        if op in ("route", "route_backward"):
            case["tokens"] = _log_between(rng, 1, 32768)
            case["experts"] = rng.choice([1, 5, 8, 16, 33, 64, 160, 256])
            case["topk"] = min(case["experts"], rng.choice([1, 2, 4, 6, 8]))
            case["score"] = rng.choice(["softmax", "sigmoid"])
            case["normalize"] = rng.choice([True, False])
            case["masked"] = rng.choice([0.0, 0.1, 0.5])
            case["type"] = rng.choice(["f32", "bf16"])
        elif op == "quantize":
            case["experts"] = rng.choice([1, 2, 8])
            case["rows"] = _log_between(rng, 1, 4096)
            case["cols"] = 128 * _log_between(rng, 1, 56)
            case["format"] = rng.choice(["mx", "nv"])
            case["tensor_scale"] = case["format"] == "nv" and rng.choice([True, False])
        else:
            case["hidden"] = 128 * _log_between(rng, 2, 56)
            case["inter"] = 128 * _log_between(rng, 1, 16)
            case["experts"] = rng.choice([1, 2, 5, 8, 16, 33, 64, 256])
            case["topk"] = min(case["experts"], rng.choice([1, 2, 4, 8]))
            case["routing"] = rng.choice(["uniform", "zipf"])
            case["drop"] = rng.choice([0.0, 0.1])
            case["act"] = rng.choice(["silu", "gelu"])
            if op == "fp4_experts":
                case["tokens"] = _log_between(rng, 1, 8192)
                case["format"] = rng.choice(["mx", "nv"])
                case["block"] = rng.choice([True, False])
            else:
                case["tokens"] = _log_between(rng, 1, 32)
                case["weights"] = rng.choice(["bf16", "mx", "nv"])
        w = work(case)
        if all(w[k] <= largest[op][k] for k in w):
            return case


def _popularity(case):
    if case["routing"] == "uniform":
        return [1.0 / case["experts"]] * case["experts"]
    w = [(e + 1) ** -1.1 for e in range(case["experts"])]
    s = sum(w)
    return [v / s for v in w]


def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, K = case["tokens"], case["experts"], case["topk"]
        size = 2 if case["type"] == "bf16" else 4
        if op == "route":
            select = T * E * 4 if case["masked"] else 0
            return {"bytes": T * E * size + select + T * K * 8, "flops": T * E * 4}
        return {"bytes": 2 * T * E * size + T * K * 8, "flops": T * E * 6}
    if op == "quantize":
        n = case["experts"] * case["rows"] * case["cols"]
        # Read, written in 4 bits with scales, read back and written.
        return {"bytes": n * (2 + 2 * (0.5 + 1 / _BLOCK[case["format"]]) + 2), "flops": n * 6}
    T, D, F, E, K = (case[k] for k in ("tokens", "hidden", "inter", "experts", "topk"))
    rows = T * K * (1.0 - case["drop"])
    # Experts that the call's tokens reach (expected over the routing).
    used = sum(1.0 - (1.0 - min(1.0, K * p * (1.0 - case["drop"]))) ** T for p in _popularity(case))
    if op == "fp4_experts":
        per = 0.5 + 1 / _BLOCK[case["format"]]
        m = 3 * F if case["block"] else F       # rows of D weights that an expert has
        # Tokens in, weights, results; the quantised rows out and in again.
        inner = D + (F if case["block"] else 0)
        return {"bytes": T * D * 2 + used * D * m * per + rows * (D if case["block"] else F) * 2
                + 2 * rows * inner * per, "flops": rows * 2 * D * m}
    per = 2 if case["weights"] == "bf16" else 0.5 + 1 / _BLOCK[case["weights"]]
    return {"bytes": used * 3 * D * F * per + 2 * T * D * 2 + T * K * 8,
            "flops": rows * 6 * D * F}


def _normal(gen, shape, std):
    t = torch.empty(shape, dtype=_BF16, device="cuda")
    return t.normal_(0.0, std, generator=gen)


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _random_fp4(gen, shape, fmt):
    """Codes and scales (the values they stand for: about unit-variance products) of weights
    [E, rows, cols], and each expert's scale."""
    E, rows, cols = shape
    codes = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda",
                          generator=gen)
    # Block scales spread over two binades below their largest.
    blocks = (E, rows, cols // _BLOCK[fmt])
    r = torch.rand(blocks, device="cuda", generator=gen)
    if fmt == "mx":
        base = round(math.log2(1.0 / (3.3 * math.sqrt(cols))))
        scales = (base - 1 + torch.floor(3 * r) + 127).to(torch.uint8)
        return codes, scales, None
    scales = _e4m3_bits(64.0 + 192.0 * r)
    ts = (0.5 + torch.rand(E, device="cuda", generator=gen)) / (160 * 3.3 * math.sqrt(cols))
    return codes, scales, ts


def _e4m3_bits(v):
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    op = case["op"]
    if own:
        import combine_topk_ids_expert_gb300 as ep
        state["ep"] = ep
    if op in ("route", "route_backward"):
        T, E, K = case["tokens"], case["experts"], case["topk"]
        logits = torch.randn((T, E), device="cuda", generator=gen).mul_(1.5)
        state["logits"] = logits.to(_TYPES[case["type"]])
        if case["masked"]:
            # What the experts are chosen by: the logits, and nothing where a token may not go;
            # the last tokens are padding.
            off = torch.rand((T, E), device="cuda", generator=gen) < case["masked"]
            off[T - T // 16:] = True
            state["select"] = torch.where(off, -math.inf, state["logits"].float())
        else:
            state["select"] = None
        if op == "route_backward":
            state["grad"] = torch.randn((T, K), device="cuda", generator=gen)
            pick = state["logits"].float() if state["select"] is None else state["select"]
            state["ids"] = _choose(pick, K)
        return state
    if op == "quantize":
        E, rows, cols = case["experts"], case["rows"], case["cols"]
        std = 1.0 if E == 1 else cols ** -0.5
        x = _normal(gen, (E, rows, cols), std)
        # A few columns carry much larger values, as activations and weights do.
        x[..., torch.randperm(cols, device="cuda", generator=gen)[:cols // 64]] *= 16
        state["x"] = x
        state["tensor_scale"] = None
        if case["tensor_scale"]:
            state["tensor_scale"] = x.abs().amax((1, 2)).float() / (448 * 6)
        return state
    T, D, F, E, K = (case[k] for k in ("tokens", "hidden", "inter", "experts", "topk"))
    # Routing: K distinct experts for each token by popularity; some pairs dropped.
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen)))
    noise += torch.tensor(_popularity(case), device="cuda").log()
    ids = noise.topk(K, dim=1).indices.to(torch.int32)
    dropped = torch.randperm(T * K, device="cuda", generator=gen)[:round(case["drop"] * T * K)]
    ids.view(-1)[dropped] = -1
    scores = torch.rand((T, K), device="cuda", generator=gen).add_(0.1)
    scores /= scores.sum(1, keepdim=True)
    state.update(ids=ids, scores=scores, x=_normal(gen, (T, D), 1.0))
    flat = ids.flatten()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.bincount(flat[flat >= 0], minlength=E).tolist()
    n, spans = 0, []
    for e, c in enumerate(counts):
        if c:
            spans.append((e, n, n + c))
        n += c
    # Experts with rows, their first rows and ends; the (token, k) pair of each row.
    state.update(n=n, spans=spans, pairs=order[:n],
                 spans_gpu=torch.tensor(spans, device="cuda", dtype=torch.int64).view(-1, 3))
    if op == "fp4_experts":
        fmt = case["format"]
        if case["block"]:
            state["w_gate_up"] = _random_fp4(gen, (E, 2 * F, D), fmt)
            state["w_down"] = _random_fp4(gen, (E, D, F), fmt)
        else:
            state["w"] = _random_fp4(gen, (E, F, D), fmt)
    elif case["weights"] == "bf16":
        state["w_gate_up"] = _normal(gen, (E, 2 * F, D), D ** -0.5)
        state["w_down"] = _normal(gen, (E, D, F), F ** -0.5)
    else:
        state["w_gate_up"] = _random_fp4(gen, (E, 2 * F, D), case["weights"])
        state["w_down"] = _random_fp4(gen, (E, D, F), case["weights"])
    if own:
        ep = state["ep"]
        state["buf"] = ep.Buffer(num_max_tokens_per_rank=T, hidden=D, num_experts=E, num_ranks=1,
                                 topk=K, dtype=_BF16, layout="packed")
        for k in ("w", "w_gate_up", "w_down"):
            if isinstance(state.get(k), tuple):
                codes, scales, ts = state[k]
                fmt = case["format"] if op == "fp4_experts" else case["weights"]
                state[k] = ep.FP4(codes, ep.tile_fp4_scales(scales), fmt, ts)
    return state


# ---- plain forms ---------------------------------------------------------------------


def _choose(select, k):
    """The k largest of each row, ties to the lowest index; -1 for what must not be chosen."""
    order = torch.sort(select, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    return torch.where(order.values[:, :k] > -math.inf, ids, -1).to(torch.int32)


def _probabilities(logits, score):
    v = logits.float()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    e = torch.exp(v - v.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    case = s["case"]
    ids = _choose(s["logits"].float() if s["select"] is None else s["select"], case["topk"])
    p = _probabilities(s["logits"], case["score"]).gather(1, ids.clamp(min=0).long())
    p = torch.where(ids >= 0, p, 0.0)
    if case["normalize"]:
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return {"ids": ids, "scores": p}


def _plain_route_backward(s):
    case, ids = s["case"], s["ids"]
    there = ids >= 0
    at = ids.clamp(min=0).long()
    p = _probabilities(s["logits"], case["score"])
    chosen = torch.where(there, p.gather(1, at), 0.0)
    g = torch.where(there, s["grad"], 0.0)
    if case["normalize"]:
        total = chosen.sum(1, keepdim=True)
        share = torch.where(total > 0, chosen / total, 0.0)
        g = torch.where(total > 0, (g - (g * share).sum(1, keepdim=True)) / total, 0.0)
    g = torch.where(there, g, 0.0)
    full = torch.zeros_like(p).scatter_add_(1, at, g)
    if case["score"] == "sigmoid":
        grad = full * p * (1.0 - p)
    else:
        grad = p * (full - (g * chosen).sum(1, keepdim=True))
    return {"grad_logits": grad.to(s["logits"].dtype)}


def _nearest(a, step):
    """a (not negative) to the nearest multiple of step, ties to the even one."""
    return torch.round(a / step) * step


def _plain_quantize(x, fmt, tensor_scale):
    """(4-bit values, block scales) of x [.., cols] in 64 bits, tensor_scale's shape [..]."""
    v = x.double().unflatten(-1, (-1, _BLOCK[fmt]))
    most = v.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        exponent = torch.frexp(most).exponent - 1
        scale = torch.exp2((exponent - 2).clamp(-127, 127).double())
        unit = scale = torch.where(most > 0, scale, 2.0 ** -127)
    else:
        g = 1.0 if tensor_scale is None else tensor_scale.double()[..., None, None]
        t = (most / (6 * g)).clamp(max=448)
        exponent = (torch.frexp(t).exponent - 1).clamp(min=-6)
        scale = _nearest(t, torch.exp2((exponent - 3).double()))
        unit = scale * g
    a = torch.where(unit > 0, v.abs() / unit, 0.0).clamp(max=6)
    q = _nearest(a, torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)))
    return torch.copysign(q, v), scale


def _plain_quantize_and_back(s):
    x, ts = s["x"], s["tensor_scale"]
    out = torch.empty_like(x)
    for e in range(x.shape[0]):
        g = None if ts is None else ts[e].expand(x.shape[1])
        q, scale = _plain_quantize(x[e], s["case"]["format"], g)
        v = (q * scale).float() * (1.0 if ts is None else ts[e])
        out[e] = v.flatten(-2).to(_BF16)
    return {"values": out}


def _fp4_values(w, used, fmt):
    """The used experts' 4-bit weights in 32 bits."""
    codes, scales, ts = w
    c = codes[used]
    c = torch.stack((c & 15, c >> 4), dim=-1).flatten(-2).int()
    v = torch.tensor(_GRID + tuple(-g for g in _GRID), device="cuda")[c]
    if fmt == "mx":
        s = torch.exp2(scales[used].float() - 127)
    else:
        s = scales[used].view(torch.float8_e4m3fn).float() * ts[used][:, None, None]
    return (v.unflatten(-1, (-1, _BLOCK[fmt])) * s[..., None]).flatten(-2)


def _weights(w, used, fmt):
    return w[used].float() if isinstance(w, torch.Tensor) else _fp4_values(w, used, fmt)


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _batches(state):
    """(experts, their rows [experts, C], which of these are rows) for products of many experts
    at once; one expert at a time where their row counts differ too much for that."""
    spans, gpu = state["spans"], state["spans_gpu"]
    most = max((hi - lo for _, lo, hi in spans), default=0)
    if most * len(spans) <= 4 * state["n"] + 1024:
        parts = [(gpu[i:i + 32], most) for i in range(0, len(spans), 32)]
    else:
        parts = [(gpu[i:i + 1], hi - lo) for i, (_, lo, hi) in enumerate(spans)]
    for part, c in parts:
        at = part[:, 1:2] + torch.arange(c, device="cuda")
        here = at < part[:, 2:3]
        yield part[:, 0], torch.where(here, at, 0), here


def _plain_fp4_experts(s):
    case, F = s["case"], s["case"]["inter"]
    q, scale = _plain_quantize(s["x"], case["format"], None)
    x = (q * scale).float().flatten(-2)[s["pairs"] // case["topk"]]
    y = torch.empty((s["n"], case["hidden"] if case["block"] else F), dtype=_BF16, device="cuda")
    for used, at, here in _batches(s):
        r = torch.where(here[..., None], x[at], 0.0)
        if case["block"]:
            r = r @ _fp4_values(s["w_gate_up"], used, case["format"]).mT
            q, scale = _plain_quantize(_act(r[..., :F], case["act"]) * r[..., F:], case["format"],
                                       None)
            r = (q * scale).float().flatten(-2) @ _fp4_values(s["w_down"], used, case["format"]).mT
        else:
            r = r @ _fp4_values(s["w"], used, case["format"]).mT
        y[at[here]] = r[here].to(_BF16)
    return {"y": y}


def _plain_layer(s):
    case, F, K = s["case"], s["case"]["inter"], s["case"]["topk"]
    x = s["x"].float()[s["pairs"] // K]
    y = torch.zeros((s["scores"].numel(), s["x"].shape[1]), device="cuda")
    for used, at, here in _batches(s):
        gu = torch.where(here[..., None], x[at], 0.0) @ _weights(s["w_gate_up"], used,
                                                                 case["weights"]).mT
        h = _act(gu[..., :F], case["act"]) * gu[..., F:]
        r = h @ _weights(s["w_down"], used, case["weights"]).mT
        y[s["pairs"][at[here]]] = r[here]
    y = y.view(*s["scores"].shape, -1) * s["scores"][..., None]
    return {"out": y.sum(1).to(_BF16)}


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        if op == "quantize":
            return _plain_quantize_and_back(state)
        return {"route": _plain_route, "route_backward": _plain_route_backward,
                "fp4_experts": _plain_fp4_experts, "layer": _plain_layer}[op](state)
    ep = state["ep"]
    if op == "route":
        ids, scores = ep.route(state["logits"], case["topk"], score=case["score"],
                               normalize=case["normalize"], select=state["select"])
        return {"ids": ids, "scores": scores}
    if op == "route_backward":
        return {"grad_logits": ep.route_backward(state["grad"], state["logits"], state["ids"],
                                                 score=case["score"],
                                                 normalize=case["normalize"])}
    if op == "quantize":
        q = ep.quantize_fp4(state["x"], case["format"], state["tensor_scale"])
        return {"values": q.dequantize(_BF16)}
    buf = state["buf"]
    if op == "fp4_experts":
        d = buf.dispatch_fp4(state["x"], state["scores"], state["ids"], format=case["format"])
        if case["block"]:
            y = buf.expert_ffn_fp4(d.recv_x, state["w_gate_up"], state["w_down"], act=case["act"])
        else:
            y = buf.expert_gemm_fp4(d.recv_x, state["w"])
        return {"y": y[:state["n"]]}
    return {"out": buf.moe_layer(state["x"], state["scores"], state["ids"], state["w_gate_up"],
                                 state["w_down"], act=case["act"])}


# ---- in 64 bits --------------------------------------------------------------------------


def exact(case, seed):
    if case["op"] in ("fp4_experts", "layer") and work(case)["flops"] > 1.2e13:
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    f64, inf = torch.float64, math.inf
    op = case["op"]

    def gate(g):
        if case["act"] == "silu":
            return g * torch.special.expit(g)
        inner = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        return g * torch.special.expit(2.0 * inner)        # (1 + tanh v) / 2 = expit(2 v)

    if op in ("route", "route_backward"):
        logits = s["logits"].to(f64)
        p = torch.special.expit(logits) if case["score"] == "sigmoid" \
            else torch.softmax(logits, dim=1)
        if op == "route":
            # One expert after the other: the first of the largest that are left.
            left = (logits if s["select"] is None else s["select"].to(f64)).clone()
            ids, E = [], case["experts"]
            column = torch.arange(E, device="cuda")
            for _ in range(case["topk"]):
                most = left.amax(1, keepdim=True)
                first = torch.where(left == most, column, E).amin(1)
                first = torch.where(most[:, 0] == -inf, -1, first)
                ids.append(first)
                left[column == first[:, None]] = -inf
            ids = torch.stack(ids, dim=1)
        else:
            ids = s["ids"].long()
        here = ids >= 0
        chosen = torch.zeros_like(p)
        rows = torch.arange(p.shape[0], device="cuda")[:, None].expand_as(ids)
        chosen[rows[here], ids[here]] = 1.0
        total = (p * chosen).sum(1, keepdim=True) if case["normalize"] else torch.ones_like(p[:, :1])
        if op == "route":
            scores = torch.zeros(ids.shape, dtype=f64, device="cuda")
            scores[here] = (p / total)[rows[here], ids[here]]
            return {"ids": ids.to(torch.int32), "scores": scores.nan_to_num(0.0)}
        g = torch.zeros_like(p)
        g[rows[here], ids[here]] = s["grad"].to(f64)[here]
        scores = torch.where(total > 0, p * chosen / total, 0.0)
        # d scores_i / d p_j = ([i = j] - scores_i) / total where normalised, over the chosen.
        dp = g / total
        if case["normalize"]:
            dp = chosen * (g - torch.einsum("te,te->t", g, scores)[:, None]) / total
        dp = torch.where(total > 0, dp, 0.0)
        if case["score"] == "sigmoid":
            return {"grad_logits": dp * p * torch.special.expit(-logits)}
        return {"grad_logits": p * dp - p * torch.einsum("te,te->t", p, dp)[:, None]}

    grid = torch.tensor(_GRID, dtype=f64, device="cuda")
    middle = (grid[1:] + grid[:-1]) / 2

    def fp4(x, fmt, g):
        """Values that x [.., cols] stands for after quantisation, by the grid's midpoints."""
        v = x.to(f64).unflatten(-1, (-1, _BLOCK[fmt]))
        most = v.abs().amax(-1, keepdim=True)
        if fmt == "mx":
            e = torch.floor(torch.log2(most.clamp(min=2.0 ** -149)))
            e = torch.where(torch.exp2(e) > most, e - 1, e)
            e = torch.where(torch.exp2(e + 1) <= most, e + 1, e)
            unit = torch.exp2((e - 2).clamp(-127, 127))
        else:
            codes = torch.arange(127, dtype=torch.uint8, device="cuda")
            steps = codes.view(torch.float8_e4m3fn).to(f64)
            t = most / (6 * g)
            above = torch.searchsorted(steps, t).clamp(1, 126)
            lo, hi = steps[above - 1], steps[above]
            up = (t - lo > hi - t) | ((t - lo == hi - t) & (above % 2 == 0))
            unit = torch.where(up, hi, lo) * g
        a = v.abs()
        i = torch.zeros(a.shape, dtype=torch.int64, device="cuda")
        for j in range(7):      # a tie goes to the even code
            border = middle[j] * unit
            i += ((a > border) | ((a == border) & (j % 2 == 1) & (unit > 0))).long()
        i = torch.where(unit > 0, i, 0)
        return (torch.where(v < 0, -grid[i], grid[i]) * unit).flatten(-2)

    if op == "quantize":
        out = torch.empty(s["x"].shape, dtype=f64, device="cuda")
        for e in range(case["experts"]):
            g = 1.0 if s["tensor_scale"] is None else s["tensor_scale"][e].to(f64)
            out[e] = fp4(s["x"][e], case["format"], g)
        return {"values": out}

    def weights(w, e, fmt):
        if isinstance(w, torch.Tensor):
            return w[e].to(f64)
        codes, scales, ts = w
        c = torch.empty((codes.shape[1], 2 * codes.shape[2]), dtype=torch.int64, device="cuda")
        c[:, 0::2] = codes[e] % 16
        c[:, 1::2] = codes[e] // 16
        v = torch.where(c >= 8, -grid[c % 8], grid[c % 8])
        b = torch.exp2(scales[e].to(f64) - 127.0) if fmt == "mx" \
            else scales[e].view(torch.float8_e4m3fn).to(f64) * ts[e].to(f64)
        return v.mul_(b.repeat_interleave(_BLOCK[fmt], dim=1))

    n, F, K = s["n"], case["inter"], case["topk"]
    tokens = s["pairs"] // K
    if op == "fp4_experts":
        x = fp4(s["x"], case["format"], 1.0)
        fmt = case["format"]
        y = torch.zeros((n, case["hidden"] if case["block"] else F), dtype=f64, device="cuda")
        for e, lo, hi in s["spans"]:
            if case["block"]:
                r = torch.mm(x[tokens[lo:hi]], weights(s["w_gate_up"], e, fmt).t())
                h = fp4(gate(r[:, :F]) * r[:, F:], fmt, 1.0)
                y[lo:hi] = torch.mm(h, weights(s["w_down"], e, fmt).t())
            else:
                y[lo:hi] = torch.mm(x[tokens[lo:hi]], weights(s["w"], e, fmt).t())
        return {"y": y}
    out = torch.zeros(s["x"].shape, dtype=f64, device="cuda")
    x, scores = s["x"].to(f64), s["scores"].flatten().to(f64)
    for e, lo, hi in s["spans"]:
        r = torch.mm(x[tokens[lo:hi]], weights(s["w_gate_up"], e, case["weights"]).t())
        h = gate(r[:, :F]) * r[:, F:]
        y = torch.mm(h, weights(s["w_down"], e, case["weights"]).t())
        out.index_add_(0, tokens[lo:hi], y * scores[s["pairs"][lo:hi], None])
    return {"out": out}
