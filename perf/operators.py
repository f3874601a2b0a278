"""The experts' operators between dispatch and combine: their cases, inputs and plain forms.

  ffn            the experts' gated feed-forward block over the receive rows,
                 y = (act(x Wg^T) * (x Wu^T)) Wd^T for each expert's own rows
  ffn_backward   its gradients: of the rows, of the gate/up weights and of the down weights
  w4_gemv        the product of each expert's few rows with 4-bit weights and group scales
  w4_ffn         the gated feed-forward block on 4-bit weights (single tokens, small batches)

A case names one operator and its sizes. ``own`` false: the plain forms, elementary torch
operations in 32 bits rounded once at the end. ``own`` true: the package's entry points.
"""
import math

import torch

own = False

_BF16 = torch.bfloat16


def listed():
    return [
        # A micro-batch of a small model's training step, routed with one pair in ten dropped
        # by a capacity limit: odd row counts, latency counts as much as rate.
        {"name": "ffn small", "op": "ffn", "tokens": 331, "hidden": 1024, "inter": 512,
         "experts": 16, "topk": 4, "routing": "uniform", "drop": 0.1, "act": "gelu", "train": True},
        # Prefill of a short prompt, 8 experts, weights read once for a few rows each.
        {"name": "ffn prefill 128", "op": "ffn", "tokens": 128, "hidden": 4096, "inter": 2048,
         "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "act": "silu", "train": False},
        # The mixtral workload's rows through the block, saving what the backward pass needs.
        {"name": "ffn mixtral", "op": "ffn", "tokens": 4096, "hidden": 4096, "inter": 2048,
         "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "act": "silu", "train": True},
        # The deepseek workload's rows (Zipf-skewed over 256 experts), inference.
        {"name": "ffn deepseek", "op": "ffn", "tokens": 8192, "hidden": 7168, "inter": 2048,
         "experts": 256, "topk": 8, "routing": "zipf", "drop": 0.0, "act": "silu", "train": False},
        # The backward pass of the first case.
        {"name": "backward small", "op": "ffn_backward", "tokens": 331, "hidden": 1024,
         "inter": 512, "experts": 16, "topk": 4, "routing": "uniform", "drop": 0.1, "act": "gelu"},
        # The backward pass of the mixtral workload's block.
        {"name": "backward mixtral", "op": "ffn_backward", "tokens": 4096, "hidden": 4096,
         "inter": 2048, "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "act": "silu"},
        # Fine-grained experts under skew: the deepseek workload's rows on 64 experts, many of
        # them with fewer rows than a tile.
        {"name": "backward skewed", "op": "ffn_backward", "tokens": 8192, "hidden": 7168,
         "inter": 2048, "experts": 64, "topk": 8, "routing": "zipf", "drop": 0.0, "act": "silu"},
        # One projection of one dense layer for one token.
        {"name": "w4 one row", "op": "w4_gemv", "tokens": 1, "hidden": 4096, "inter": 4096,
         "experts": 1, "topk": 1, "routing": "uniform", "drop": 0.0, "group": 128, "zeros": False,
         "scale": "bf16"},
        # One projection of 8 experts for a batch of 13 decoded tokens, fine groups, zero points.
        {"name": "w4 batch 13", "op": "w4_gemv", "tokens": 13, "hidden": 4096, "inter": 2048,
         "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "group": 32, "zeros": True,
         "scale": "f32"},
        # One decoded token through 8 of 256 experts.
        {"name": "w4 ffn decode 1", "op": "w4_ffn", "tokens": 1, "hidden": 7168, "inter": 2048,
         "experts": 256, "topk": 8, "routing": "uniform", "drop": 0.0, "group": 128,
         "zeros": False, "scale": "bf16", "act": "silu"},
        # A decode batch of 64 tokens over the 8 experts of the mixtral workload: 16 rows each.
        {"name": "w4 ffn decode 64", "op": "w4_ffn", "tokens": 64, "hidden": 4096, "inter": 2048,
         "experts": 8, "topk": 2, "routing": "uniform", "drop": 0.0, "group": 64, "zeros": True,
         "scale": "bf16", "act": "silu"},
        # A decode batch of 32 tokens over 256 experts: one row for most of them.
        {"name": "w4 ffn decode 32", "op": "w4_ffn", "tokens": 32, "hidden": 7168, "inter": 2048,
         "experts": 256, "topk": 8, "routing": "uniform", "drop": 0.0, "group": 128,
         "zeros": False, "scale": "bf16", "act": "silu"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    largest = {c["op"]: max(work(d)["flops"] for d in listed() if d["op"] == c["op"])
               for c in listed()}
    op = rng.choice(["ffn", "ffn_backward", "w4_gemv", "w4_ffn"])
    while True:
        case = {"op": op}
        if op in ("ffn", "ffn_backward"):
            case["tokens"] = _log_between(rng, 1, 8192)
            case["hidden"] = 128 * _log_between(rng, 2, 56)
            case["inter"] = 128 * _log_between(rng, 1, 16)
            case["experts"] = rng.choice([1, 2, 5, 8, 16, 33, 64])
            case["topk"] = min(case["experts"], rng.choice([1, 2, 4, 8]))
            case["routing"] = rng.choice(["uniform", "zipf"])
            case["drop"] = rng.choice([0.0, 0.1])
            case["act"] = rng.choice(["silu", "gelu"])
            if op == "ffn":
                case["train"] = rng.choice([True, False])
        else:
            case["tokens"] = _log_between(rng, 1, 64)
            case["group"] = rng.choice([32, 64, 128])
            case["hidden"] = case["group"] * _log_between(rng, 512 // case["group"],
                                                          7168 // case["group"])
            case["inter"] = 128 * _log_between(rng, 2, 32 if op == "w4_gemv" else 16)
            case["experts"] = rng.choice([1, 3, 8, 32, 64, 256])
            case["topk"] = min(case["experts"], rng.choice([1, 2, 4, 8]))
            case["routing"] = "uniform"
            case["drop"] = 0.0
            case["zeros"] = rng.choice([True, False])
            case["scale"] = rng.choice(["bf16", "f32"])
            if op == "w4_ffn":
                case["act"] = rng.choice(["silu", "gelu"])
        if 3072 not in (case["hidden"], case["inter"], 2 * case["inter"]) \
                and work(case)["flops"] <= largest[op]:
            return case


def _popularity(case):
    if case["routing"] == "uniform":
        return [1.0 / case["experts"]] * case["experts"]
    w = [(e + 1) ** -1.1 for e in range(case["experts"])]
    s = sum(w)
    return [v / s for v in w]


def work(case):
    T, D, F, E, K = (case[k] for k in ("tokens", "hidden", "inter", "experts", "topk"))
    rows = T * K * (1.0 - case["drop"])
    # Experts that the call's tokens reach (expected over the routing).
    used = sum(1.0 - (1.0 - min(1.0, K * p * (1.0 - case["drop"]))) ** T for p in _popularity(case))
    if case["op"] == "ffn":
        saved = rows * 3 * F * 2 if case["train"] else 0.0
        return {"bytes": used * 3 * D * F * 2 + rows * 2 * D * 2 + saved,
                "flops": rows * 6 * D * F}
    if case["op"] == "ffn_backward":
        return {"bytes": used * 3 * D * F * 2 + E * 3 * D * F * 2 + rows * (3 * D + 3 * F) * 2,
                "flops": rows * 12 * D * F}
    per = 0.5 + ((2 if case["scale"] == "bf16" else 4) + (1 if case["zeros"] else 0)) / case["group"]
    if case["op"] == "w4_gemv":
        return {"bytes": used * D * F * per + rows * (D + F) * 2, "flops": rows * 2 * D * F}
    return {"bytes": used * 3 * D * F * per + rows * 2 * D * 2, "flops": rows * 6 * D * F}


def _normal(gen, shape, std):
    t = torch.empty(shape, dtype=_BF16, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def _w4(gen, experts, dout, din, case):
    """Random 4-bit weights: codes, group scales (about unit-variance products) and zero points."""
    q = torch.randint(0, 256, (experts, dout, din // 2), dtype=torch.uint8, device="cuda",
                      generator=gen)
    shape = (experts, dout, din // case["group"])
    s = torch.rand(shape, device="cuda", generator=gen).add_(0.5).mul_(1.0 / (4.6 * math.sqrt(din)))
    s = s.to(_BF16) if case["scale"] == "bf16" else s
    z = None
    if case["zeros"]:
        z = torch.randint(0, 16, shape, dtype=torch.uint8, device="cuda", generator=gen)
    return q, s, z


def prepare(case, seed):
    T, D, F, E, K = (case[k] for k in ("tokens", "hidden", "inter", "experts", "topk"))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    # Routing: K distinct experts for each token by popularity; some pairs dropped.
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen)))
    noise += torch.tensor(_popularity(case), device="cuda").log()
    ids = noise.topk(K, dim=1).indices.to(torch.int32)
    dropped = torch.randperm(T * K, device="cuda", generator=gen)[:round(case["drop"] * T * K)]
    ids.view(-1)[dropped] = -1
    # Receive rows, expert by expert in the order of the pairs, in a buffer for every pair;
    # what is past the rows in use is whatever was there before.
    flat = ids.flatten()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    counts = torch.bincount(flat[flat >= 0], minlength=E).tolist()
    n, spans = 0, []
    for e, c in enumerate(counts):
        if c:
            spans.append((e, n, n + c))
        n += c
    capacity = (T + 3) // 4 * 4 * K

    def rows(width, std):
        t = torch.full((capacity, width), float("nan"), dtype=_BF16, device="cuda")
        t[:n] = _normal(gen, (n, width), std)
        return t

    x = torch.full((capacity, D), float("nan"), dtype=_BF16, device="cuda")
    x[:n] = _normal(gen, (T, D), 1.0)[(order[:n] // K).long()]
    # Experts with rows, their first rows and row counts: on the host and on the GPU.
    state = {"case": case, "x": x, "n": n, "spans": spans,
             "spans_gpu": torch.tensor(spans, device="cuda", dtype=torch.int64).view(-1, 3)}
    if case["op"] in ("ffn", "ffn_backward"):
        state["w_gate_up"] = _normal(gen, (E, 2 * F, D), D ** -0.5)
        state["w_down"] = _normal(gen, (E, D, F), F ** -0.5)
    if case["op"] == "ffn_backward":
        # Pre-activations as the forward pass leaves them: unit variance.
        gate_up = rows(2 * F, 1.0)
        g, u = gate_up[:, :F].float(), gate_up[:, F:].float()
        state["gate_up"] = gate_up
        state["h"] = (_act(g, case["act"])[0] * u).to(_BF16)
        state["grad_y"] = rows(D, 0.02)
    if case["op"] == "w4_gemv":
        state["w"] = _w4(gen, E, F, D, case)
    if case["op"] == "w4_ffn":
        state["w_gate_up"] = _w4(gen, E, 2 * F, D, case)
        state["w_down"] = _w4(gen, E, D, F, case)
    if own:
        import combine_topk_ids_expert_gb300 as ep

        buf = ep.Buffer(num_max_tokens_per_rank=T, hidden=D, num_experts=E, num_ranks=1, topk=K,
                        dtype=_BF16, layout="packed")
        buf.dispatch_layout(ids, T)
        state["buf"], state["ids"] = buf, ids
        for k in ("w", "w_gate_up", "w_down"):
            if isinstance(state.get(k), tuple):
                state[k] = ep.W4(*state[k])
    return state


def _act(g, act):
    """The gate's activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g))


def _weights(w, used):
    """The used experts' weights in 32 bits."""
    if isinstance(w, torch.Tensor):
        return w[used].float()
    q, s = w[0][used], w[1][used].float()
    q = torch.stack((q & 15, q >> 4), dim=-1).view(*s.shape, -1)
    z = 8.0 if w[2] is None else w[2][used].float()[..., None]
    return ((q.float() - z) * s[..., None]).flatten(2)


def _batches(state):
    """(experts, their rows [experts, C], which of these are rows) for products of many experts
    at once; one expert at a time where their row counts differ too much for that."""
    spans, gpu = state["spans"], state["spans_gpu"]
    most = max((hi - lo for _, lo, hi in spans), default=0)
    if most * len(spans) <= 4 * state["n"] + 1024:
        parts = [(gpu, most)] if spans else []
    else:
        parts = [(gpu[i:i + 1], hi - lo) for i, (_, lo, hi) in enumerate(spans)]
    for part, c in parts:
        at = part[:, 1:2] + torch.arange(c, device="cuda")
        here = at < part[:, 2:3]
        yield part[:, 0], torch.where(here, at, 0), here


def _take(t, at, here):
    """Rows of t in 32 bits, zeros where a batch has none."""
    return torch.where(here[..., None], t[at].float(), 0.0)


def _put(out, at, here, rows):
    out[at[here]] = rows[here].to(out.dtype)


def _plain_ffn(s):
    case, x, n = s["case"], s["x"], s["n"]
    F, train = case["inter"], case.get("train", False)
    r = {"y": torch.empty((n, x.shape[1]), dtype=_BF16, device="cuda")}
    if train:
        r["h"] = torch.empty((n, F), dtype=_BF16, device="cuda")
        r["gate_up"] = torch.empty((n, 2 * F), dtype=_BF16, device="cuda")
    for used, at, here in _batches(s):
        gu = _take(x, at, here) @ _weights(s["w_gate_up"], used).mT
        h = _act(gu[..., :F], case["act"])[0] * gu[..., F:]
        _put(r["y"], at, here, h @ _weights(s["w_down"], used).mT)
        if train:
            _put(r["h"], at, here, h)
            _put(r["gate_up"], at, here, gu)
    return r


def _plain_backward(s):
    case, x, n = s["case"], s["x"], s["n"]
    F = case["inter"]
    grad_x = torch.empty((n, x.shape[1]), dtype=_BF16, device="cuda")
    grad_w_gate_up = torch.zeros_like(s["w_gate_up"])
    grad_w_down = torch.zeros_like(s["w_down"])
    for used, at, here in _batches(s):
        gy, xe = _take(s["grad_y"], at, here), _take(x, at, here)
        gu = _take(s["gate_up"], at, here)
        a, da = _act(gu[..., :F], case["act"])
        gh = gy @ _weights(s["w_down"], used)
        ggu = torch.cat((gh * gu[..., F:] * da, gh * a), dim=-1)
        _put(grad_x, at, here, ggu @ _weights(s["w_gate_up"], used))
        grad_w_gate_up[used] = (ggu.mT @ xe).to(_BF16)
        grad_w_down[used] = (gy.mT @ _take(s["h"], at, here)).to(_BF16)
    return {"grad_x": grad_x, "grad_w_gate_up": grad_w_gate_up, "grad_w_down": grad_w_down}


def _plain_gemv(s):
    y = torch.empty((s["n"], s["case"]["inter"]), dtype=_BF16, device="cuda")
    for used, at, here in _batches(s):
        _put(y, at, here, _take(s["x"], at, here) @ _weights(s["w"], used).mT)
    return {"y": y}


def run(state):
    case, n = state["case"], state["n"]
    if not own:
        return {"ffn": _plain_ffn, "w4_ffn": _plain_ffn, "w4_gemv": _plain_gemv,
                "ffn_backward": _plain_backward}[case["op"]](state)
    buf, x = state["buf"], state["x"]
    if case["op"] == "ffn":
        got = buf.expert_ffn(x, state["w_gate_up"], state["w_down"], act=case["act"],
                             save=case["train"])
        if not case["train"]:
            return {"y": got[:n]}
        y, h, gate_up = got
        return {"y": y[:n], "h": h[:n], "gate_up": gate_up[:n]}
    if case["op"] == "ffn_backward":
        gx, gw_gu, gw_d = buf.expert_ffn_backward(state["grad_y"], x, state["w_gate_up"],
                                                  state["w_down"], state["gate_up"], state["h"],
                                                  act=case["act"])
        return {"grad_x": gx[:n], "grad_w_gate_up": gw_gu, "grad_w_down": gw_d}
    if case["op"] == "w4_gemv":
        return {"y": buf.expert_gemv_w4(x, state["w"])[:n]}
    return {"y": buf.expert_ffn_w4(x, state["w_gate_up"], state["w_down"], act=case["act"])[:n]}


def exact(case, seed):
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    F, n, spans = case["inter"], s["n"], s["spans"]
    f64 = torch.float64

    def weights(w, e):
        if isinstance(w, torch.Tensor):
            return w[e].to(f64)
        q, scale, zero = w
        codes = torch.empty((q.shape[1], 2 * q.shape[2]), dtype=f64, device="cuda")
        codes[:, 0::2] = torch.remainder(q[e].to(f64), 16.0)
        codes[:, 1::2] = torch.floor(q[e].to(f64) / 16.0)
        g = case["group"]
        codes -= 8.0 if zero is None else zero[e].to(f64).repeat_interleave(g, dim=1)
        return codes.mul_(scale[e].to(f64).repeat_interleave(g, dim=1))

    def gate(g):
        if case["act"] == "silu":
            return g * torch.special.expit(g)
        inner = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        return g * torch.special.expit(2.0 * inner)        # (1 + tanh v) / 2 = expit(2 v)

    def gate_slope(g):
        if case["act"] == "silu":
            p = torch.special.expit(g)
            return p + g * p * torch.special.expit(-g)
        v = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        dv = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g ** 2)
        p = torch.special.expit(v)
        return p + g * dv * p * torch.special.expit(-v)

    def out(*shape):
        return torch.zeros(shape, dtype=f64, device="cuda")

    if case["op"] == "w4_gemv":
        y = out(n, F)
        for e, lo, hi in spans:
            y[lo:hi] = torch.mm(s["x"][lo:hi].to(f64), weights(s["w"], e).t())
        return {"y": y}
    D = case["hidden"]
    if case["op"] in ("ffn", "w4_ffn"):
        train = case.get("train", False)
        r = {"y": out(n, D)}
        if train:
            r |= {"h": out(n, F), "gate_up": out(n, 2 * F)}
        for e, lo, hi in spans:
            gu = torch.mm(s["x"][lo:hi].to(f64), weights(s["w_gate_up"], e).t())
            g, u = gu.split(F, dim=1)
            h = gate(g) * u
            r["y"][lo:hi] = torch.mm(h, weights(s["w_down"], e).t())
            if train:
                r["h"][lo:hi], r["gate_up"][lo:hi] = h, gu
        return r
    r = {"grad_x": out(n, D), "grad_w_gate_up": out(*s["w_gate_up"].shape),
         "grad_w_down": out(*s["w_down"].shape)}
    for e, lo, hi in spans:
        gy = s["grad_y"][lo:hi].to(f64)
        g, u = s["gate_up"][lo:hi].to(f64).split(F, dim=1)
        gh = torch.mm(gy, s["w_down"][e].to(f64))
        gg, gu = gh * u * gate_slope(g), gh * gate(g)
        wg, wu = s["w_gate_up"][e].to(f64).split(F, dim=0)
        r["grad_x"][lo:hi] = torch.mm(gg, wg) + torch.mm(gu, wu)
        xe = s["x"][lo:hi].to(f64)
        r["grad_w_gate_up"][e, :F] = torch.mm(gg.t(), xe)
        r["grad_w_gate_up"][e, F:] = torch.mm(gu.t(), xe)
        r["grad_w_down"][e] = torch.mm(gy.t(), s["h"][lo:hi].to(f64))
    return r
