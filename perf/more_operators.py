"""Timed cases of the experts' products: the 8-bit integer product with a scale for each row and
each channel and the quantiser of its rows, and the experts' gated feed-forward block in bf16 with
its gradients.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, through this package's entry points.
"""
import math

import torch

own = False

I8_MAX = 127.0


# ------------------------------------------------------------------ cases

def _route(tokens, experts, topk, align, empty, skew):
    return {"tokens": tokens, "experts": experts, "topk": topk, "align": align, "empty": empty,
            "skew": skew}


def _quant(name, rows, channels, route):
    return {"name": name, "op": "quant", "rows": rows, "channels": channels, **route}


def _i8(name, rows, k, n, gated, weights, route):
    return {"name": name, "op": "i8", "rows": rows, "k": k, "n": n, "gated": gated,
            "weights": weights, **route}


def _ffn(name, rows, hidden, inter, save, weights, route):
    return {"name": name, "op": "ffn", "rows": rows, "hidden": hidden, "inter": inter,
            "save": save, "weights": weights, **route}


def _ffn_grad(name, rows, hidden, inter, weights, again, route):
    return {"name": name, "op": "ffn_grad", "rows": rows, "hidden": hidden, "inter": inter,
            "weights": weights, "again": again, **route}


def listed():
    return [
        # one decoded token in front of the experts: the call's own latency
        _quant("quantise, one token", "tokens", 7168, _route(1, 64, 8, 1, 0.0, 0.0)),
        # a prompt batch's activations in front of the second product
        _quant("quantise, expert rows", "expanded", 2048, _route(4096, 64, 8, 128, 0.0, 0.0)),
        # a small model's product on ragged segments, a tenth of the slots empty
        _i8("int8, ragged", "expanded", 624, 520, False, False, _route(100, 16, 4, 8, 0.1, 0.0)),
        # one decoded token: gate and up of its eight experts, read from the token's own row
        _i8("int8, one token", "tokens", 7168, 4096, True, False, _route(1, 64, 8, 1, 0.0, 0.0)),
        # the way back down of a decode batch, some experts popular and some idle
        _i8("int8, decode, skewed", "expanded", 2048, 7168, False, False,
            _route(128, 64, 8, 64, 0.0, 1.2)),
        # gate and up of a prompt batch, 512 rows an expert on average
        _i8("int8, prompt", "expanded", 7168, 4096, True, True, _route(4096, 64, 8, 128, 0.0, 0.0)),
        # one decoded token through its experts, bf16 weights
        _ffn("block, one token", "tokens", 7168, 2048, False, True, _route(1, 64, 8, 1, 0.0, 0.0)),
        # a small ragged batch with empty slots
        _ffn("block, ragged", "expanded", 648, 360, True, True, _route(100, 16, 4, 8, 0.2, 0.0)),
        # a decode batch, 16 rows an expert on average
        _ffn("block, decode", "tokens", 7168, 2048, False, True, _route(128, 64, 8, 1, 0.0, 0.0)),
        # a training batch, gate and up kept for the gradient
        _ffn("block, training", "expanded", 7168, 2048, True, False,
             _route(4096, 64, 8, 128, 0.0, 0.0)),
        # gradients of a small ragged batch
        _ffn_grad("block gradient, ragged", "expanded", 648, 360, True, True,
                  _route(100, 16, 4, 8, 0.2, 0.0)),
        # gradients of a training batch
        _ffn_grad("block gradient, training", "expanded", 7168, 2048, True, False,
                  _route(4096, 64, 8, 128, 0.0, 0.0)),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quant", "i8", "ffn", "ffn_grad"])
    tokens, experts = _log(rng, 1, 4096), rng.choice([8, 16, 24, 32, 64])
    topk = rng.randint(1, 8)
    empty = rng.choice([0.0, 0.1, 0.2]) if tokens * topk >= 8 else 0.0
    route = _route(tokens, experts, topk, rng.choice([1, 8, 64, 128]), empty,
                   rng.choice([0.0, 0.0, 0.8, 1.2]))
    rows, weights = rng.choice(["tokens", "expanded"]), rng.random() < 0.5
    if op == "quant":
        c = _quant("", rows, 16 * _log(rng, 16, 448), route)
    elif op == "i8":
        gated = rng.random() < 0.5
        c = _i8("", rows, 16 * _log(rng, 16, 448), 16 * _log(rng, 16, 256), gated,
                gated and weights, route)
    elif op == "ffn":
        c = _ffn("", rows, 8 * _log(rng, 32, 896), 8 * _log(rng, 16, 256), rng.random() < 0.5,
                 weights, route)
    else:
        c = _ffn_grad("", rows, 8 * _log(rng, 32, 896), 8 * _log(rng, 16, 256), weights,
                      rng.random() < 0.5, route)
    del c["name"]
    return c


def work(case):
    T, E = case["tokens"], case["experts"]
    slots = T * case["topk"] * (1.0 - case["empty"])
    # experts that a token of the batch meets, for uniform routing
    met = E * (1.0 - (1.0 - slots / T / E) ** T)
    rows = T if case["rows"] == "tokens" else slots
    if case["op"] == "quant":
        C = case["channels"]
        return {"bytes": rows * (3 * C + 4), "flops": rows * C * 3}
    if case["op"] == "i8":
        k, n = case["k"], case["n"]
        return {"bytes": met * n * (k + 4) + rows * (k + 4) + slots * n * (1 if case["gated"] else 2),
                "flops": 2 * slots * k * n}
    H, I = case["hidden"], case["inter"]  # noqa: E741
    extra = 4 * slots if case["weights"] else 0
    if case["op"] == "ffn":
        out = 2 * I + 2 * H + (4 * I if case["save"] else 0)
        return {"bytes": met * 6 * H * I + rows * 2 * H + slots * out + extra,
                "flops": 6 * slots * H * I}
    # in: gradient of y, gate and up, h (or written again); out: gradients of gate and up and of x
    row = 2 * H + 4 * I + 2 * I + 4 * I + 2 * H
    return {"bytes": (met + E) * 6 * H * I + rows * 2 * H + slots * row + 2 * extra,
            "flops": 12 * slots * H * I}


# ------------------------------------------------------------------ inputs

def _ids(case, gen, dev):
    """Distinct experts for each token, uniform or by a popularity that falls as a power of the
    rank, some slots empty."""
    T, E, K = case["tokens"], case["experts"], case["topk"]
    u = torch.rand((T, E), generator=gen, device=dev, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    rank = torch.randperm(E, generator=gen, device=dev) + 1
    score = -torch.log(-torch.log(u)) - case["skew"] * torch.log(rank.double())
    ids = score.topk(K, dim=1).indices
    gone = torch.rand((T, K), generator=gen, device=dev) < case["empty"]
    return ids.masked_fill(gone, -1).contiguous()


def _routing(case, gen, dev):
    """The ids, and where each slot's row lies in the expanded layout: experts in order, each
    segment starting at a multiple of the alignment, slots in order inside it.  ``table`` has the
    rows of each expert that got some, the shorter lists filled up with their first row."""
    T, E, K, A = case["tokens"], case["experts"], case["topk"], case["align"]
    ids = _ids(case, gen, dev)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    room = (counts + A - 1) // A * A
    start = room.cumsum(0) - room
    slot = torch.argsort(key, stable=True)[:int(counts.sum())]
    expert = key[slot]
    rank = torch.arange(slot.numel(), device=dev) - (counts.cumsum(0) - counts)[expert]
    capacity = (T * min(K, E) + (A - 1) * E + A - 1) // A * A
    row = start[expert] + rank
    active = torch.nonzero(counts).reshape(-1)
    place = torch.arange(max(1, int(counts.max())), device=dev)
    filled = place < counts[active][:, None]
    table = start[active][:, None] + torch.where(filled, place, 0)
    source = torch.zeros(capacity, dtype=torch.long, device=dev)
    source[row] = slot // K
    gather = source[table] if case["rows"] == "tokens" else table
    return {"ids": ids, "slot": slot, "expert": expert, "row": row, "capacity": capacity,
            "active": active, "filled": filled, "table": table, "gather": gather}


def _handle(case, r):
    import combine_ep_layout_08_amd as ep
    h = ep.Handle(case["tokens"], case["topk"], case["experts"], case["align"])
    h.layout(r["ids"])
    return h


def _normal(shape, gen, dev, scale=1.0):
    return (torch.randn(shape, generator=gen, device=dev) * scale).bfloat16()


def _stream(shape, gen, dev):
    """Rows of a residual stream: a few channels much larger than the others."""
    x = torch.randn(shape, generator=gen, device=dev)
    big = torch.rand(shape[-1], generator=gen, device=dev) < 0.005
    return (x * torch.where(big, 20.0, 1.0)).bfloat16()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    r = _routing(case, gen, dev)
    cap, E = r["capacity"], case["experts"]
    rows = case["tokens"] if case["rows"] == "tokens" else cap
    tokens = case["rows"] == "tokens"
    s = {"case": case, "op": op, "routing": r}
    h = _handle(case, r) if own else None
    if op == "quant":
        C = case["channels"]
        s["x"] = _stream((rows, C), gen, dev) if tokens else _normal((rows, C), gen, dev)
        s["q"] = torch.zeros((rows, C), dtype=torch.int8, device=dev)
        s["scale"] = torch.zeros(rows, device=dev)
        if own:
            import combine_ep_layout_08_amd as ep
            s["call"] = ep.bind_quantize_i8(s["x"], out_q=s["q"], out_scale=s["scale"],
                                            handle=None if tokens else h)
        return s
    if op == "i8":
        k, n = case["k"], case["n"]
        s["x"], s["scale"] = _codes(torch.randn((rows, k), generator=gen, device=dev))
        w = torch.randn((E * n, k), generator=gen, device=dev)
        s["w"], s["w_scale"] = _codes(w.mul_(k ** -0.5))
        s["w"], s["w_scale"] = s["w"].reshape(E, n, k), s["w_scale"].reshape(E, n)
        s["weights"] = torch.rand(cap, generator=gen, device=dev) if case["weights"] else None
        s["out"] = torch.zeros((cap, n // 2 if case["gated"] else n), dtype=torch.bfloat16,
                               device=dev)
        if own:
            import combine_ep_layout_08_amd as ep
            s["call"] = ep.bind_expert_i8(h, s["x"], s["scale"], s["w"], s["w_scale"],
                                          gated=case["gated"], row_weights=s["weights"],
                                          token_rows=tokens, out=s["out"])
        return s
    H, I = case["hidden"], case["inter"]  # noqa: E741
    s["x"] = _normal((rows, H), gen, dev)
    s["w13"] = _normal((E, 2 * I, H), gen, dev, 1.5 * H ** -0.5)
    s["w2"] = _normal((E, H, I), gen, dev, I ** -0.5)
    s["weights"] = torch.rand(cap, generator=gen, device=dev) if case["weights"] else None
    like = dict(dtype=torch.bfloat16, device=dev)
    if op == "ffn":
        s["h"], s["y"] = torch.zeros((cap, I), **like), torch.zeros((cap, H), **like)
        s["saved"] = torch.zeros((cap, 2 * I), **like) if case["save"] else None
        if own:
            import combine_ep_layout_08_amd as ep
            s["call"] = ep.bind_expert_ffn(h, s["x"], s["w13"], s["w2"], row_weights=s["weights"],
                                           token_rows=tokens, out_h=s["h"], saved=s["saved"],
                                           out=s["y"])
        return s
    s["handle"] = h
    s["grad"] = _normal((cap, H), gen, dev, 1e-2)
    s["saved"] = _normal((cap, 2 * I), gen, dev, 1.5)
    if case["again"]:
        s["h"] = torch.zeros((cap, I), **like)
    else:
        gate, up = s["saved"].float().chunk(2, 1)
        act = gate / (1.0 + torch.exp(-gate)) * up
        s["h"] = (act if s["weights"] is None else act * s["weights"][:, None]).bfloat16()
    s["grad_gate_up"], s["grad_x"] = torch.zeros((cap, 2 * I), **like), torch.zeros((cap, H), **like)
    s["grad_w13"], s["grad_w2"] = torch.empty_like(s["w13"]), torch.empty_like(s["w2"])
    s["grad_weights"] = torch.zeros(cap, device=dev) if case["weights"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _codes(v):
    """8-bit codes of fp32 rows and the rows' scales."""
    s = v.abs().amax(1).clamp_min(1e-12)
    s = s / torch.full_like(s, I8_MAX)        # by a number, torch multiplies with its reciprocal
    return torch.round(v / s[:, None]).to(torch.int8), s


def _gated(gate, up, s):
    r = s["routing"]
    h = gate / (1.0 + torch.exp(-gate)) * up
    return h if s["weights"] is None else h * s["weights"][r["table"]][..., None]


def _product(x, w):
    """x . w^T for each expert."""
    return torch.matmul(w, x.transpose(1, 2).contiguous()).transpose(1, 2)


def _put(s, out, values):
    r = s["routing"]
    out[r["table"][r["filled"]]] = values[r["filled"]].to(out.dtype)


def _plain_quant(s):
    if s["case"]["rows"] == "tokens":
        s["q"], s["scale"] = _codes(s["x"].float())
    else:
        rows = s["routing"]["row"]
        s["q"][rows], s["scale"][rows] = _codes(s["x"][rows].float())


def _plain_i8(s):
    r = s["routing"]
    v = _product(s["x"][r["gather"]].float(), s["w"][r["active"]].float())
    v = v * s["scale"][r["gather"]][..., None] * s["w_scale"][r["active"]][:, None]
    if s["case"]["gated"]:
        v = _gated(*v.chunk(2, 2), s)
    _put(s, s["out"], v)


def _plain_ffn(s):
    r = s["routing"]
    gate_up = _product(s["x"][r["gather"]].float(), s["w13"][r["active"]].float())
    if s["saved"] is not None:
        _put(s, s["saved"], gate_up)
    h = _gated(*gate_up.chunk(2, 2), s).bfloat16()      # the rows that the second product reads
    _put(s, s["h"], h)
    _put(s, s["y"], _product(h.float(), s["w2"][r["active"]].float()))


def _plain_ffn_grad(s):
    r = s["routing"]
    seen, table, keep = r["active"], r["table"], r["filled"][..., None]
    gy = s["grad"][table].float() * keep
    gate, up = s["saved"][table].float().chunk(2, 2)
    gh = torch.matmul(gy, s["w2"][seen].float())
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    if s["weights"] is not None:
        _put(s, s["grad_weights"], (gh * silu * up).sum(2))
        gh = gh * s["weights"][table][..., None]
    slope = sig * (1.0 + gate * (1.0 - sig))
    ggu = torch.cat((gh * up * slope, gh * silu), 2).bfloat16()     # read by two products
    _put(s, s["grad_gate_up"], ggu)
    ggu = ggu.float()
    _put(s, s["grad_x"], torch.matmul(ggu, s["w13"][seen].float()))
    if s["case"]["again"]:
        _put(s, s["h"], _gated(gate, up, s))
    s["grad_w13"].zero_()
    s["grad_w2"].zero_()
    x, h = s["x"][r["gather"]].float(), s["h"][table].float()
    s["grad_w13"][seen] = torch.matmul(ggu.transpose(1, 2).contiguous(), x).bfloat16()
    s["grad_w2"][seen] = torch.matmul(gy.transpose(1, 2).contiguous(), h).bfloat16()


def run(state):
    s, op = state, state["op"]
    if op == "quant":
        s["call"]() if own else _plain_quant(s)
        return {"q": s["q"], "scale": s["scale"]}
    if op == "i8":
        s["call"]() if own else _plain_i8(s)
        return {"y": s["out"]}
    if op == "ffn":
        s["call"]() if own else _plain_ffn(s)
        return {"h": s["h"], "saved": s["saved"], "y": s["y"]}
    if own:
        s["handle"].expert_ffn_backward(
            s["grad"], s["x"], s["w13"], s["w2"], s["saved"], s["h"],
            row_weights=s["weights"], token_rows=s["case"]["rows"] == "tokens",
            remake_h=s["case"]["again"], grad_gate_up=s["grad_gate_up"], grad_x=s["grad_x"],
            grad_w13=s["grad_w13"], grad_w2=s["grad_w2"], grad_row_weights=s["grad_weights"])
    else:
        _plain_ffn_grad(s)
    return {"x": s["grad_x"], "w13": s["grad_w13"], "w2": s["grad_w2"], "gate_up": s["grad_gate_up"],
            "weights": s["grad_weights"], "h": s["h"] if s["case"]["again"] else None}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    global own
    mode, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mode
    op, r, dev = s["op"], s["routing"], s["x"].device
    cap = r["capacity"]
    wide = torch.float64
    tokens = case["rows"] == "tokens"

    def new(*shape):
        return torch.zeros(shape, dtype=wide, device=dev)

    if op == "quant":
        at = torch.arange(case["tokens"], device=dev) if tokens else r["row"]
        x = s["x"][at].to(wide)
        scale = torch.maximum(x.abs().max(1).values, torch.full_like(x[:, 0], 1e-12)) / I8_MAX
        out = new(s["x"].shape[0])
        out[at] = scale
        return {"q": None, "scale": out}          # whole numbers

    def silu(v):
        return v * torch.sigmoid(v)

    def factor(rows):
        return 1.0 if s["weights"] is None else s["weights"][rows].to(wide).unsqueeze(1)

    def segments():
        for e in torch.unique(r["expert"]).tolist():
            mine = r["expert"] == e
            rows = r["row"][mine]
            yield e, rows, r["slot"][mine] // case["topk"] if tokens else rows

    if op == "i8":
        y = new(*s["out"].shape)
        for e, rows, src in segments():
            v = torch.einsum("rk,r->rk", s["x"][src].to(wide), s["scale"][src].to(wide)) @ \
                (s["w"][e].to(wide) * s["w_scale"][e].to(wide).unsqueeze(1)).t()
            if case["gated"]:
                half = case["n"] // 2
                v = silu(v[:, :half]) * v[:, half:] * factor(rows)
            y[rows] = v
        return {"y": y}
    H, I = case["hidden"], case["inter"]  # noqa: E741
    if op == "ffn":
        h, y, saved = new(cap, I), new(cap, H), new(cap, 2 * I)
        for e, rows, src in segments():
            saved[rows] = s["x"][src].to(wide) @ s["w13"][e].to(wide).t()
            h[rows] = silu(saved[rows, :I]) * saved[rows, I:] * factor(rows)
            # the second product is of the rounded rows
            y[rows] = h[rows].to(torch.bfloat16).to(wide) @ s["w2"][e].to(wide).t()
        return {"h": h, "saved": saved if case["save"] else None, "y": y}
    E = case["experts"]
    gx, gu, gr, h = new(cap, H), new(cap, 2 * I), new(cap), new(cap, I)
    g13 = torch.zeros((E, 2 * I, H), dtype=wide, device=dev)
    g2 = torch.zeros((E, H, I), dtype=wide, device=dev)
    for e, rows, src in segments():
        a, b = s["saved"][rows].to(wide).split(I, 1)
        p = torch.sigmoid(a)
        gy = s["grad"][rows].to(wide)
        gh = gy @ s["w2"][e].to(wide)
        gr[rows] = (gh * a * p * b).sum(1)
        gh = gh * factor(rows)
        gu[rows] = torch.cat((gh * b * (p + a * p * (1.0 - p)), gh * a * p), 1)
        low = gu[rows].to(torch.bfloat16).to(wide)         # what the products read
        gx[rows] = low @ s["w13"][e].to(wide)
        g13[e] = low.t() @ s["x"][src].to(wide)
        h[rows] = a * p * b * factor(rows)
        kept = h[rows].to(torch.bfloat16) if case["again"] else s["h"][rows]
        g2[e] = gy.t() @ kept.to(wide)
    return {"x": gx, "w13": g13, "w2": g2, "gate_up": gu,
            "weights": gr if case["weights"] else None, "h": h if case["again"] else None}
