"""Timed cases of the expert layer's operators: the sum and root-mean-square norm in front of
dispatch (with its FP8 output) and its gradient, the experts' products with 4-bit weights, and
the gated activation between those products, with its 8-bit checkpoint and the gradient taken
from that checkpoint.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, through this package's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, tokens, hidden, residual, y, scales, weight):
    return {"name": name, "op": "norm", "tokens": tokens, "hidden": hidden, "residual": residual,
            "y": y, "scales": scales, "weight": weight}


def _norm_grad(name, tokens, hidden, residual, weight):
    return {"name": name, "op": "norm_grad", "tokens": tokens, "hidden": hidden,
            "residual": residual, "weight": weight}


def _w4(name, tokens, experts, topk, k, n, fmt, group, x, rows, align, empty, skew):
    return {"name": name, "op": "w4", "tokens": tokens, "experts": experts, "topk": topk, "k": k,
            "n": n, "format": fmt, "group": group, "x": x, "rows": rows, "align": align,
            "empty": empty, "skew": skew}


def _act(name, tokens, experts, topk, inter, align, empty, skew, out, checkpoint, weights):
    return {"name": name, "op": "act", "tokens": tokens, "experts": experts, "topk": topk,
            "inter": inter, "align": align, "empty": empty, "skew": skew, "out": out,
            "checkpoint": checkpoint, "weights": weights}


def _act_grad(name, tokens, experts, topk, inter, align, empty, skew, saved, weights, again):
    return {"name": name, "op": "act_grad", "tokens": tokens, "experts": experts, "topk": topk,
            "inter": inter, "align": align, "empty": empty, "skew": skew, "saved": saved,
            "weights": weights, "again": again}


def listed():
    return [
        # one decoded token between two layers: the call's own latency
        _norm("norm, one token", 1, 7168, True, True, "f32", "bf16"),
        # a prefill batch: bf16 rows for the router, FP8 rows with packed exponents for dispatch
        _norm("norm, prefill", 4096, 7168, True, True, "ue8m0", "bf16"),
        # gradients of a ragged small batch, a hidden size that fills no power of two
        _norm_grad("norm gradient, ragged", 333, 1280, False, "f32"),
        # gradients of a training batch, with the gradient that comes along the residual
        _norm_grad("norm gradient, training", 4096, 7168, True, "bf16"),
        # a small model's first product, a tenth of the slots empty
        _w4("product, tiny", 64, 16, 4, 256, 512, "int4", 32, "bf16", "expanded", 1, 0.1, 0.0),
        # one decoded token: gate and up of its eight experts, read from the token's own row
        _w4("product, one token", 1, 64, 8, 7168, 4096, "int4", 128, "bf16", "tokens", 1, 0.0, 0.0),
        # a decode batch after FP8 dispatch, 16 rows an expert on average
        _w4("product, decode", 128, 64, 8, 7168, 4096, "mxfp4", 32, "f32", "expanded", 128, 0.0,
            0.0),
        # the way back down of a decode batch, some experts popular and some idle
        _w4("product, down, skewed", 96, 64, 8, 2048, 7168, "int4", 64, "bf16", "expanded", 64,
            0.0, 1.2),
        # a decode batch's activation, weighted by the router
        _act("activation, decode", 32, 256, 8, 2048, 128, 0.0, 0.0, "bf16", "none", True),
        # a training batch's activation: FP8 rows for the next product, 8-bit checkpoint
        _act("activation, training", 4096, 256, 8, 2048, 128, 0.0, 0.0, "f32", "f32", False),
        # gradients of a small ragged batch with empty slots, from a bf16 copy
        _act_grad("activation gradient, ragged", 100, 16, 4, 640, 8, 0.2, 0.0, "bf16", True, False),
        # gradients of a training batch from the 8-bit checkpoint, the rows made again for the
        # weights' gradient
        _act_grad("activation gradient, training", 4096, 256, 8, 2048, 128, 0.0, 0.0, "f32", True,
                  True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "w4", "act", "act_grad"])
    if op == "norm":
        scales = rng.choice(["none", "f32", "ue8m0"])
        unit = 8 if scales == "none" else 128
        c = _norm("", _log(rng, 1, 4096), unit * _log(rng, 256 // unit, 7168 // unit),
                  rng.random() < 0.7, scales == "none" or rng.random() < 0.5, scales,
                  rng.choice(["bf16", "f32"]))
    elif op == "norm_grad":
        c = _norm_grad("", _log(rng, 1, 4096), 8 * _log(rng, 32, 896), rng.random() < 0.7,
                       rng.choice(["bf16", "f32"]))
    elif op == "w4":
        fmt, group = rng.choice([("int4", 32), ("int4", 64), ("int4", 128), ("mxfp4", 32)])
        experts = rng.choice([8, 16, 24, 32, 64])
        c = _w4("", _log(rng, 1, 128), experts, rng.randint(1, 8), 128 * _log(rng, 2, 56),
                8 * _log(rng, 32, 512), fmt, group, rng.choice(["bf16", "f32", "ue8m0"]),
                rng.choice(["tokens", "expanded"]), rng.choice([1, 8, 16, 128]),
                rng.choice([0.0, 0.1]), rng.choice([0.0, 0.8, 1.2]))
    else:
        args = ("", _log(rng, 1, 4096), rng.choice([8, 16, 64, 128, 256]), rng.randint(1, 8),
                128 * _log(rng, 2, 16), rng.choice([1, 8, 64, 128]), rng.choice([0.0, 0.1, 0.2]),
                rng.choice([0.0, 1.2]))
        kind = ["bf16", "f32", "ue8m0"]
        if op == "act":
            c = _act(*args, rng.choice(kind), rng.choice(["none", "f32", "ue8m0"]),
                     rng.random() < 0.5)
        else:
            c = _act_grad(*args, rng.choice(kind), rng.random() < 0.5, rng.random() < 0.5)
    if op in ("w4", "act", "act_grad") and c["tokens"] * c["topk"] < 8:
        c["empty"] = 0.0                      # a batch with nothing routed computes nothing
    del c["name"]
    return c


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H = case["tokens"], case["hidden"]
        weight = H * (2 if case["weight"] == "bf16" else 4)
        if op == "norm":
            row = 2 * H + (4 * H if case["residual"] else 0) + (2 * H if case["y"] else 0) + 4
            row += {"none": 0, "f32": H + H // 32, "ue8m0": H + H // 128}[case["scales"]]
            return {"bytes": T * row + weight, "flops": T * H * 8}
        row = 6 * H + (2 * H if case["residual"] else 0) + 4
        return {"bytes": T * row + weight + 4 * H, "flops": T * H * 12}
    slots = case["tokens"] * case["topk"] * (1.0 - case["empty"])
    if op == "w4":
        # experts that a token of the batch meets, for uniform routing
        met = case["experts"] * (1.0 - (1.0 - slots / case["tokens"] / case["experts"]) **
                                 case["tokens"])
        weights = met * case["n"] * case["k"] * (
            0.5 + (2.0 / case["group"] if case["format"] == "int4" else 1.0 / 32))
        rows = case["tokens"] if case["rows"] == "tokens" else slots
        x = rows * case["k"] * (2 if case["x"] == "bf16" else 1)
        return {"bytes": weights + x + slots * case["n"] * 2,
                "flops": 2 * slots * case["k"] * case["n"]}
    inter = case["inter"]
    eight = lambda kind, n: {"none": 0, "bf16": 2 * n, "f32": n + n / 32,  # noqa: E731
                             "ue8m0": n + n / 128}[kind]
    if op == "act":
        row = 4 * inter + eight(case["out"], inter) + eight(case["checkpoint"], 2 * inter)
        return {"bytes": slots * (row + (4 if case["weights"] else 0)), "flops": slots * inter * 8}
    row = 2 * inter + eight(case["saved"], 2 * inter) + 4 * inter
    row += (2 * inter if case["again"] else 0) + (8 if case["weights"] else 0)
    return {"bytes": slots * row, "flops": slots * inter * 20}


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
    segment starting at a multiple of the alignment, slots in order inside it."""
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
    return {"ids": ids, "counts": counts, "start": start, "slot": slot, "expert": expert,
            "row": start[expert] + rank, "rank": rank, "capacity": capacity}


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
    s = {"case": case, "op": op}
    if op == "norm":
        T, H = case["tokens"], case["hidden"]
        s["x"] = _stream((T, H), gen, dev)
        s["residual"] = _stream((T, H), gen, dev) if case["residual"] else None
        w = 1.0 + 0.2 * torch.randn(H, generator=gen, device=dev)
        s["weight"] = w.bfloat16() if case["weight"] == "bf16" else w
        if own:
            import combine_ep_layout_08_amd as ep
            s["call"] = ep.bind_add_rmsnorm(
                s["x"], s["weight"], residual=s["residual"], eps=EPS, want_y=case["y"],
                scale_format=None if case["scales"] == "none" else case["scales"], want_rstd=True)
    elif op == "norm_grad":
        T, H = case["tokens"], case["hidden"]
        s["z"] = _stream((T, H), gen, dev)
        s["grad"] = _normal((T, H), gen, dev, 1e-2)
        s["grad_residual"] = _normal((T, H), gen, dev, 1e-2) if case["residual"] else None
        w = 1.0 + 0.2 * torch.randn(H, generator=gen, device=dev)
        s["weight"] = w.bfloat16() if case["weight"] == "bf16" else w
        s["rstd"] = (1.0 / torch.sqrt(s["z"].double().square().mean(1) + EPS)).float()
    elif op == "w4":
        E, N, K = case["experts"], case["n"], case["k"]
        r = s["routing"] = _routing(case, gen, dev)
        w = torch.randn((E, N, K // case["group"], case["group"]), generator=gen, device=dev)
        s["codes"], s["scales"] = _weights(w.mul_(K ** -0.5), case["format"])
        rows = case["tokens"] if case["rows"] == "tokens" else r["capacity"]
        x = _normal((rows, K), gen, dev)
        s["x"], s["sf"] = (x, None) if case["x"] == "bf16" else _fp8(x.float(), case["x"])
        # the batch as its active experts see it: each with its rows, the shorter ones repeated
        seen = s["active"] = torch.nonzero(r["counts"]).reshape(-1)
        most = max(1, int(r["counts"].max()))
        place = torch.arange(most, device=dev)
        s["filled"] = place < r["counts"][seen][:, None]
        s["table"] = r["start"][seen][:, None] + torch.where(s["filled"], place, 0)
        source = torch.zeros(r["capacity"], dtype=torch.long, device=dev)
        source[r["row"]] = r["slot"] // case["topk"]
        s["gather"] = source[s["table"]] if case["rows"] == "tokens" else s["table"]
        s["out"] = torch.zeros((r["capacity"], N), dtype=torch.bfloat16, device=dev)
        if own:
            import combine_ep_layout_08_amd as ep
            s["handle"] = _handle(case, r)
            s["call"] = s["handle"].bind_expert_w4(
                s["x"], ep.pack_w4(s["codes"], s["scales"]), sf=s["sf"],
                token_rows=case["rows"] == "tokens", out=s["out"])
    else:
        inter = case["inter"]
        r = s["routing"] = _routing(case, gen, dev)
        cap = r["capacity"]
        s["gate_up"] = _normal((cap, 2 * inter), gen, dev, 1.5)
        s["weights"] = torch.rand(cap, generator=gen, device=dev) if case["weights"] else None
        if own:
            s["handle"] = _handle(case, r)
        if op == "act":
            eight = case["out"] != "bf16"
            s["h"] = torch.zeros((cap, inter), dtype=torch.uint8 if eight else torch.bfloat16,
                                 device=dev)
            s["h_sf"] = _scales_like(cap, inter, case["out"], dev) if eight else None
            if case["checkpoint"] != "none":
                s["saved"] = torch.zeros((cap, 2 * inter), dtype=torch.uint8, device=dev)
                s["saved_sf"] = _scales_like(cap, 2 * inter, case["checkpoint"], dev)
            if own:
                s["call"] = s["handle"].bind_swiglu(
                    s["gate_up"], row_weights=s["weights"],
                    scale_format=case["out"] if eight else None, out=s["h"], out_sf=s["h_sf"],
                    checkpoint=None if case["checkpoint"] == "none" else case["checkpoint"],
                    saved=s.get("saved"), saved_sf=s.get("saved_sf"))
        else:
            s["saved"], s["saved_sf"] = s.pop("gate_up"), None
            if case["saved"] != "bf16":
                s["saved"], s["saved_sf"] = _fp8(s["saved"].float(), case["saved"])
            s["grad"] = _normal((cap, inter), gen, dev, 1e-2)
            s["grad_gate_up"] = torch.zeros((cap, 2 * inter), dtype=torch.bfloat16, device=dev)
            s["grad_weights"] = torch.zeros(cap, device=dev) if case["weights"] else None
            s["h"] = (torch.zeros((cap, inter), dtype=torch.bfloat16, device=dev)
                      if case["again"] else None)
    return s


def _scales_like(rows, cols, kind, dev):
    packs = cols // 128 if kind == "f32" else (cols // 128 + 3) // 4
    return torch.zeros((rows, packs), dtype=torch.float32 if kind == "f32" else torch.int32,
                       device=dev)


def _weights(w, fmt):
    """4-bit codes, two a byte with the even channel in the low half, and a scale for each group,
    from weights [experts, n, groups, group]."""
    amax = w.abs().amax(3, keepdim=True)
    if fmt == "int4":
        scale = (amax / 7.0).bfloat16()
        code = (w / scale.float()).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
    else:
        e = torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2.0
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
        v = w / torch.exp2(e)
        code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8)
        code += (v < 0).to(torch.uint8) * 8
        scale = (e + 127.0).to(torch.uint8)
    code = code.reshape(w.shape[0], w.shape[1], -1)
    return (code[..., 0::2] + code[..., 1::2] * 16).contiguous(), scale.squeeze(3).contiguous()


# ------------------------------------------------------------------ plain forms

def _pack(e):
    """Exponents [rows, blocks] as 4-byte packs, the lowest block in the low byte."""
    e = torch.nn.functional.pad(e.to(torch.uint8), (0, -e.shape[1] % 4))
    return e.contiguous().view(torch.int32)


def _fp8(v, kind):
    """E4M3 codes of fp32 rows in blocks of 128 channels, and the blocks' scales."""
    b = v.reshape(v.shape[0], -1, 128)
    s = b.abs().amax(2).clamp_min(1e-12)
    s = s / torch.full_like(s, E4M3_MAX)      # by a number, torch multiplies with its reciprocal
    if kind == "ue8m0":
        bits = s.view(torch.int32)
        e = (bits >> 23) + ((bits & 0x7FFFFF) != 0).int()
        s, packed = (e << 23).view(torch.float32), _pack(e)
    q = (b / s[..., None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(v.shape).view(torch.uint8), packed if kind == "ue8m0" else s


def _unpack(sf, blocks):
    """The scales' values [rows, blocks]."""
    if sf.dtype == torch.float32:
        return sf
    e = sf.contiguous().view(torch.uint8)[:, :blocks].int()
    return (e << 23).view(torch.float32)


def _values(q, sf):
    """What 8-bit rows stand for."""
    b = q.view(torch.float8_e4m3fn).float().reshape(q.shape[0], -1, 128)
    return (b * _unpack(sf, b.shape[1])[..., None]).reshape(q.shape)


def _seen(q, sf):
    """Codes and scales as the numbers that they are."""
    if q is None:
        return None
    if sf.dtype == torch.int32:
        sf = sf.view(torch.uint8).view(torch.float8_e8m0fnu)
    return [q.view(torch.float8_e4m3fn), sf]


def _plain_norm(s, kind, want_y):
    z = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    z = z.bfloat16()
    f = z.float()
    rstd = (1.0 / torch.sqrt(f.double().square().mean(1) + EPS)).float()
    y = f * rstd[:, None] * s["weight"].float()
    q, sf = (None, None) if kind == "none" else _fp8(y, kind)
    return y.bfloat16() if want_y else None, z, q, sf, rstd


def _plain_norm_grad(s):
    z, g, r = s["z"].float(), s["grad"].float(), s["rstd"][:, None]
    gw = g * s["weight"].float()
    n = z * r
    c = (gw * n).mean(1, keepdim=True)
    gx = (gw - n * c) * r
    if s["grad_residual"] is not None:
        gx = gx + s["grad_residual"].float()
    return gx.bfloat16(), (g * n).sum(0)


def _plain_weights(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(2)
    if scales.dtype == torch.bfloat16:
        v, f = c.float() - 8.0, scales.float()
    else:
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)[c.int()]
        f = (scales.int() << 23).view(torch.float32)
    return (v.reshape(*f.shape, -1) * f[..., None]).reshape(c.shape)


def _plain_w4(s):
    if s["active"].numel():
        w = _plain_weights(s["codes"][s["active"]], s["scales"][s["active"]])
        x = s["x"][s["gather"]]
        if s["sf"] is not None:
            flat = s["gather"].reshape(-1)
            x = _values(s["x"][flat], s["sf"][flat]).reshape(x.shape)
        y = torch.matmul(w, x.float().transpose(1, 2).contiguous()).transpose(1, 2)
        s["out"][s["table"][s["filled"]]] = y[s["filled"]].bfloat16()
    return s["out"]


def _plain_act(s):
    rows = s["routing"]["row"]
    gu = s["gate_up"][rows].float()
    g, u = gu.chunk(2, 1)
    h = g / (1.0 + torch.exp(-g)) * u
    if s["weights"] is not None:
        h = h * s["weights"][rows][:, None]
    if s["h_sf"] is None:
        s["h"][rows] = h.bfloat16()
    else:
        s["h"][rows], s["h_sf"][rows] = _fp8(h, s["case"]["out"])
    if s["case"]["checkpoint"] != "none":
        s["saved"][rows], s["saved_sf"][rows] = _fp8(gu, s["case"]["checkpoint"])


def _plain_act_grad(s):
    rows = s["routing"]["row"]
    gu = s["saved"][rows]
    gu = gu.float() if s["saved_sf"] is None else _values(gu, s["saved_sf"][rows])
    g, u = gu.chunk(2, 1)
    gh = s["grad"][rows].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    whole = silu * u
    wgh = gh
    if s["weights"] is not None:
        w = s["weights"][rows][:, None]
        s["grad_weights"][rows] = (gh * whole).sum(1)
        whole, wgh = whole * w, gh * w
    slope = sig * (1.0 + g * (1.0 - sig))
    s["grad_gate_up"][rows] = torch.cat((wgh * u * slope, wgh * silu), 1).bfloat16()
    if s["h"] is not None:
        s["h"][rows] = whole.bfloat16()


def run(state):
    s, case = state, state["case"]
    op = s["op"]
    if op == "norm":
        y, z, q, sf, rstd = s["call"]() if own else _plain_norm(s, case["scales"], case["y"])
        return {"y": y, "z": z if case["residual"] else None, "q": _seen(q, sf), "rstd": rstd}
    if op == "norm_grad":
        if own:
            import combine_ep_layout_08_amd as ep
            gx, gw = ep.add_rmsnorm_backward(s["grad"], s["z"], s["weight"], s["rstd"],
                                             grad_residual=s["grad_residual"])
        else:
            gx, gw = _plain_norm_grad(s)
        return {"x": gx, "weight": gw}
    if op == "w4":
        return {"y": s["call"]() if own else _plain_w4(s)}
    if op == "act":
        if own:
            s["call"]()
        else:
            _plain_act(s)
        h = s["h"] if s["h_sf"] is None else _seen(s["h"], s["h_sf"])
        return {"h": h, "saved": _seen(s.get("saved"), s.get("saved_sf"))}
    if own:
        s["handle"].swiglu_backward(s["grad"], s["saved"], s["saved_sf"],
                                    row_weights=s["weights"], grad_gate_up=s["grad_gate_up"],
                                    grad_row_weights=s["grad_weights"], out=s["h"])
    else:
        _plain_act_grad(s)
    return {"gate_up": s["grad_gate_up"], "weights": s["grad_weights"], "h": s["h"]}


# ------------------------------------------------------------------ in 64 bits

def _exact_codes(rows, kind):
    """The 8-bit rows' codes and scales as real numbers."""
    T, C = rows.shape
    top = rows.abs().reshape(T, C // 128, 128).max(2).values
    scale = torch.maximum(top, torch.full_like(top, 1e-12)) / E4M3_MAX
    out = scale
    if kind == "ue8m0":
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
        # the bytes behind the last block are zero, and 2^-127 as exponents
        out = torch.nn.functional.pad(scale, (0, -(C // 128) % 4), value=2.0 ** -127)
    q = rows / scale.repeat_interleave(128, 1)
    # nearest number with three bits behind the leading one, or multiple of 2^-9
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3.0)
    return [(q / step).round() * step, out]


def _exact_eight(q, sf):
    """Real numbers behind stored codes and scales."""
    v = q.view(torch.float8_e4m3fn).to(torch.float64)
    if sf.dtype == torch.int32:
        e = sf.contiguous().view(torch.uint8)[:, :q.shape[1] // 128].to(torch.float64)
        sf = torch.pow(2.0, e - 127.0)
    return v * sf.to(torch.float64).repeat_interleave(128, 1)


def exact(case, seed):
    global own
    mode, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mode
    op = s["op"]
    if op == "norm":
        z = s["x"].to(torch.float64)
        if s["residual"] is not None:
            z = z + s["residual"].to(torch.float64)
        v = z.to(torch.bfloat16).to(torch.float64)        # the norm is of the rounded sum
        rstd = torch.rsqrt((v * v).sum(1) / v.shape[1] + EPS)
        y = torch.einsum("th,t,h->th", v, rstd, s["weight"].to(torch.float64))
        q = None if case["scales"] == "none" else _exact_codes(y, case["scales"])
        return {"y": y if case["y"] else None, "z": z if case["residual"] else None, "q": q,
                "rstd": rstd}
    if op == "norm_grad":
        # y_h = w_h z_h r(z); dr/dz_h = -r^3 z_h / H
        z, g = s["z"].to(torch.float64), s["grad"].to(torch.float64)
        r, w = s["rstd"].to(torch.float64), s["weight"].to(torch.float64)
        along = torch.einsum("th,th,h->t", g, z, w) * r ** 3 / z.shape[1]
        gx = torch.einsum("th,h,t->th", g, w, r) - torch.einsum("t,th->th", along, z)
        if s["grad_residual"] is not None:
            gx = gx + s["grad_residual"].to(torch.float64)
        return {"x": gx, "weight": torch.einsum("th,th,t->h", g, z, r)}
    r = s["routing"]
    if op == "w4":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
        x = s["x"].to(torch.float64) if s["sf"] is None else _exact_eight(s["x"], s["sf"])
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=x.device)
        for e in torch.unique(r["expert"]).tolist():
            mine = r["expert"] == e
            rows, slots = r["row"][mine], r["slot"][mine]
            byte, sc = s["codes"][e].long(), s["scales"][e]
            w = torch.empty((case["n"], case["k"]), dtype=torch.float64, device=x.device)
            if case["format"] == "int4":
                w[:, 0::2], w[:, 1::2] = (byte % 16 - 8).double(), (byte // 16 - 8).double()
                sc = sc.to(torch.float64)
            else:
                w[:, 0::2], w[:, 1::2] = table[byte % 16], table[byte // 16]
                sc = torch.pow(2.0, sc.to(torch.float64) - 127.0)
            w *= sc.repeat_interleave(case["group"], 1)
            src = slots // case["topk"] if case["rows"] == "tokens" else rows
            out[rows] = x[src] @ w.t()
        return {"y": out}
    cap, inter = r["capacity"], case["inter"]
    rows = r["row"]

    def whole(part, cols=None):
        full = torch.zeros((cap,) if part.dim() == 1 else (cap, part.shape[1]),
                           dtype=torch.float64, device=part.device)
        full[rows] = part
        return full

    def whole_codes(part, kind):
        q, sf = _exact_codes(part, kind)
        sf_all = whole(sf)
        if kind == "ue8m0":                               # a zero byte is the exponent -127
            left = torch.ones(cap, dtype=torch.bool, device=q.device)
            left[rows] = False
            sf_all[left] = 2.0 ** -127
        return [whole(q), sf_all]

    if op == "act":
        gu = s["gate_up"][rows].to(torch.float64)
        h = gu[:, :inter] * torch.sigmoid(gu[:, :inter]) * gu[:, inter:]
        if s["weights"] is not None:
            h = h * s["weights"][rows].to(torch.float64).unsqueeze(1)
        saved = None if case["checkpoint"] == "none" else whole_codes(gu, case["checkpoint"])
        return {"h": whole(h) if case["out"] == "bf16" else whole_codes(h, case["out"]),
                "saved": saved}
    gu = s["saved"][rows]
    gu = gu.to(torch.float64) if s["saved_sf"] is None else _exact_eight(gu, s["saved_sf"][rows])
    a, b = gu[:, :inter], gu[:, inter:]
    p = torch.sigmoid(a)
    gh = s["grad"][rows].to(torch.float64)
    w = (torch.ones(rows.numel(), dtype=torch.float64, device=gh.device) if s["weights"] is None
         else s["weights"][rows].to(torch.float64))
    ga = torch.einsum("ri,ri,r->ri", gh, b * (p + a * p * (1.0 - p)), w)
    gb = torch.einsum("ri,ri,r->ri", gh, a * p, w)
    return {"gate_up": whole(torch.cat((ga, gb), 1)),
            "weights": None if s["weights"] is None else whole((gh * a * p * b).sum(1)),
            "h": whole(a * p * b * w.unsqueeze(1)) if case["again"] else None}
