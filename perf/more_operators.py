"""What is measured of the whole MoE layer on a few tokens (router, selection, routed and
always-on experts), and of the expert operation in 8-bit integers with a scale for each
token and output channel: the row quantisation, the products grouped by expert, and whole
passes.

Layer: with router W_r [N][d] and an optional bias b [N],

    l_te = W_r[e] x_t,   s_te = exp(l_te) / sum_e exp(l_te)   or   1 / (1 + exp(-l_te))
    the m experts of the largest s_te + b_e (equal ones: lower id first)
    w_tj = scale * s_tj / (sum_j s_tj where renormalised, else 1)
    y_t  = sum_j w_tj FFN_tj(x_t) + sum over the always-on experts of FFN(x_t)
    FFN_e(x) = W_down[e] (silu(W_gate[e] x) * (W_up[e] x)),   silu(z) = z / (1 + exp(-z))

y has the type of x and the layer (bfloat16 or float32).

8-bit integers: a row v (a token's activations, or one output channel of a matrix) has the
scale max|v| / 127, and a value's code is 127 v / max|v| to the nearest integer, ties to
even.  With ids [n][m], weights w [n][m] and slots s = t*m + j sorted stably by expert (row
r holds slot slot_by_expert[r]; ids outside [0, N) take no part):

    gate_up   h_r = silu(W_gate[e] x_t) * (W_up[e] x_t), rounded to bfloat16, then quantised
    down      y_t = round( sum_j w_tj W_down[e_tj] h_row(t,j) ) to bfloat16
    pass      both, from x (quantised first), ids and w
"""
import math

import torch

own = False

# Layer shapes: experts, experts per token, token width, hidden width.
FINE = {"N": 128, "m": 8, "d": 2048, "d_ff": 768}     # many narrow experts
MID = {"N": 64, "m": 6, "d": 2048, "d_ff": 1408}      # fewer, wider ones
WIDE = {"N": 8, "m": 2, "d": 4096, "d_ff": 14336}     # few large ones


def listed():
    return [
        # one decoded token: latency
        {"name": "layer_bf16_1", "op": "layer", "type": "bf16", "layout": "tiled", "n": 1, "score": "softmax",
         "bias": False, "renorm": True, "scale": 1.0, "shared": 0, **FINE},
        # a verification pass of five tokens with two always-on experts
        {"name": "layer_bf16_5_shared", "op": "layer", "type": "bf16", "layout": "tiled", "n": 5, "score": "softmax",
         "bias": False, "renorm": False, "scale": 1.0, "shared": 2, **MID},
        # a 32-node draft tree, scores balanced by a bias
        {"name": "layer_bf16_32", "op": "layer", "type": "bf16", "layout": "tiled", "n": 32, "score": "sigmoid",
         "bias": True, "renorm": True, "scale": 2.5, "shared": 0, **FINE},
        # a small layer in fp32, odd sizes
        {"name": "layer_f32_7", "op": "layer", "type": "f32", "layout": "plain", "n": 7, "score": "sigmoid",
         "bias": True, "renorm": True, "scale": 1.0, "shared": 1, "N": 70, "m": 5, "d": 200, "d_ff": 168},
        # one decoded batch's activations, hidden width of the wider experts
        {"name": "quant_int8_129x1408", "op": "quant", "n": 129, "d": 1408},
        # a prompt chunk's activations
        {"name": "quant_int8_16384x2048", "op": "quant", "n": 16384, "d": 2048},
        # gate and up of a prompt chunk with skewed routing
        {"name": "gate_up_int8_4096", "op": "gate_up", "layout": "tiled", "n": 4096, "zipf": 1.1, **FINE},
        # down of an odd chunk, row-major codes as a checkpoint holds them
        {"name": "down_int8_2777", "op": "down", "layout": "plain", "n": 2777, "zipf": 0.0, **MID},
        # one decoded token: latency
        {"name": "pass_int8_1", "op": "pass", "layout": "tiled", "n": 1, "zipf": 0.0, "pad": 0, **FINE},
        # one pass over a 32-node draft tree
        {"name": "pass_int8_32", "op": "pass", "layout": "tiled", "n": 32, "zipf": 1.1, "pad": 0, **FINE},
        # a padded batch of prompts
        {"name": "pass_int8_8191", "op": "pass", "layout": "tiled", "n": 8191, "zipf": 1.1, "pad": 130, **FINE},
        # a prompt chunk on few large experts
        {"name": "pass_int8_2048_wide", "op": "pass", "layout": "tiled", "n": 2048, "zipf": 0.0, "pad": 0, **WIDE},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "layer", "layer", "quant", "gate_up", "down", "pass", "pass"])
    if op == "quant":
        return {"op": op, "n": _log_int(rng, 1, 16384), "d": 16 * _log_int(rng, 1, 128)}
    if rng.random() < 0.5:
        shape = dict(rng.choice([FINE, MID]))
    else:
        N = _log_int(rng, 3, 160)
        shape = {"N": N, "m": rng.randint(1, min(N, 8)), "d": 16 * rng.randint(8, 160), "d_ff": 16 * rng.randint(6, 96)}
    whole = shape["d"] % 64 == 0 and shape["d_ff"] % 64 == 0
    layout = rng.choice(["plain", "tiled"]) if whole else "plain"
    if op == "layer":
        typ = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "type": typ, "layout": layout, "n": _log_int(rng, 1, min(64, 250 // shape["m"])),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, round(rng.uniform(0.5, 16.0), 2)]), "shared": rng.choice([0, 0, 1, 2]), **shape}
    most = 8191 * 8 * 2048 * 768 // (shape["m"] * shape["d"] * shape["d_ff"])
    n = _log_int(rng, 1, min(8191, most))
    c = {"op": op, "layout": layout, "n": n, "zipf": round(rng.uniform(0, 1.3), 2), **shape}
    if op == "pass":
        c["pad"] = rng.choice([0, rng.randint(0, n // 8)])
    return c


# --------------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _randn(seed, salt, *shape):
    return torch.randn(*shape, generator=_gen(seed, salt), device="cuda", dtype=torch.float32)


def _routing(case, seed):
    """ids [n][m] int32 of the m largest logits (popularity falls as rank^-zipf), w their softmax;
    the last `pad` tokens hold no token: id -1, weight 0."""
    n, N, m = case["n"], case["N"], case["m"]
    rank = torch.randperm(N, generator=_gen(seed, 1), device="cuda").float() + 1
    top, ids = (_randn(seed, 2, n, N) - case["zipf"] * rank.log()).topk(m, dim=1)
    w = top.softmax(dim=1)
    if case.get("pad"):
        ids[n - case["pad"]:] = -1
        w[n - case["pad"]:] = 0
    return ids.to(torch.int32).contiguous(), w.contiguous()


def _quant(v):
    """Rows of v (last axis) to (int8 codes, float32 scales).  127 v / max in 64 bits: halves are exact there."""
    a = v.abs().amax(dim=-1, keepdim=True)
    q = torch.round(v.double() * 127 / torch.where(a > 0, a, torch.ones_like(a)).double())
    return q.to(torch.int8).contiguous(), (a / 127).squeeze(-1).contiguous()


def _quant_matrices(w):
    """As _quant, an expert at a time (the 64-bit values of a large layer would not fit beside it)."""
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    s = torch.empty(w.shape[:2], dtype=torch.float32, device=w.device)
    for e in range(w.shape[0]):
        q[e], s[e] = _quant(w[e])
    return q, s


def _weights(case, seed, names):
    """{name: tensor of the layer's type, or (codes, scales)} of the named matrices."""
    d, f = case["d"], case["d_ff"]
    out = {}
    for i, name in enumerate(("gate", "up", "down", "gate_shared", "up_shared", "down_shared")):
        if name not in names:
            continue
        E = case["shared"] if name.endswith("shared") else case["N"]
        w = _randn(seed, 10 + i, E, *((d, f) if name.startswith("down") else (f, d))).mul_(0.02)
        if case["op"] != "layer":
            out[name] = _quant_matrices(w.to(torch.bfloat16).float())
        else:
            out[name] = w.to(torch.bfloat16) if case["type"] == "bf16" else w
    return out


def _layer(case, weights):
    import expert_ffn_amd as efa
    N, d, f = case["N"], case["d"], case["d_ff"]
    if case["op"] == "layer":
        shared = tuple(weights[k + "_shared"] for k in ("gate", "up", "down")) if case["shared"] else None
        layer = efa.Layer(weights["gate"], weights["up"], weights["down"], m=case["m"], shared=shared)
    else:
        none = {"gate": (f, d), "up": (f, d), "down": (d, f)}  # a product alone needs only its own matrices
        have = {k: weights[k] if k in weights else (torch.empty(N, R, K, dtype=torch.int8, device="cuda"),
                                                   torch.empty(N, R, dtype=torch.float32, device="cuda"))
                for k, (R, K) in none.items()}
        layer = efa.Int8Layer(have["gate"], have["up"], have["down"], m=case["m"])
    return layer.tiled_copy() if case["layout"] == "tiled" else layer


def prepare(case, seed):
    st = {"case": case}
    op, n, d = case["op"], case["n"], case["d"]
    if own:
        import expert_ffn_amd as efa
    if op == "quant":
        # activations behind a norm: a few features are much larger than the rest
        x = _randn(seed, 3, n, d) * torch.exp(_randn(seed, 4, 1, d))
        st["x"] = x.to(torch.bfloat16)
        if own:
            st["out"] = efa.Quantized(torch.empty(n, d, dtype=torch.int8, device="cuda"),
                                      torch.empty(n, dtype=torch.float32, device="cuda"))
            st["values"] = torch.empty_like(st["x"])
        return st
    m, N, f = case["m"], case["N"], case["d_ff"]
    if op == "layer":
        typ = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        names = ("gate", "up", "down") + (("gate_shared", "up_shared", "down_shared") if case["shared"] else ())
        weights = _weights(case, seed, names)
        st["x"] = _randn(seed, 3, n, d).to(typ)
        st["router"] = (_randn(seed, 7, N, d) / math.sqrt(d)).to(typ)  # logits of unit variance
        st["bias"] = _randn(seed, 8, N) * 0.05 if case["bias"] else None
        if own:
            st["layer"] = _layer(case, weights)
            st["gate"] = efa.Router(st["router"], score=case["score"], bias=st["bias"], renorm=case["renorm"], scale=case["scale"])
            st["ws"] = st["layer"].pass_workspace(n)
            st["y"] = torch.empty_like(st["x"])
        else:
            st["weights"] = weights
        return st
    ids, w = _routing(case, seed)
    st.update(ids=ids, w=w)
    weights = _weights(case, seed, {"gate_up": ("gate", "up"), "down": ("down",), "pass": ("gate", "up", "down")}[op])
    if own:
        st["layer"] = _layer(case, weights)
        st["ws"] = st["layer"].grouped_workspace(n)
        st["y"] = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    else:
        st["weights"] = weights
    if op != "pass":
        st["group"] = _group(ids, N)
        if own:
            st["group"] = efa.Grouping(*st["group"])
    if op == "down":
        # h as gate and up leave it: rows in group order
        h = torch.nn.functional.silu(_randn(seed, 5, n * m, f) * (0.02 * math.sqrt(d))) * (_randn(seed, 6, n * m, f) * (0.02 * math.sqrt(d)))
        st["h"] = _quant(h.to(torch.bfloat16).float())
        if own:
            st["h"] = efa.Quantized(*st["h"])
    else:
        st["x"] = _randn(seed, 3, n, d).to(torch.bfloat16)
        if op == "gate_up":
            st["x"] = _quant(st["x"].float())
            if own:
                st["x"] = efa.Quantized(*st["x"])
                st["out"] = efa.Quantized(torch.empty(n * m, f, dtype=torch.int8, device="cuda"),
                                          torch.empty(n * m, dtype=torch.float32, device="cuda"))
                st["h"] = torch.empty(n * m, f, dtype=torch.bfloat16, device="cuda")
    return st


# --------------------------------------------------------------------------- the plain form

def _group(ids, N):
    """count [N], offset [N+1], slot_by_expert [n*m], distinct [N], (U, status) of valid, distinct ids."""
    n, m = ids.shape
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < N)
    key = torch.where(ok, flat, N)
    order = torch.sort(key, stable=True)[1]
    count = torch.zeros(N + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))[:N]
    offset = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count, 0)])
    slot = torch.where(torch.arange(n * m, device=ids.device) < offset[N], order, -1)
    distinct = torch.sort(torch.where(count > 0, torch.arange(N, device=ids.device), N))[0]
    distinct = torch.where(distinct < N, distinct, -1)
    status = torch.stack([(count > 0).sum(), torch.where((~ok).any(), -5, 0)])
    return tuple(t.to(torch.int32) for t in (count, offset, slot, distinct, status))


def _ffn(x, gate, up, down):
    g = x @ gate.float().T
    return (g / (1 + torch.exp(-g)) * (x @ up.float().T)) @ down.float().T


def _layer_pass(st):
    case, W, x = st["case"], st["weights"], st["x"].float()
    m = case["m"]
    # 64 bits: the selection is decided by values next to each other
    logits = st["x"].double() @ st["router"].double().T
    if case["score"] == "softmax":
        s = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-logits))
    key = logits if st["bias"] is None else s + st["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :m]
    w = torch.gather(s, 1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = (w * case["scale"]).float()
    y = torch.zeros(case["n"], case["d"], device="cuda")
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y[t] += w[t, j][:, None] * _ffn(x[t], W["gate"][e], W["up"][e], W["down"][e])
    for e in range(case["shared"]):
        y += _ffn(x, W["gate_shared"][e], W["up_shared"][e], W["down_shared"][e])
    return y.to(st["x"].dtype)


def _product(xq, xs, w, e):
    """Sums of codes, whole numbers beyond 2^24, in 64 bits; then the scales."""
    return (xq.double() @ w[0][e].double().T).float() * xs[:, None] * w[1][e][None, :]


def _gate_up(st, x, group):
    """h in bfloat16, quantised: rows in group order."""
    case, W = st["case"], st["weights"]
    at = group[1].tolist()
    h = torch.zeros(case["n"] * case["m"], case["d_ff"], device="cuda")
    for e in range(case["N"]):
        if at[e + 1] > at[e]:
            t = group[2][at[e]:at[e + 1]].long() // case["m"]
            g, u = _product(x[0][t], x[1][t], W["gate"], e), _product(x[0][t], x[1][t], W["up"], e)
            h[at[e]:at[e + 1]] = g / (1 + torch.exp(-g)) * u
    return _quant(h.to(torch.bfloat16).float())


def _down(st, h, group):
    case, W = st["case"], st["weights"]
    n, m, d = case["n"], case["m"], case["d"]
    at = group[1].tolist()
    o = torch.zeros(n * m, d, device="cuda")
    for e in range(case["N"]):
        if at[e + 1] > at[e]:
            r = slice(at[e], at[e + 1])
            o[group[2][r].long()] = _product(h[0][r], h[1][r], W["down"], e)
    return (o.view(n, m, d) * st["w"][:, :, None]).sum(dim=1).to(torch.bfloat16)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import expert_ffn_amd as efa
        if op == "layer":
            return {"y": efa.layer_pass(st["layer"], st["gate"], st["x"], y=st["y"], ws=st["ws"])}
        if op == "quant":
            q = efa.quant_rows(st["x"], out=st["out"], dtype=torch.int8)
            return {"values": efa.dequant_rows(q, out=st["values"]), "scale": q.scale}
        if op == "gate_up":
            h = efa.grouped_gate_up(st["layer"], st["x"], st["group"], out=st["out"], ws=st["ws"])
            return {"h": efa.dequant_rows(h, out=st["h"])}
        if op == "down":
            return {"y": efa.grouped_down(st["layer"], st["h"], st["ids"], st["w"], st["group"], y=st["y"], ws=st["ws"])}
        return {"y": efa.expert_grouped(st["layer"], st["x"], st["ids"], st["w"], y=st["y"], ws=st["ws"])}
    if op == "layer":
        return {"y": _layer_pass(st)}
    if op == "quant":
        q, s = _quant(st["x"].float())
        return {"values": (q.float() * s[:, None]).to(torch.bfloat16), "scale": s}
    group = st["group"] if op != "pass" else _group(st["ids"], case["N"])
    if op == "gate_up":
        q, s = _gate_up(st, st["x"], group)
        return {"h": (q.float() * s[:, None]).to(torch.bfloat16)}
    h = st["h"] if op == "down" else _gate_up(st, _quant(st["x"].float()), group)
    return {"y": _down(st, h, group)}


# --------------------------------------------------------------------------- 64 bits, from the definition

def _exact_quant(v):
    """(codes, scales) of the rows of v in float64: the whole number k with |127 v / a - k| least, of two
    such numbers the even one.  254 |v| + a and 2 a k are sums of few bits, so the comparison is exact."""
    a = v.abs().max(dim=1).values[:, None]
    one = torch.where(a > 0, a, torch.ones_like(a))
    top = 254 * v.abs() + one
    k = torch.floor(top / (2 * one))
    half = (top - 2 * one * k == 0) & (k % 2 == 1)
    return torch.sign(v) * torch.where(half, k - 1, k), (a / 127)[:, 0]


def _exact_ffn(x, *matrices):
    gate, up, down = (w.double() for w in matrices)
    z = x @ gate.T
    return (z * torch.sigmoid(z) * (x @ up.T)) @ down.T


def _exact_layer(case, st):
    n, N, m, W = case["n"], case["N"], case["m"], st["weights"]
    x = st["x"].double()
    y = torch.zeros(n, case["d"], dtype=torch.float64, device="cuda")
    l = torch.stack([(x * st["router"][e].double()).sum(dim=1) for e in range(N)], dim=1)
    s = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
    key = (l if st["bias"] is None else s + st["bias"].double()).cpu().tolist()
    s = s.cpu()
    of = {}
    for t in range(n):
        chosen = sorted(range(N), key=lambda e: (-key[t][e], e))[:m]
        total = float(sum(s[t, e] for e in chosen)) if case["renorm"] else 1.0
        for e in chosen:
            of.setdefault(e, []).append((t, case["scale"] * float(s[t, e]) / total))
    for e, rows in of.items():
        t = torch.tensor([r[0] for r in rows], device="cuda")
        w = torch.tensor([r[1] for r in rows], dtype=torch.float64, device="cuda")
        y[t] += w[:, None] * _exact_ffn(x[t], W["gate"][e], W["up"][e], W["down"][e])
    for e in range(case["shared"]):
        y += _exact_ffn(x, W["gate_shared"][e], W["up_shared"][e], W["down_shared"][e])
    return {"y": y}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "layer":
        return _exact_layer(case, st)
    if op == "quant":
        q, s = _exact_quant(st["x"].double())
        return {"values": q * s[:, None], "scale": s}
    n, m, N, W = case["n"], case["m"], case["N"], st["weights"]
    ids = st["ids"].long()
    order = torch.argsort(ids.reshape(-1) + torch.where(ids.reshape(-1) < 0, N + 1, 0), stable=True)

    def values(w, e):
        return w[0][e].double() * w[1][e].double()[:, None]

    if op == "down":
        q, s = st["h"]
        hs = torch.zeros(n * m, case["d_ff"], dtype=torch.float64, device="cuda")
        hs[order] = q.double() * s.double()[:, None]
    else:
        q, s = _exact_quant(st["x"].double()) if op == "pass" else st["x"]
        x = q.double() * s.double()[:, None]
        hs = torch.zeros(n * m, case["d_ff"], dtype=torch.float64, device="cuda")  # by slot
        for e in range(N):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                z = x[t] @ values(W["gate"], e).T
                hs[t * m + j] = z * torch.sigmoid(z) * (x[t] @ values(W["up"], e).T)
        q, s = _exact_quant(hs.to(torch.bfloat16).double())
        hs = q * s[:, None]
        if op == "gate_up":
            return {"h": hs[order]}
    y = torch.zeros(n, case["d"], dtype=torch.float64, device="cuda")
    for e in range(N):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y.index_add_(0, t, st["w"][t, j].double()[:, None] * (hs[t * m + j] @ values(W["down"], e).T))
    return {"y": y}


# --------------------------------------------------------------------------- work

def work(case):
    op, n, d = case["op"], case["n"], case["d"]
    if op == "quant":  # codes are written, and read once more for their values
        return {"bytes": n * d * (2 + 1 + 2) + 4 * n, "flops": 4 * n * d}
    N, m, f = case["N"], case["m"], case["d_ff"]
    live = n - case.get("pad", 0)
    rows = live * m
    touched = N * (1 - (1 - m / N) ** live)  # experts that some token selects, evenly routed
    if op == "layer":
        b = 2 if case["type"] == "bf16" else 4
        experts = touched + case["shared"]
        return {"bytes": b * (experts * 3 * d * f + N * d + 2 * n * d),
                "flops": 2 * (rows + n * case["shared"]) * 3 * d * f + 2 * n * N * d}
    per, channels = {"gate_up": (2, 2 * f), "down": (1, d), "pass": (3, 2 * f + d)}[op]
    moved = {"gate_up": n * (d + 4) + rows * (f + f + 4 + 2 * f), "down": rows * (f + 4 + 8) + n * d * 2,
             "pass": n * d * 4 + n * m * 8}[op]  # gate_up: codes written, and read again for their values
    return {"bytes": touched * (per * d * f + 4 * channels) + moved, "flops": 2 * rows * per * d * f}
