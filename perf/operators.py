"""What is measured of the expert operation on grouped rows: the grouping of any number
of slots by expert, the products grouped by expert (gate and up with SwiGLU, down with
the weighted sum over a token's experts) in bfloat16 and in 8-bit floating point with a
scale for each block of 128, the block quantisation, and whole passes.

With ids [n][m], weights w [n][m] and slots s = t*m + j sorted stably by expert (row r
holds slot slot_by_expert[r]; ids outside [0, N) take no part):

    gate_up   h_r = round( silu(W_gate[e] x_t) * (W_up[e] x_t) ),   silu(z) = z / (1 + exp(-z))
    down      y_t = round( sum_j w_tj W_down[e_tj] h_row(t,j) )
    pass      both, from x, ids and w

round is to bfloat16; with 8-bit weights x and h are quantised in blocks of 128 along a
row (the pass quantises x first): with k the smallest integer >= -127 such that
max|v| <= 448 * 2^k over the block, the code is e4m3(v * 2^-k), to nearest even, and
stands for code * 2^k.  Weights hold one k for each block of 128 x 128.
"""
import math

import numpy as np
import torch

own = False

# Layer shapes: experts, experts per token, token width, hidden width.
FINE = {"N": 128, "m": 8, "d": 2048, "d_ff": 768}     # many narrow experts
MID = {"N": 64, "m": 6, "d": 2048, "d_ff": 1408}      # fewer, wider ones
WIDE = {"N": 8, "m": 2, "d": 4096, "d_ff": 14336}     # few large ones


def listed():
    return [
        # a short prompt's slots, a little above what one verification pass may hold
        {"name": "group_576", "op": "group", "n": 96, "zipf": 0.0, "pad": 0, **MID},
        # a padded batch of prompts whose last 500 rows hold no token
        {"name": "group_131072_padded", "op": "group", "n": 16384, "zipf": 1.1, "pad": 500, **FINE},
        # one decoded batch's activations, hidden width of the wider experts
        {"name": "quant_129x1408", "op": "quant", "n": 129, "d": 1408},
        # a prompt chunk's activations
        {"name": "quant_16384x2048", "op": "quant", "n": 16384, "d": 2048},
        # gate and up of a prompt chunk with skewed routing, weights as the verification passes hold them
        {"name": "gate_up_bf16_4096", "op": "gate_up", "type": "bf16", "layout": "tiled", "n": 4096, "zipf": 1.1, **FINE},
        # down of an odd chunk, row-major weights as a checkpoint holds them
        {"name": "down_bf16_2777", "op": "down", "type": "bf16", "layout": "plain", "n": 2777, "zipf": 0.0, **MID},
        # one pass over a 32-node draft tree
        {"name": "pass_bf16_32", "op": "pass", "type": "bf16", "layout": "tiled", "n": 32, "zipf": 1.1, "pad": 0, **FINE},
        # a prompt chunk on few large experts
        {"name": "pass_bf16_2048_wide", "op": "pass", "type": "bf16", "layout": "tiled", "n": 2048, "zipf": 0.0, "pad": 0, **WIDE},
        # gate and up in 8 bits, a prompt chunk
        {"name": "gate_up_fp8_4096", "op": "gate_up", "type": "fp8", "layout": "tiled", "n": 4096, "zipf": 0.0, **MID},
        # down in 8 bits
        {"name": "down_fp8_4096", "op": "down", "type": "fp8", "layout": "tiled", "n": 4096, "zipf": 1.1, **FINE},
        # one decoded token: latency
        {"name": "pass_fp8_1", "op": "pass", "type": "fp8", "layout": "tiled", "n": 1, "zipf": 0.0, "pad": 0, **FINE},
        # a padded batch of prompts in 8 bits
        {"name": "pass_fp8_8191", "op": "pass", "type": "fp8", "layout": "tiled", "n": 8191, "zipf": 1.1, "pad": 130, **FINE},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "quant", "gate_up", "down", "pass", "pass"])
    if op == "group":
        N = _log_int(rng, 3, 1024)
        m = rng.randint(1, min(N, 16))
        n = _log_int(rng, 1, 131072 // m)
        return {"op": op, "n": n, "N": N, "m": m, "zipf": round(rng.uniform(0, 1.3), 2), "pad": rng.randint(0, n // 4)}
    if op == "quant":
        return {"op": op, "n": _log_int(rng, 1, 16384), "d": 16 * _log_int(rng, 1, 128)}
    typ = rng.choice(["bf16", "fp8"])
    if rng.random() < 0.5:
        shape = dict(rng.choice([FINE, MID]))
    else:
        N = _log_int(rng, 3, 160)
        shape = {"N": N, "m": rng.randint(1, min(N, 8)), "d": 16 * rng.randint(8, 160), "d_ff": 16 * rng.randint(6, 96)}
    whole = shape["d"] % 64 == 0 and shape["d_ff"] % 64 == 0
    most = 8191 * 8 * 2048 * 768 // (shape["m"] * shape["d"] * shape["d_ff"])
    n = _log_int(rng, 1, min(8191, most))
    c = {"op": op, "type": typ, "layout": rng.choice(["plain", "tiled"]) if whole else "plain", "n": n,
         "zipf": round(rng.uniform(0, 1.3), 2), **shape}
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


def _pow2(k):
    """2^k as float32, -126 <= k <= 127 (0 below)."""
    return ((k.to(torch.int32) + 127).clamp(min=0) << 23).view(torch.float32)


def _exponent(amax):
    """Smallest k >= -127 with amax <= 448 * 2^k (448 = 1.75 * 2^8), from the bits of float32."""
    b = amax.view(torch.int32)
    return ((b >> 23) - 135 + ((b & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=-127)


def _quant_weights(w):
    """float32 [N][R][K] -> e4m3 codes [N][R][K], bytes k + 127 [N][R/128][K/128]."""
    N, R, K = w.shape
    Rb, Kb = -(-R // 128), -(-K // 128)
    p = torch.zeros(N, Rb * 128, Kb * 128, device=w.device)
    p[:, :R, :K] = w
    p = p.view(N, Rb, 128, Kb, 128)
    k = _exponent(p.abs().amax(dim=(2, 4)).contiguous())
    q = (p * _pow2(-k)[:, :, None, :, None]).view(N, Rb * 128, Kb * 128)[:, :R, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), (k + 127).to(torch.uint8)


def _quant_rows(x):
    """float32 [n][K] -> e4m3 codes [n][K], bytes k + 127 [n][K/128]."""
    n, K = x.shape
    Kb = -(-K // 128)
    p = torch.zeros(n, Kb * 128, device=x.device)
    p[:, :K] = x
    p = p.view(n, Kb, 128)
    k = _exponent(p.abs().amax(dim=2).contiguous())
    q = (p * _pow2(-k)[:, :, None]).view(n, Kb * 128)[:, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), (k + 127).to(torch.uint8)


def _row_values(q, s):
    """The values that codes and scale bytes of rows stand for, float32."""
    return q.float() * _pow2(s.to(torch.int32) - 127).repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _weight_values(q, s):
    """One expert's values: codes [R][K], scale bytes [R/128][K/128]."""
    f = _pow2(s.to(torch.int32) - 127).repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
    return q.float() * f[:q.shape[0], :q.shape[1]]


def _weights(case, seed, names):
    """{name: bf16 tensor, or (codes, scale bytes)} of the named matrices."""
    N, d, f = case["N"], case["d"], case["d_ff"]
    out = {}
    for i, name in enumerate(("gate", "up", "down")):
        if name in names:
            w = _randn(seed, 10 + i, N, *((d, f) if name == "down" else (f, d))).mul_(0.02)
            out[name] = w.to(torch.bfloat16) if case["type"] == "bf16" else _quant_weights(w.to(torch.bfloat16).float())
    return out


def _layer(case, weights):
    import expert_ffn_amd as efa
    N, d, f = case["N"], case["d"], case["d_ff"]
    if case["type"] == "bf16":
        none = {"gate": (N, f, d), "up": (N, f, d), "down": (N, d, f)}  # a product alone needs only its own matrices
        have = {k: weights[k] if k in weights else torch.empty(s, dtype=torch.bfloat16, device="cuda") for k, s in none.items()}
        layer = efa.Layer(have["gate"], have["up"], have["down"], m=case["m"])
    else:
        b = lambda v: -(-v // 128)  # noqa: E731
        none = {"gate": (f, d), "up": (f, d), "down": (d, f)}
        have = {k: weights[k] if k in weights else (torch.empty(N, R, K, dtype=torch.float8_e4m3fn, device="cuda"),
                                                   torch.empty(N, b(R), b(K), dtype=torch.uint8, device="cuda"))
                for k, (R, K) in none.items()}
        layer = efa.Fp8Layer(have["gate"], have["up"], have["down"], m=case["m"])
    return layer.tiled_copy() if case["layout"] == "tiled" else layer


def prepare(case, seed):
    st = {"case": case}
    op = case["op"]
    if op == "quant":
        # activations behind a norm: a few features are much larger than the rest
        x = _randn(seed, 3, case["n"], case["d"]) * torch.exp(_randn(seed, 4, 1, case["d"]))
        st["x"] = x.to(torch.bfloat16)
        if own:
            import expert_ffn_amd as efa
            st["out"] = efa.Quantized(torch.empty(case["n"], case["d"], dtype=torch.float8_e4m3fn, device="cuda"),
                                      torch.empty(case["n"], -(-case["d"] // 128), dtype=torch.uint8, device="cuda"))
            st["values"] = torch.empty_like(st["x"])
        return st
    ids, w = _routing(case, seed)
    st.update(ids=ids, w=w)
    if op == "group":
        if own:
            import expert_ffn_amd as efa
            N = case["N"]
            st["out"] = efa.Grouping(*(torch.empty(k, dtype=torch.int32, device="cuda") for k in (N, N + 1, ids.numel(), N, 2)))
            st["ws"] = efa.group_workspace(case["n"], case["m"], case["N"])
        return st
    n, m, d, f = case["n"], case["m"], case["d"], case["d_ff"]
    fp8 = case["type"] == "fp8"
    weights = _weights(case, seed, {"gate_up": ("gate", "up"), "down": ("down",), "pass": ("gate", "up", "down")}[op])
    if own:
        import expert_ffn_amd as efa
        st["layer"] = _layer(case, weights)
        st["ws"] = st["layer"].grouped_workspace(n)
        st["y"] = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    else:
        st["weights"] = weights
    if op != "pass":
        st["group"] = _group(ids, case["N"])
        if own:
            st["group"] = efa.Grouping(*st["group"])
    if op == "down":
        # h as gate and up leave it: rows in group order
        h = torch.nn.functional.silu(_randn(seed, 5, n * m, f) * (0.02 * math.sqrt(d))) * (_randn(seed, 6, n * m, f) * (0.02 * math.sqrt(d)))
        st["h"] = _quant_rows(h) if fp8 else h.to(torch.bfloat16)
        if own and fp8:
            st["h"] = efa.Quantized(*st["h"])
    else:
        x = _randn(seed, 3, n, d)
        st["x"] = x.to(torch.bfloat16)
        if op == "gate_up":
            if fp8:
                st["x"] = _quant_rows(st["x"].float())
            if own:
                if fp8:
                    st["x"] = efa.Quantized(*st["x"])
                    st["out"] = efa.Quantized(torch.empty(n * m, f, dtype=torch.float8_e4m3fn, device="cuda"),
                                              torch.empty(n * m, -(-f // 128), dtype=torch.uint8, device="cuda"))
                st["h"] = torch.empty(n * m, f, dtype=torch.bfloat16, device="cuda")
    return st


# --------------------------------------------------------------------------- the plain form

def _group(ids, N):
    """count [N], offset [N+1], slot_by_expert [n*m], distinct [N], (U, status)."""
    n, m = ids.shape
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < N)
    key = torch.where(ok, flat, N)
    order = torch.sort(key, stable=True)[1]
    experts = torch.arange(N, device=ids.device)
    count = torch.zeros(N + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))[:N]
    offset = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count, 0)])
    slot = torch.where(torch.arange(n * m, device=ids.device) < offset[N], order, -1)
    distinct = torch.sort(torch.where(count > 0, experts, N))[0]
    distinct = torch.where(distinct < N, distinct, -1)
    row = torch.sort(key.view(n, m), dim=1)[0]
    bad = (~ok).any() | ((row[:, 1:] == row[:, :-1]) & (row[:, 1:] < N)).any()
    status = torch.stack([(count > 0).sum(), torch.where(bad, -5, 0)])
    return tuple(t.to(torch.int32) for t in (count, offset, slot, distinct, status))


def _matrix(w, e):
    return w[e].float() if isinstance(w, torch.Tensor) else _weight_values(w[0][e], w[1][e])


def _gate_up(st, x, group):
    """h in float32, rows in group order."""
    case, W = st["case"], st["weights"]
    at = group[1].tolist()
    h = torch.zeros(case["n"] * case["m"], case["d_ff"], device="cuda")
    for e in range(case["N"]):
        if at[e + 1] > at[e]:
            xe = x[group[2][at[e]:at[e + 1]].long() // case["m"]]
            g, u = xe @ _matrix(W["gate"], e).T, xe @ _matrix(W["up"], e).T
            h[at[e]:at[e + 1]] = g / (1 + torch.exp(-g)) * u
    return h


def _down(st, h, group):
    case, W = st["case"], st["weights"]
    n, m, d = case["n"], case["m"], case["d"]
    at = group[1].tolist()
    o = torch.zeros(n * m, d, device="cuda")
    for e in range(case["N"]):
        if at[e + 1] > at[e]:
            o[group[2][at[e]:at[e + 1]].long()] = h[at[e]:at[e + 1]] @ _matrix(W["down"], e).T
    return (o.view(n, m, d) * st["w"][:, :, None]).sum(dim=1).to(torch.bfloat16)


def run(st):
    case = st["case"]
    op, fp8 = case["op"], case.get("type") == "fp8"
    if own:
        import expert_ffn_amd as efa
        if op == "group":
            return tuple(efa.group_slots(st["ids"], case["N"], out=st["out"], ws=st["ws"]))
        if op == "quant":
            q = efa.quant_rows(st["x"], out=st["out"])
            return {"values": efa.dequant_rows(q, out=st["values"]), "scale": q.scale}
        if op == "gate_up":
            if not fp8:
                return {"h": efa.grouped_gate_up(st["layer"], st["x"], st["group"], out=st["h"])}
            return {"h": efa.dequant_rows(efa.grouped_gate_up(st["layer"], st["x"], st["group"], out=st["out"]), out=st["h"])}
        if op == "down":
            return {"y": efa.grouped_down(st["layer"], st["h"], st["ids"], st["w"], st["group"], y=st["y"], ws=st["ws"])}
        return {"y": efa.expert_grouped(st["layer"], st["x"], st["ids"], st["w"], y=st["y"], ws=st["ws"])}
    if op == "group":
        return _group(st["ids"], case["N"])
    if op == "quant":
        q = _quant_rows(st["x"].float())
        return {"values": _row_values(*q).to(torch.bfloat16), "scale": q[1]}
    group = st["group"] if op != "pass" else _group(st["ids"], case["N"])
    if op == "gate_up":
        if not fp8:
            return {"h": _gate_up(st, st["x"].float(), group).to(torch.bfloat16)}
        return {"h": _row_values(*_quant_rows(_gate_up(st, _row_values(*st["x"]), group))).to(torch.bfloat16)}
    if op == "down":
        return {"y": _down(st, _row_values(*st["h"]) if fp8 else st["h"].float(), group)}
    if not fp8:
        h = _gate_up(st, st["x"].float(), group).to(torch.bfloat16).float()  # h is held in the layer's type
    else:
        h = _gate_up(st, _row_values(*_quant_rows(st["x"].float())), group)
        h = _row_values(*_quant_rows(h))
    return {"y": _down(st, h, group)}


# --------------------------------------------------------------------------- 64 bits, from the definition

def _two_to(k):
    """2^k as float64, exactly: pow may be off by a last place, and half steps are exact here."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_e4m3(v):
    """v (float64, |v| <= 448) to the nearest e4m3 value, ties to even: steps of 2^-3 of the
    power of two below, 2^-9 below 2^-6."""
    step = _two_to((torch.frexp(v)[1] - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quant(v, exponent=False):
    """The values that the blocks of 128 of v's rows (float64) stand for."""
    K = v.shape[1]
    out, ks = torch.empty_like(v), []
    for c in range(0, K, 128):
        b = v[:, c:c + 128]
        f, e = torch.frexp(b.abs().amax(dim=1))  # 448 = 0.875 * 2^9
        k = (e - 9 + (f > 0.875).to(e.dtype)).clamp(min=-127)
        k = torch.where(f == 0, torch.full_like(k, -127), k)
        p = _two_to(k)[:, None]
        out[:, c:c + 128] = _exact_e4m3(b / p) * p
        ks.append(k)
    return (out, torch.stack(ks, dim=1)) if exponent else out


def _exact_matrix(w, e):
    if isinstance(w, torch.Tensor):
        return w[e].double()
    v = w[0][e].float().double()
    p = _two_to(w[1][e].to(torch.int64) - 127)
    for i in range(p.shape[0]):
        v[128 * i:128 * i + 128] *= p[i].repeat_interleave(128)[:v.shape[1]]
    return v


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quant":
        v, k = _exact_quant(st["x"].double(), exponent=True)
        return {"values": v, "scale": k + 127}
    if op == "group":
        ids = st["ids"].cpu().numpy()
        n, m = ids.shape
        N, flat = case["N"], ids.reshape(-1)
        ok = (flat >= 0) & (flat < N)
        slots = np.nonzero(ok)[0]
        count = np.bincount(flat[slots], minlength=N)
        by = np.full(n * m, -1, np.int64)
        by[:slots.size] = slots[np.argsort(flat[slots], kind="stable")]
        present = np.nonzero(count)[0]
        distinct = np.full(N, -1, np.int64)
        distinct[:present.size] = present
        pairs = (slots // m) * N + flat[slots]
        bad = slots.size < n * m or np.unique(pairs).size < slots.size
        return (count, np.concatenate([[0], np.cumsum(count)]), by, distinct, np.array([present.size, -5 if bad else 0]))
    n, m, N, fp8, W = case["n"], case["m"], case["N"], case["type"] == "fp8", st["weights"]
    ids = st["ids"].long()
    if op != "down":
        if op == "pass":
            x = _exact_quant(st["x"].double()) if fp8 else st["x"].double()
        else:
            x = _row_values(*st["x"]).double() if fp8 else st["x"].double()
        hs = torch.zeros(n * m, case["d_ff"], dtype=torch.float64, device="cuda")  # by slot
        for e in range(N):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                z = x[t] @ _exact_matrix(W["gate"], e).T
                hs[t * m + j] = z * torch.sigmoid(z) * (x[t] @ _exact_matrix(W["up"], e).T)
        hs = _exact_quant(hs) if fp8 else hs
        if op == "gate_up":
            return {"h": hs[torch.argsort(ids.reshape(-1), stable=True)]}
        hs = hs if fp8 else hs.to(torch.bfloat16).double()
    else:
        h = _row_values(*st["h"]).double() if fp8 else st["h"].double()
        hs = torch.empty_like(h)
        hs[torch.argsort(ids.reshape(-1), stable=True)] = h
    y = torch.zeros(n, case["d"], dtype=torch.float64, device="cuda")
    for e in range(N):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y.index_add_(0, t, st["w"][t, j].double()[:, None] * (hs[t * m + j] @ _exact_matrix(W["down"], e).T))
    return {"y": y}


# --------------------------------------------------------------------------- work

def work(case):
    op, n = case["op"], case["n"]
    if op == "quant":
        return {"bytes": n * case["d"] * 2 * 2 + n * -(-case["d"] // 128), "flops": 2 * n * case["d"]}
    N, m = case["N"], case["m"]
    if op == "group":
        return {"bytes": 4 * (2 * n * m + 3 * N + 3), "flops": 0}
    d, f = case["d"], case["d_ff"]
    live = n - case.get("pad", 0)
    rows = live * m
    fp8 = case["type"] == "fp8"
    touched = N * (1 - (1 - m / N) ** live)  # experts that some token selects, evenly routed
    per = {"gate_up": 2, "down": 1, "pass": 3}[op] * d * f
    weights = touched * per * (1 + 1 / 16384 if fp8 else 2)
    a = 1 + 1 / 128 if fp8 else 2  # bytes of an activation
    moved = {"gate_up": n * d * a + rows * f * 2, "down": rows * f * a + n * d * 2 + rows * 8,
             "pass": n * d * 4 + n * m * 8}[op]
    return {"bytes": weights + moved, "flops": 2 * rows * per}
