"""The grouped calls on square tiles, whose rule every test here asks for: what the tests of
``test_gpu_grouped`` with narrow layers ask of thin tiles, the most experts, and the shapes
of the timed layers.  Tolerances are those that ``test_gpu_grouped`` derives."""
import pytest
import torch

import expert_ffn_amd as efa
from expert_ffn_amd import _abi

from .gpu_cases import say
from .test_gpu_grouped import (
    BF, H8, Case, _cancelling, _check_h, _check_pass, _down_case, _exact_sum, _gpu_layer, _ids, _pow2, _randn,
    _row_values, _run_parts, _weight_values, _within,
)

pytestmark = pytest.mark.gpu

BOTH = [(t, s) for t in ("bf16", "fp8") for s in ("plain", "tiled")]


def _tiles(layer, n):
    return tuple(efa.grouped_square(layer, n, m) for m in (_abi.MOE_MAT_GATE_UP, _abi.MOE_MAT_DOWN))


def _square_case(N, m, d, f, typ, layout, n, seed=1):
    say("square", N, m, d, f, typ, layout, n)
    case = Case(N, m, d, f, typ, layout, seed=seed)
    assert _tiles(case.layer, n) == (True, True)
    return case


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("N,m,n", [(1000, 3, 4200), (1024, 2, 6200)])
def test_square_tiles_of_the_most_experts(N, m, n, typ):
    """Sixteen experts a lane, many of them without a row."""
    case = _square_case(N, m, 512, 528, typ, "plain", n, seed=4)
    ids, w = _ids(5, n, m, N, zipf=0.7, pad=11)
    _check_pass(case, _randn(6, n, 512).to(BF).cuda(), ids, w, "most experts")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_no_valid_id(typ, layout):
    """No tile at all: y zeros, or unchanged when accumulating; h left as it was."""
    n = 900
    case = _square_case(8, 2, 512, 576, typ, layout, n)
    x = _randn(1, n, 512).to(BF).cuda()
    ids = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.full((n, 2), float("nan"), device="cuda")
    info = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert (efa.expert_grouped(case.layer, x, ids, w, info=info) == 0).all() and info.tolist() == [0, -5, 0]
    y = _randn(2, n, 512).to(BF).cuda()
    was = y.clone()
    efa.expert_grouped(case.layer, x, ids, w, y=y, accumulate=True)
    assert torch.equal(y, was)
    h = _marked_h(typ, n * 2, 576)
    case.gate_up(x, ids, out=h)
    _assert_marked(h, 0)


def _marked_h(typ, S, f):
    if typ == "bf16":
        return torch.full((S, f), 7.0, dtype=BF, device="cuda")
    return efa.Quantized(torch.full((S, f), 5.0, device="cuda").to(H8),
                         torch.full((S, -(-f // 128)), 9, dtype=torch.uint8, device="cuda"))


def _assert_marked(h, rows):
    if isinstance(h, torch.Tensor):
        assert (h[rows:] == 7).all()
    else:
        assert (h.q[rows:].float() == 5).all() and (h.scale[rows:] == 9).all()


@pytest.mark.parametrize("typ,layout", BOTH)
@pytest.mark.parametrize("pad", [1, 333])
def test_rows_behind_the_last_group_are_left(pad, typ, layout):
    n, f = 1000, 704
    case = _square_case(8, 2, 512, f, typ, layout, n)
    x = _randn(1, n, 512).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8, pad=pad)
    g, h = case.gate_up(x, ids, out=_marked_h(typ, n * 2, f))
    rows = int(g.offset[-1])
    assert rows == (n - pad) * 2
    _assert_marked(h, rows)
    _check_h(case, h, x, g, "h")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_nan_stays_in_its_token(typ, layout):
    n = 700
    case = _square_case(8, 2, 512, 640, typ, layout, n)
    x = _randn(1, n, 512).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8)
    clean = efa.expert_grouped(case.layer, x, ids, w)
    keep = torch.arange(n, device="cuda") != n // 2
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[n // 2, 17] = bad
        y = efa.expert_grouped(case.layer, xb, ids, w)
        assert y[n // 2].isnan().any()
        assert torch.equal(y[keep], clean[keep])


def _fp8_layer(case, layout, **codes):
    """The plain layer with some codes replaced: name -> (expert, row, code byte)."""
    mats = {}
    for name in ("gate", "up", "down"):
        q, s = getattr(case.layer, name)
        if name in codes:
            e, r, c = codes[name]
            q = q.clone()
            q.view(torch.uint8)[e, r] = c
        mats[name] = (q, s)
    layer = efa.Fp8Layer(mats["gate"], mats["up"], mats["down"], m=case.m)
    return layer.tiled_copy() if layout == "tiled" else layer


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("n,square", [(9, False), (700, True)])
def test_a_column_of_nan_leaves_its_block_as_it_is(n, square, layout):
    """An h that is not finite takes no part in its block's maximum: every other code and
    every scale byte are those of a layer where that column of h is zero."""
    say("column of nan", n, layout)
    N, f, e, c = 8, 640, 3, 200
    case = Case(N, 2, 512, f, "fp8", "plain")
    zero, nan = (_fp8_layer(case, layout, gate=(e, c, v)) for v in (0, 0x7f))
    assert _tiles(nan, n) == (square, square)
    x = efa.quant_rows(_randn(1, n, 512).to(BF).cuda())
    ids, w = _ids(2, n, 2, N)
    ids[0, 0], ids[0, 1] = e, (e + 1) % N  # one row of it at least
    g = efa.group_slots(ids, N)
    a, b = (efa.grouped_gate_up(layer, x, g) for layer in (zero, nan))
    at = g.offset.tolist()
    rows = torch.zeros(n * 2, dtype=torch.bool, device="cuda")
    rows[at[e]:at[e + 1]] = True
    assert rows.any() and not rows.all()
    hit = torch.zeros(n * 2, f, dtype=torch.bool, device="cuda")
    hit[rows, c] = True
    qa, qb = a.q.view(torch.uint8), b.q.view(torch.uint8)
    assert torch.equal(a.scale, b.scale)
    assert torch.equal(qa[~hit], qb[~hit])
    assert (qa[hit] & 0x7f == 0).all() and (qb[hit] & 0x7f == 0x7f).all()


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("n,square", [(9, False), (700, True)])
def test_h_that_overflows(n, square, layout):
    """x of about 2^120: h is infinite where the gate is positive (NaN codes) and zero where
    it is negative, which leaves a block's power of two at its least."""
    say("overflow", n, layout)
    N, d, f = 8, 512, 640
    case = Case(N, 2, d, f, "fp8", layout)
    assert _tiles(case.layer, n) == (square, square)
    x = _randn(1, n, d).to(BF).cuda()
    t = n // 2
    x[t] *= 2.0 ** 110
    xq = efa.quant_rows(x)
    ids, w = _ids(2, n, 2, N)
    g, h = case.gate_up(x, ids)
    ref, tol = case.exact_h(case.x_values(torch.where(torch.arange(n, device="cuda")[:, None] == t, x * 0, x)), g)
    for r in torch.nonzero(g.slot_by_expert // 2 == t)[:, 0].tolist():
        e = int(ids.reshape(-1)[g.slot_by_expert[r]])
        xv = _row_values(xq)[t]
        gate, up = case.W[0][e] @ xv, case.W[1][e] @ xv
        # far from zero by every sum's error (less than 2^-9 of the magnitudes), the product beyond fp32
        mag = (case.W[0][e].abs() @ xv.abs()).minimum(case.W[1][e].abs() @ xv.abs())
        clear = (gate.abs() > 2.0 ** -8 * mag) & (up.abs() > 2.0 ** -8 * mag)
        assert clear.float().mean() > 0.8 and (gate[clear].abs() * up[clear].abs()).log2().min() > 130
        code = h.q.view(torch.uint8)[r] & 0x7f
        assert (code[clear & (gate > 0)] == 0x7f).all()
        assert (code[clear & (gate < 0)] == 0).all()
        assert (h.scale[r] == 0).all()  # (no sum is within 2^90 of zero but by chance of 2^-20)
    others = (g.slot_by_expert // 2 != t) & (torch.arange(2 * n, device="cuda") < g.offset[-1])
    v = _row_values(h)[others]
    step = _pow2(h.scale[others].long() - 127).repeat_interleave(128, dim=1)[:, :f]
    bound = tol[others] + torch.maximum(2.0 ** -4 * (ref.abs() + tol)[others], 2.0 ** -10 * step)
    _within(v, ref[others], bound, "other rows")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_layouts_and_repeats(typ, layout):
    """Skewed groups against the formulas; the same bits from call to call."""
    n = 800
    case = _square_case(8, 2, 512, 704, typ, layout, n)
    x = _randn(1, n, 512).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8, zipf=1.0)
    y = _check_pass(case, x, ids, w, layout)
    for _ in range(4):
        assert torch.equal(efa.expert_grouped(case.layer, x, ids, w), y)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_many_slots_a_token(typ):
    n, N, m = 400, 160, 130
    case = _square_case(N, m, 512, 464, typ, "plain", n, seed=n)
    ids, w = _ids(5, n, m, N)
    ids[n // 2, 1:129] = -1
    ids[0, :64] = N
    _check_pass(case, _randn(6, n, 512).to(BF).cuda(), ids, w, "many slots")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_repeated_and_out_of_range_ids(typ, layout):
    n = 300
    case = _square_case(8, 4, 512, 448, typ, layout, n)
    ids, w = _ids(2, n, 4, 8)
    ids[3] = ids[3, 0]
    ids[5, 1], ids[6, 2], ids[7, 3] = 8, -2147483648, 2147483647
    _check_pass(case, _randn(1, n, 512).to(BF).cuda(), ids, w, "ids")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_accumulate_and_always_on_experts(typ, layout):
    n = 640
    case, shared = (_square_case(N, 2, 512, f, typ, layout, n, seed=s) for N, f, s in ((8, 512, 1), (2, 448, 20)))
    x = _randn(1, n, 512).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8)
    y = efa.expert_grouped(case.layer, x, ids, w)
    routed = y.double()
    sids = torch.arange(2, dtype=torch.int32, device="cuda").repeat(n, 1).contiguous()
    ones = torch.ones(n, 2, device="cuda")
    assert efa.expert_grouped(shared.layer, x, sids, ones, y=y, accumulate=True) is y
    g, h = shared.gate_up(x, sids)
    want, tol = shared.exact_y(_check_h(shared, h, x, g, "h"), sids, ones, g)
    _within(y, routed + want, tol + 2.0 ** -8 * (routed + want).abs() + 2.0 ** -8 * tol, "accumulated")


@pytest.mark.parametrize("typ,layout", BOTH)
def test_captured_and_replayed(typ, layout):
    """Two graphs that share a workspace, and the parts as a third, replayed with eager passes
    of other lengths (thin and square) on the same workspace between."""
    n, d = 500, 512
    case = _square_case(8, 2, d, 576, typ, layout, n)
    ws = case.layer.grouped_workspace(n)
    x = _randn(1, n, d).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8, pad=n // 4)
    w = w.nan_to_num()
    graphs, outs = [], []
    for k in range(3):
        y = torch.empty(n, d, dtype=BF, device="cuda")

        def call():
            if k < 2:
                return efa.expert_grouped(case.layer, x, ids, w, y=y, ws=ws)
            return _run_parts(case.layer, x, ids, w, typ == "fp8")[2]
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for i in range(4):
        x.copy_(_randn(30 + i, n, d).to(BF))
        ids.copy_(_ids(40 + i, n, 2, 8, pad=17 * i)[0])
        want = efa.expert_grouped(case.layer, x, ids, w)
        for k in (5, 200):
            efa.expert_grouped(case.layer, x[:k], ids[:k], w[:k], ws=ws)
        for graph, y in zip(graphs, outs):
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_side_streams(typ):
    n = 900
    case = _square_case(8, 2, 512, 512, typ, "tiled", n)
    xs = [_randn(i, n, 512).to(BF).cuda() for i in range(2)]
    ids, w = _ids(2, n, 2, 8)
    want = [efa.expert_grouped(case.layer, x, ids, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[efa.expert_grouped(case.layer, xs[i], ids, w, stream=streams[i]) for i in range(2)] for _ in range(5)]
    torch.cuda.synchronize()
    for ys in got:
        assert all(torch.equal(y, v) for y, v in zip(ys, want))


# --- the terms of a token's sum: 11 bits, a power of two for each 64 columns ----------------

TERM = dict(rounding=2.0 ** -11, block=2.0 ** -39)  # half a step; half of fp16's least step against 2^14


@pytest.mark.parametrize("typ,layout", BOTH)
@pytest.mark.parametrize("N,m,n,d", [(8, 2, 400, 512), (16, 8, 300, 528), (64, 4, 500, 80)])
def test_terms_that_cancel(N, m, n, d, typ, layout):
    """Terms that leave little of their sum are off by their own roundings and no more."""
    if layout == "tiled":
        d = -(-d // 64) * 64
    say("cancel", N, m, n, d, typ, layout)
    case = _down_case(N, m, d, 768, typ, layout, seed=n)
    assert efa.grouped_square(case.layer, n, _abi.MOE_MAT_DOWN)
    ids, w, g, h, hv = _cancelling(case, n, 80 + n)
    y = efa.grouped_down(case.layer, h, ids, w, g)
    want, tol = _exact_sum(case, hv, ids, w, g, case.eps(768), **TERM)
    _within(y, want, tol, "y")


def _random_down(W, m, n, seed, fp8):
    """A layer with this bf16 W_down [N][d][f] (any gate and up), and h, ids and w for it."""
    N, d, f = W.shape
    gate = torch.zeros(N, f, d, dtype=BF, device="cuda")
    layer = efa.Layer(gate, gate, W, m=m)
    layer = layer.fp8_copy() if fp8 else layer
    ids, w = _ids(seed, n, m, N)
    g = efa.group_slots(ids, N)
    h = _randn(seed + 1, n * m, f).to(BF).cuda()
    h = efa.quant_rows(h) if fp8 else h
    assert efa.grouped_square(layer, n, _abi.MOE_MAT_DOWN)
    return layer, h, ids, w, g


@pytest.mark.parametrize("power", [-118, -40, 0, 40, 110])
@pytest.mark.parametrize("typ,spread", [("bf16", 0), ("bf16", 24), ("fp8", 0), ("fp8", 5)])
def test_terms_of_every_magnitude(typ, spread, power):
    """Columns of y up to 2^24 apart side by side, terms of 2^-118 to 2^110: each column to
    its own precision."""
    say("magnitudes", typ, spread, power)
    N, m, d, f, n = 4, 2, 336, 512, 300
    scale = torch.randint(-spread, 1, (1, d, 1), generator=torch.Generator().manual_seed(1))
    W = (_randn(2, N, d, f) * _pow2(scale + power)).to(BF).cuda()
    layer, h, ids, w, g = _random_down(W, m, n, 3, typ == "fp8")
    case = Case.__new__(Case)
    case.N, case.m, case.d, case.f, case.fp8 = N, m, d, f, typ == "fp8"
    case.W = [None, None, _weight_values(*layer.down) if case.fp8 else W.double()]
    y = efa.grouped_down(layer, h, ids, w, g)
    want, tol = _exact_sum(case, _row_values(h) if case.fp8 else h.double(), ids, w, g, case.eps(f), **TERM)
    _within(y, want, tol + 2.0 ** -134, "y")  # (bf16's least step is 2^-133)


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_column_that_is_not_finite(bad, layout):
    """A NaN or an infinity in one row of an expert's W_down reaches that column of the tokens
    that use the expert; every other value has the bits of a layer where that row is zero."""
    N, m, d, f, n, e, c = 8, 2, 576, 512, 600, 3, 130
    W = (_randn(2, N, d, f) * 0.05).to(BF).cuda()
    W[e, c] = 0
    layer, h, ids, w, g = _random_down(W, m, n, 3, False)
    h[:, 7] = 1.0
    Wb = W.clone()
    Wb[e, c, 7] = bad
    other = efa.Layer(layer.w_gate, layer.w_up, Wb, m=m)
    layer, other = (v.tiled_copy() if layout == "tiled" else v for v in (layer, other))
    a, b = (efa.grouped_down(v, h, ids, w, g) for v in (layer, other))
    hit = torch.zeros(n, d, dtype=torch.bool, device="cuda")
    hit[(ids == e).any(1), c] = True
    assert hit.any() and torch.isfinite(a).all() and torch.equal(a[~hit], b[~hit])
    assert (b[hit].isnan() if bad != bad else b[hit] == bad).all()


class _GpuCase(Case):
    """A Case with weights made on the GPU."""

    def __init__(self, N, m, d, f, typ, layout):
        self.N, self.m, self.d, self.f, self.fp8 = N, m, d, f, typ == "fp8"
        plain, self.layer = _gpu_layer(N, m, d, f, typ, layout, 1)
        self.W = ([_weight_values(*p) for p in (plain.gate, plain.up, plain.down)] if self.fp8 else
                  [v.double() for v in (plain.w_gate, plain.w_up, plain.w_down)])


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("N,m,d,f", [(128, 8, 2048, 768), (64, 6, 2048, 1408), (8, 2, 4096, 14336)])
def test_layers_of_the_timed_shapes(N, m, d, f, typ):
    say("shapes", N, m, d, f, typ)
    case = _GpuCase(N, m, d, f, typ, "tiled")
    for n, square in ((1, False), (5, False), (513, True)):
        assert _tiles(case.layer, n) == (square, square)
        ids, w = _ids(3, n, m, N, zipf=1.1, pad=n // 10)
        _check_pass(case, _randn(4, n, d).to(BF).cuda(), ids, w, "n = %d" % n)
