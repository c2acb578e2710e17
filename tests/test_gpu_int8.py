"""The expert operation in 8-bit integers (a scale for each token and output channel) on the
GPU: the row quantisation bit for bit, the grouped products and passes against their
formulas in 64 bits.

Tolerances, per value.  Sums of codes are whole numbers below 2^31, exact in int32; a sum
becomes fp32, times the token's scale, times the channel's: three roundings, 2^-22 |g| with
room.  silu(g) * u: 1.1 |u| dg + |silu(g)| du + 2^-20 |h| (|silu'| < 1.1; the exponential and
the division are good to a few 2^-23), then 2^-8 |h| to bf16, then half a step of the
row's scale.  y sums m terms w O: each is off by 2^-22 |w O|, and behind square tiles by
another 2^-11 |w O| and 2^-39 of its 64 columns' largest; m additions 2^-23 of the magnitudes
each; then 2^-8 |y| to bf16.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import expert_ffn_amd as efa
from expert_ffn_amd import _abi

from .gpu_cases import say

pytestmark = pytest.mark.gpu

BF, I8, F32 = torch.bfloat16, torch.int8, torch.float32


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _ids(seed, n, m, N, zipf=0.0, pad=0):
    logits = _randn(seed, n, N) - zipf * torch.log(torch.arange(N) + 1.0)
    top, ids = logits.topk(m, dim=1)
    ids, w = ids.to(torch.int32), top.softmax(1)
    if pad:
        ids[n - pad:] = -1
        w[n - pad:] = float("nan")  # the weight of no expert is not read
    return ids.cuda().contiguous(), w.cuda().contiguous()


def _codes(v):
    """(codes, scales) of rows of finite float64 values that bf16 holds, ties to even, exactly: |254 v| +
    max and 2 max k hold few enough bits for values within 2^20 of the row's largest; what is smaller is 0."""
    a = v.abs().amax(1, keepdim=True)
    one = torch.where(a > 0, a, torch.ones_like(a))
    top = 254 * v.abs() + one
    k = torch.floor(top / (2 * one))
    k = torch.where((top == 2 * one * k) & (k % 2 == 1), k - 1, k)
    return (torch.sign(v) * k).to(I8), (a[:, 0] / 127).to(F32)


def _values(q, s):
    return q.double() * s.double()[..., None]


class Case:
    def __init__(self, N, m, d, f, layout="plain", seed=1, scale=0.05):
        self.N, self.m, self.d, self.f = N, m, d, f
        W = [(_randn(seed + i, N, *s) * scale).to(BF).cuda() for i, s in enumerate(((f, d), (f, d), (d, f)))]
        layer = efa.Layer(*W, m=m).int8_copy()
        self.W = [(q.double(), s.double()) for q, s in (layer.gate, layer.up, layer.down)]
        self.layer = layer.tiled_copy() if layout == "tiled" else layer

    def product(self, i, e, q, s):
        """Matrix i of expert e times rows: sums of codes in whole numbers (exact in float64, so that a sum of
        zero is zero), then the scales."""
        return (q.double() @ self.W[i][0][e].T) * s.double()[:, None] * self.W[i][1][e][None, :]

    def square(self, n, mat):
        return efa.grouped_square(self.layer, n, mat)

    def gate_up(self, x, ids, out=None, ws=None):
        g = efa.group_slots(ids, self.N)
        return g, efa.grouped_gate_up(self.layer, efa.quant_rows(x, dtype=I8), g, out=out, ws=ws)

    def exact_h(self, xq, xs, g):
        at, slot = g.offset.tolist(), g.slot_by_expert.long()
        h = torch.zeros(slot.numel(), self.f, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(h)
        for e in range(self.N):
            r = slice(at[e], at[e + 1])
            if at[e] == at[e + 1]:
                continue
            t = slot[r] // self.m
            a, b = self.product(0, e, xq[t], xs[t]), self.product(1, e, xq[t], xs[t])
            s = a * torch.sigmoid(a)
            h[r] = s * b
            tol[r] = 2.0 ** -22 * (1.1 * (b * a).abs() + (s * b).abs()) + 2.0 ** -20 * h[r].abs() + 1e-40
        return h, tol

    def check_h(self, h, x, g, what):
        want, tol = self.exact_h(*_codes(x.double()), g)
        rows = int(g.offset[-1])
        want, tol = want[:rows], tol[:rows]
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
        q, s = h.q[:rows], h.scale[:rows].double()
        assert torch.isfinite(s).all() and (q != -128).all(), what
        most, off = want.abs().amax(1), tol.amax(1)
        assert ((127 * s - most).abs() <= off + 2.0 ** -23 * most + 1e-40).all(), what
        assert (q.abs().amax(1)[s > 0] == 127).all(), what
        over = (_values(q, s) - want).abs() - tol - 0.5 * s[:, None] * (1 + 2.0 ** -20)
        assert (over <= 1e-40).all(), "%s: %.3g over at %s" % (what, over.max(), np.unravel_index(int(over.argmax()), over.shape))

    def exact_y(self, h, ids, w, g):
        n, at, slot = ids.shape[0], g.offset.tolist(), g.slot_by_expert.long()
        y = torch.zeros(n, self.d, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(y)
        square = self.square(n, efa.MOE_MAT_DOWN)
        for e in range(self.N):
            if at[e] == at[e + 1]:
                continue
            r = slice(at[e], at[e + 1])
            s = slot[r]
            o = self.product(2, e, h.q[r], h.scale[r])
            wt = w.reshape(-1)[s].double()[:, None]
            y.index_add_(0, s // self.m, wt * o)
            do = (2.0 ** -22 + self.m * 2.0 ** -22) * o.abs()
            if square:
                pad = torch.nn.functional.pad(o.abs(), (0, -self.d % 64)).view(o.shape[0], -1, 64).amax(2)
                do = do + 2.0 ** -11 * o.abs() + 2.0 ** -39 * pad.repeat_interleave(64, 1)[:, :self.d]
            tol.index_add_(0, s // self.m, wt.abs() * do)
        return y, tol + 2.0 ** -8 * (y.abs() + tol) + 1e-40


def _within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert (over <= 0).all(), "%s: %.3g over at %s" % (what, over.max(), np.unravel_index(int(over.argmax()), over.shape))


def _check_pass(case, x, ids, w, what):
    """The parts against their formulas, and the whole pass against the parts, bit for bit."""
    g, h = case.gate_up(x, ids)
    case.check_h(h, x, g, what + " h")
    y = efa.grouped_down(case.layer, h, ids, w, g)
    want, tol = case.exact_y(h, ids, w, g)
    _within(y, want, tol, what + " y")
    info = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    ws = case.layer.grouped_workspace(ids.shape[0])
    ws.fill_(255)  # whatever a workspace holds (NaN, -1) is not read
    whole = efa.expert_grouped(case.layer, x, ids, w, ws=ws, info=info)
    assert torch.equal(whole, y), what
    assert info[:2].tolist() == g.u_and_err.tolist() and int(info[2]) == 0
    return y


# --- rows -------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (130, 128), (1, 512), (5, 528), (129, 1408), (7, 2048), (6, 2064),
                                    (3, 8192), (2, 8208), (2, 16400), (1, 65536), (4099, 32)])
def test_rows_bit_for_bit(rows, K):
    say("int8 rows", rows, K)
    x = (_randn(rows + K, rows, K) * torch.exp(_randn(7, 1, K))).to(BF).cuda()
    got = efa.quant_rows(x, dtype=I8)
    q, s = _codes(x.double())
    assert torch.equal(got.q, q) and torch.equal(got.scale, s)
    back = efa.dequant_rows(got)
    assert torch.equal(back, (q.float() * s[:, None]).to(BF))


def test_rows_at_halves_and_at_the_ends_of_the_range():
    """Every bf16 significand as a row's maximum against every other at six exponents, by whole numbers."""
    say("int8 halves")
    sig = torch.arange(128, 256).double()
    vals = torch.cat([sig * 2.0 ** -p for p in range(6)] + [torch.zeros(16).double()])
    rows = torch.cat([sig[:, None], vals.repeat(128, 1)], 1)
    rows = torch.where(rows > sig[:, None], torch.zeros_like(rows), rows)
    rows = torch.nn.functional.pad(rows, (0, -rows.shape[1] % 16))
    sign = torch.where(torch.arange(rows.shape[1]) % 3 == 1, -1.0, 1.0)
    want = np.array([[int(round(Fraction(127 * int(v * 32), int(a * 32)))) for v in r] for r, a in zip(rows.tolist(), sig.tolist())])
    for scale in (1.0, 2.0 ** -120, 2.0 ** -133, 2.0 ** 120):  # to subnormal values, which lose bits, and near the largest
        x = (rows * sign * scale).to(BF)
        got = efa.quant_rows(x.cuda(), dtype=I8)
        if scale > 2.0 ** -121:
            assert np.array_equal(got.q.cpu().numpy(), want * sign.int().numpy()), scale
        q, s = _codes(x.double())
        assert torch.equal(got.q.cpu(), q) and torch.equal(got.scale.cpu(), s), scale


def test_rows_of_zeros_and_not_finite():
    say("int8 odd rows")
    for K in (32, 2048, 4096, 40960):
        x = _randn(3, 6, K).to(BF)
        x[1] = 0
        x[2, K - 1] = float("inf")
        x[3, 5] = float("nan")
        x[4, 0] = float("-inf")
        got = efa.quant_rows(x.cuda(), dtype=I8)
        q, s = got.q.cpu(), got.scale.cpu()
        assert (q[1] == 0).all() and s[1] == 0
        assert (q[2:5] == 0).all() and torch.isnan(s[2:5]).all()
        wq, ws = _codes(x[[0, 5]].double())
        assert torch.equal(q[[0, 5]], wq) and torch.equal(s[[0, 5]], ws)
        back = efa.dequant_rows(got).cpu()
        assert torch.isnan(back[2:5]).all() and (back[1] == 0).all()


def test_weights_are_rows():
    w = (_randn(5, 3, 48, 80) * 0.1).to(BF).cuda()
    q, s = efa.quant_weights(w, dtype=I8)
    r = efa.quant_rows(w.view(-1, 80), dtype=I8)
    assert torch.equal(q.view(-1, 80), r.q) and torch.equal(s.view(-1), r.scale)


# --- products and passes ----------------------------------------------------------------

SHAPES = [  # N, m, d, f
    (1, 1, 16, 16), (3, 2, 48, 80), (5, 5, 144, 176), (8, 2, 64, 128), (16, 4, 192, 64), (7, 3, 320, 1040),
    (128, 8, 256, 192), (40, 4, 2048, 768)]


@pytest.mark.parametrize("N,m,d,f", SHAPES)
@pytest.mark.parametrize("n", [1, 2, 5, 17, 33, 130])
def test_pass(N, m, d, f, n):
    say("int8 pass", N, m, d, f, n)
    case = Case(N, m, d, f, layout="tiled" if d % 64 == 0 and f % 64 == 0 and n % 2 else "plain", seed=n)
    x = (_randn(n, n, d) * torch.exp(_randn(3, 1, d))).to(BF).cuda()
    ids, w = _ids(n + 1, n, m, N, zipf=0.7, pad=n // 4)
    y = _check_pass(case, x, ids, w, "pass %s" % ((N, m, d, f, n),))
    if n // 4:
        assert (y[n - n // 4:] == 0).all()


@pytest.mark.parametrize("N,m,d,f,n", [
    (8, 1, 3440, 32, 16), (8, 1, 3456, 32, 16), (2, 1, 64, 18416, 3), (2, 1, 64, 18432, 3), (4, 2, 128, 192, 32),
    (4, 2, 128, 192, 33), (64, 8, 256, 192, 8), (1024, 4, 64, 48, 16), (4, 1, 16400, 32, 70), (2, 1, 32, 65536, 2),
    (2, 1, 32, 65536, 70), (3, 1, 65536, 32, 70)])
def test_where_the_form_of_a_pass_changes(N, m, d, f, n):
    """Passes of 64 slots and one more, codes that just fit shared memory and just do not, rows of many rounds."""
    say("int8 pass", N, m, d, f, n)
    case = Case(N, m, d, f, layout="tiled" if d % 64 == 0 and f % 64 == 0 else "plain")
    ids, w = _ids(n, n, m, N)
    _check_pass(case, _randn(n, n, d).to(BF).cuda(), ids, w, "pass %s" % ((N, m, d, f, n),))


@pytest.mark.parametrize("counts", [[300, 0, 1, 257, 64, 0, 192, 33], [1200, 0, 1, 1030, 300, 64, 897, 257],
                                    [0, 0, 4000, 0, 0, 0, 0, 0]])
@pytest.mark.parametrize("layout", ["plain", "tiled"])
def test_many_rows(counts, layout):
    say("int8 many rows", counts, layout)
    N, d, f = len(counts), 576, 640
    ids = torch.repeat_interleave(torch.arange(N), torch.tensor(counts))
    n = ids.numel()
    ids = ids[torch.randperm(n, generator=torch.Generator().manual_seed(4))].to(torch.int32)[:, None].cuda().contiguous()
    case = Case(N, 1, d, f, layout=layout)
    assert case.square(n, efa.MOE_MAT_GATE_UP) == case.square(n, efa.MOE_MAT_DOWN) == (n > 1000)
    _check_pass(case, _randn(9, n, d).to(BF).cuda(), ids, _randn(2, n, 1).cuda(), "rows")


def test_square_tiles_of_odd_sizes():
    """Contractions of a few units and part of one, columns that end inside a tile, skewed rows, several slots a token."""
    say("int8 square odd sizes")
    for N, m, d, f, n, layout in ((6, 3, 400, 1040, 3000, "plain"), (12, 5, 1104, 432, 2100, "plain"),
                                  (5, 2, 448, 3200, 1500, "tiled"), (24, 8, 2064, 1008, 300, "plain")):
        case = Case(N, m, d, f, layout=layout, seed=N)
        x = (_randn(n, n, d) * torch.exp(_randn(3, 1, d))).to(BF).cuda()
        ids, w = _ids(n + 1, n, m, N, zipf=1.0, pad=n // 10)
        assert case.square(n, efa.MOE_MAT_GATE_UP) and case.square(n, efa.MOE_MAT_DOWN)
        _check_pass(case, x, ids, w, "square %s" % ((N, m, d, f, n),))


@pytest.mark.parametrize("n,f,square", [(3, 16, False), (300, 16, False), (4000, 256, True)])
def test_largest_codes_do_not_overflow(n, f, square):
    """Every code 127 over the longest contraction: sums of 65536 * 127^2, above 2^24 by far."""
    say("int8 longest", n)
    N, d = 2, 65536
    q = torch.full((N, f, d), 127, dtype=I8, device="cuda")
    s = torch.full((N, f), 2.0 ** -20, device="cuda")
    dn = (torch.full((N, d, f), -127, dtype=I8, device="cuda"), torch.full((N, d), 2.0 ** -7, device="cuda"))
    layer = efa.Int8Layer((q, s), (q, s), dn, m=1)
    assert efa.grouped_square(layer, n, efa.MOE_MAT_GATE_UP) == square
    x = torch.full((n, d), 127.0, dtype=BF, device="cuda")
    ids = (torch.arange(n, dtype=torch.int32, device="cuda") % 2)[:, None].contiguous()
    g = efa.group_slots(ids, N)
    h = efa.grouped_gate_up(layer, efa.quant_rows(x, dtype=I8), g)
    z = 65536.0 * 127 * 127 * 2.0 ** -20
    want = z / (1 + np.exp(-z)) * z
    assert (h.q == 127).all()
    assert ((h.scale.double() * 127 - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want).all()
    y = efa.grouped_down(layer, h, ids, torch.ones(n, 1, device="cuda"), g)
    o = -float(f) * 127 * 127 * 2.0 ** -7 * h.scale.double()[:, None].expand(n, d)
    o = o[torch.argsort(g.slot_by_expert.long())]
    assert ((y.double() - o).abs() <= (2.0 ** -8 + 2.0 ** -10) * o.abs()).all()


def test_rows_that_are_not_finite_stay_their_own():
    say("int8 nan rows")
    for n in (6, 400, 2500):
        case = Case(4, 2, 576, 640)
        assert case.square(n, efa.MOE_MAT_DOWN) == (n == 2500)
        x = _randn(1, n, 576).to(BF).cuda()
        ids, w = _ids(2, n, 2, 4)
        want = efa.expert_grouped(case.layer, x, ids, w)
        x[3, 7] = float("nan")
        x[5, 0] = float("inf")
        y = efa.expert_grouped(case.layer, x, ids, w)
        assert torch.isnan(y[[3, 5]]).all()
        keep = [t for t in range(n) if t not in (3, 5)]
        assert torch.equal(y[keep], want[keep])


def test_a_channel_that_is_not_finite():
    W = [(_randn(i, 3, *s) * 0.05).to(BF) for i, s in enumerate(((96, 64), (96, 64), (64, 96)))]
    W[2][1, 10, 3] = float("inf")
    layer = efa.Layer(*(w.cuda() for w in W), m=1).int8_copy()
    ids = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    y = efa.expert_grouped(layer, _randn(5, 3, 64).to(BF).cuda(), ids, torch.ones(3, 1, device="cuda"))
    bad = torch.isnan(y).cpu()
    assert bad[1, 10] and int(bad.sum()) == 1


def test_no_valid_id_and_ids_twice():
    case = Case(6, 3, 128, 192)
    x = _randn(1, 4, 128).to(BF).cuda()
    y = efa.expert_grouped(case.layer, x, torch.full((4, 3), 9, dtype=torch.int32, device="cuda"),
                           torch.full((4, 3), float("nan"), device="cuda"))
    assert (y == 0).all()
    ids = torch.tensor([[1, 1, 1], [0, 5, 0], [2, -1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda")
    _check_pass(case, x, ids, torch.rand(4, 3, device="cuda"), "ids twice")


@pytest.mark.parametrize("n", [9, 600, 2500])
def test_accumulate_and_rows_behind_the_last(n):
    say("int8 accumulate", n)
    case = Case(8, 2, 576, 640)
    x = _randn(1, n, 576).to(BF).cuda()
    ids, w = _ids(3, n, 2, 8, pad=n // 3)
    g, h = case.gate_up(x, ids)
    rows = int(g.offset[-1])
    out = efa.Quantized(torch.full_like(h.q, 77), torch.full_like(h.scale, 5.0))
    case.gate_up(x, ids, out=out)
    assert torch.equal(out.q[:rows], h.q[:rows]) and torch.equal(out.scale[:rows], h.scale[:rows])
    assert (out.q[rows:] == 77).all() and (out.scale[rows:] == 5.0).all()
    y0 = _randn(8, n, 576).to(BF).cuda()
    y = efa.grouped_down(case.layer, h, ids, w, g, y=y0.clone(), accumulate=True)
    want, tol = case.exact_y(h, ids, w, g)
    _within(y, want + y0.double(), tol + 2.0 ** -8 * y0.double().abs(), "accumulate")
    assert torch.equal(efa.expert_grouped(case.layer, x, ids, w, y=y0.clone(), accumulate=True), y)
    assert torch.equal(y[n - n // 3:], y0[n - n // 3:])


def test_a_layer_of_always_on_experts():
    case = Case(2, 2, 128, 192)
    x = _randn(1, 21, 128).to(BF).cuda()
    ids = torch.arange(2, dtype=torch.int32, device="cuda").repeat(21, 1).contiguous()
    _check_pass(case, x, ids, torch.ones(21, 2, device="cuda"), "always on")


def test_other_stream_and_captured():
    say("int8 streams and graphs")
    case = Case(16, 4, 576, 640, layout="plain")
    for n in (7, 300, 1200):
        x = _randn(1, n, 576).to(BF).cuda()
        ids, w = _ids(3, n, 4, 16)
        want = efa.expert_grouped(case.layer, x, ids, w)
        q = efa.quant_rows(x, dtype=I8)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        y = efa.expert_grouped(case.layer, x, ids, w, stream=st)
        q2 = efa.quant_rows(x, dtype=I8, stream=st)
        back = efa.dequant_rows(q2, stream=st)
        st.synchronize()
        assert torch.equal(y, want) and torch.equal(q.q, q2.q) and torch.equal(back, efa.dequant_rows(q))
        ws, y = case.layer.grouped_workspace(n), torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            efa.expert_grouped(case.layer, x, ids, w, y=y, ws=ws)
        for seed in range(3):
            x.copy_(_randn(seed + 20, n, 576).to(BF))
            i2, w2 = _ids(seed + 30, n, 4, 16)
            ids.copy_(i2)
            w.copy_(w2)
            graph.replay()
            eager = efa.expert_grouped(case.layer, x, ids, w)
            torch.cuda.synchronize()
            assert torch.equal(y, eager), seed


def test_layer_copies_agree():
    case = Case(4, 2, 256, 320)
    x = _randn(1, 50, 256).to(BF).cuda()
    ids, w = _ids(3, 50, 2, 4)
    y = efa.expert_grouped(case.layer, x, ids, w)
    assert torch.equal(efa.expert_grouped(case.layer.tiled_copy(), x, ids, w), y)
    assert case.layer.expert_bytes == 3 * 256 * 320 + 4 * (2 * 320 + 256)


def test_near_the_bf16_layer():
    """What 8 bits cost on a layer of normal weights and activations: two operands of a step of max / 127 each."""
    W = [(_randn(i, 8, *s) * 0.02).to(BF).cuda() for i, s in enumerate(((768, 2048), (768, 2048), (2048, 768)))]
    layer = efa.Layer(*W, m=2)
    x = _randn(7, 40, 2048).to(BF).cuda()
    ids, w = _ids(3, 40, 2, 8)
    a, b = efa.expert_grouped(layer, x, ids, w).double(), efa.expert_grouped(layer.int8_copy(), x, ids, w).double()
    # A row of 2048 normal values has its largest at 3.5 of its norm's share, so a step of 2.8 % and an error of
    # 2.8 / sqrt(12) = 0.8 %: of gate and up 1.1 % each (two operands), of h 1.7 % by them and 1.4 % by its own step
    # (largest about 6), of W_down 0.8 %: 2.3 % together; half as much again for the spread of the maxima.
    assert (a - b).norm() <= 0.035 * a.norm()
    assert _abi.MOE_INT8 == 4


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("top,sx", [(1.0, 2.0 ** -10), (2.0 ** 106, 2.0 ** -118), (2.0 ** -126, 2.0 ** 118)])
def test_terms_of_square_tiles_beside_columns_of_any_scale(top, sx, layout):
    """Columns whose scales are far below their neighbours', zero or NaN, and scales near the ends of fp32.  With
    127^2 K < 2^b and S the largest scale of a term's 64 columns (2^-126 at least) the term is rounded to fp16 in steps of at most
    2^-10 of itself, or of 2^-24 (2^b S) 2^-14 where fp16 is subnormal: half of either, and fp32's roundings before
    and behind (three, 2^-24 each), then bf16's."""
    say("int8 scales", top, layout)
    N, d, K, n = 2, 576, 512, 9000
    b = 23  # 127^2 * 512 < 2^23
    g = torch.Generator().manual_seed(5)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int32).to(I8).cuda()
    ratio = torch.tensor([1.0, 2.0 ** -3 * 1.3, 2.0 ** -9 * 1.7, 2.0 ** -15 * 1.1, 2.0 ** -19, 2.0 ** -24 * 1.9, 2.0 ** -40, 0.0])
    sd = (top * ratio.double().repeat(d // 8)[None] * torch.tensor([[1.0], [0.77]])).float()
    sd[1, 64:128] *= 2.0 ** -12  # another largest in one block
    sd[0, 70] = float("nan")
    sd = sd.cuda()
    any_q = (codes(N, K, d), torch.ones(N, K, device="cuda"))
    wd = codes(N, d, K)
    wd[:, :, 1:] = torch.where(torch.arange(d, device="cuda")[None, :, None] % 5 == 0, 0, wd[:, :, 1:])  # sums of one product
    layer = efa.Int8Layer(any_q, any_q, (wd, sd), m=1)
    assert efa.grouped_square(layer, n, efa.MOE_MAT_DOWN)
    if layout == "tiled":
        layer = layer.tiled_copy()
    ids = (torch.arange(n, dtype=torch.int32, device="cuda") % 2)[:, None].contiguous()
    gr = efa.group_slots(ids, N)
    h = efa.Quantized(codes(n, K), torch.full((n,), sx, device="cuda") * (1 + 0.9 * torch.rand(n, generator=g).cuda()))
    y = efa.grouped_down(layer, h, ids, torch.ones(n, 1, device="cuda"), gr).double()
    row = torch.empty(n, dtype=torch.long, device="cuda")
    row[gr.slot_by_expert.long()] = torch.arange(n, device="cuda")
    for e in range(N):
        t = torch.arange(e, n, 2, device="cuda")
        sums = h.q[row[t]].double() @ wd[e].double().T
        s = h.scale[row[t]].double()[:, None]
        want = sums * sd[e].double() * s
        most = torch.nan_to_num(sd[e]).double().view(-1, 64).amax(1).clamp(min=2.0 ** -126).repeat_interleave(64)
        tol = (2.0 ** -11 + 3 * 2.0 ** -24) * want.abs() + 2.0 ** -39 * 2.0 ** b * most * s
        tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-40
        bad = torch.isnan(sd[e])
        assert torch.isnan(y[t][:, bad]).all()
        _within(y[t][:, ~bad], want[:, ~bad], tol[:, ~bad], "scales %g expert %d" % (top, e))
        assert (y[t][:, sd[e] == 0] == 0).all()
