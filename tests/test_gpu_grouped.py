"""The expert operation on grouped rows on the GPU against its formulas in 64 bits
(torch float64, per expert), in bf16 and with 8-bit weights; the grouping and the block
quantisation are checked bit for bit.

Tolerances, per value: a sum of K products in fp32 is off by at most K * 2^-23 * sum|a b|
(every addition rounds or truncates, the products are exact); silu(g) * u by
1.1 |u| dg + |silu(g)| du + 2^-20 |h| (|silu'| < 1.1; the exponential and the division
are good to a few 2^-23); then one rounding, 2^-8 |h| to bf16, or to e4m3 half a step,
2^-4 |h| or 2^-10 of the block's power of two.  y sums m terms, each a bf16 (2^-8), and
is rounded to bf16 (2^-8).

The e4m3 matrix instruction adds the products of 8 consecutive k after it has cut each to
multiples of 2^-13 of the power of two of the group's largest (in the operands' exponents;
2^16 + 2^2 gives 2^16 within a group and the exact sum across groups).  A group of 8
loses less than 7 * 2^-13 of its largest |a b|, all groups less than 7 * 2^-13 * sum|a b|.
That bound is for single values; over a whole output the cuts are small against the
roundings, which the norm of the difference shows: two independent roundings to bf16 are
at most sqrt(2/3) * 2^-8 of the norm of y.
"""
import numpy as np
import pytest
import torch

import expert_ffn_amd as efa
import oracle
from expert_ffn_amd import _abi

from .gpu_cases import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
H8 = torch.float8_e4m3fn


def _randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def _ids(seed, n, m, N, zipf=0.0, pad=0):
    logits = _randn(seed, n, N) - zipf * torch.log(torch.arange(N) + 1.0)
    top, ids = logits.topk(m, dim=1)
    ids, w = ids.to(torch.int32), top.softmax(1)
    if pad:
        ids[n - pad:] = -1
        w[n - pad:] = float("nan")  # the weight of no expert is not read
    return ids.cuda().contiguous(), w.cuda().contiguous()


def _ids_of_counts(counts, seed):
    """ids [n][1] with counts[e] tokens on expert e, shuffled."""
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    p = torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(seed))
    return ids[p].to(torch.int32)[:, None].cuda().contiguous()


class Case:
    """A layer, its weights' values in 64 bits, and the calls on it."""

    def __init__(self, N, m, d, f, typ, layout="plain", seed=1, scale=0.05):
        self.N, self.m, self.d, self.f, self.fp8 = N, m, d, f, typ == "fp8"
        W = [(_randn(seed + i, N, *s) * scale).to(BF).cuda() for i, s in enumerate(((f, d), (f, d), (d, f)))]
        layer = efa.Layer(*W, m=m)
        if self.fp8:
            layer = layer.fp8_copy()
            self.W = [_weight_values(*p) for p in (layer.gate, layer.up, layer.down)]
        else:
            self.W = [w.double() for w in W]
        self.layer = layer.tiled_copy() if layout == "tiled" else layer

    def eps(self, K):
        """Bound of a sum of K products' error, relative to the sum of their magnitudes."""
        return K * 2.0 ** -23 + (7 * 2.0 ** -13 if self.fp8 else 0.0)

    def x_values(self, x):
        return _row_values(efa.quant_rows(x)) if self.fp8 else x.double()

    def gate_up(self, x, ids, out=None):
        g = efa.group_slots(ids, self.N)
        xin = efa.quant_rows(x) if self.fp8 else x
        return g, efa.grouped_gate_up(self.layer, xin, g, out=out)

    def exact_h(self, xv, g):
        """h and the bound of its error before rounding, float64 [S][f], zeros past the last row."""
        at, slot = g.offset.tolist(), g.slot_by_expert.long()
        h = torch.zeros(slot.numel(), self.f, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(h)
        eps = self.eps(self.d)
        for e in range(self.N):
            r = slice(at[e], at[e + 1])
            x = xv[slot[r] // self.m]
            a, b = x @ self.W[0][e].T, x @ self.W[1][e].T
            da, db = eps * (x.abs() @ self.W[0][e].abs().T), eps * (x.abs() @ self.W[1][e].abs().T)
            s = a * torch.sigmoid(a)
            h[r] = s * b
            tol[r] = 1.1 * b.abs() * da + s.abs() * db + 1.1 * da * db + 2.0 ** -20 * h[r].abs()
        return h, tol

    def exact_y(self, hv, ids, w, g):
        """y and the bound of its error, float64 [n][d]."""
        n, at, slot = ids.shape[0], g.offset.tolist(), g.slot_by_expert.long()
        y = torch.zeros(n, self.d, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(y)
        eps = self.eps(self.f)
        for e in range(self.N):
            r = slice(at[e], at[e + 1])
            s = slot[r]
            o = hv[r] @ self.W[2][e].T
            do = eps * (hv[r].abs() @ self.W[2][e].abs().T)
            wt = w.reshape(-1)[s].double()[:, None]
            y.index_add_(0, s // self.m, wt * o)
            tol.index_add_(0, s // self.m, wt.abs() * (do + (2.0 ** -8 + self.m * 2.0 ** -22) * o.abs()))
        return y, tol + 2.0 ** -8 * (y.abs() + tol)


def _pow2(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _row_values(v):
    f = _pow2(v.scale.long() - 127).repeat_interleave(128, dim=1)[:, :v.q.shape[1]]
    return v.q.double() * f


def _weight_values(q, s):
    f = _pow2(s.long() - 127).repeat_interleave(128, dim=1).repeat_interleave(128, dim=2)
    return q.double() * f[:, :q.shape[1], :q.shape[2]]


def _within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert (over <= 0).all(), "%s: %.3g over at %s" % (what, over.max(), np.unravel_index(int(over.argmax()), over.shape))


def _check_h(case, h, x, g, what):
    want, tol = case.exact_h(case.x_values(x), g)
    rows = int(g.offset[-1])
    if not case.fp8:
        _within(h[:rows], want[:rows], (tol + 2.0 ** -8 * (want.abs() + tol))[:rows], what)
        return h.double()
    k = h.scale.long()[:rows] - 127
    step = _pow2(k).repeat_interleave(128, dim=1)[:, :case.f]
    v = _row_values(h)
    _within(v[:rows], want[:rows], tol[:rows] + torch.maximum(2.0 ** -4 * (want.abs() + tol)[:rows], 2.0 ** -10 * step),
            what)
    # the power of two is the smallest that holds the block's maximum, up to that one's error
    pad = -case.f % 128
    hm = torch.nn.functional.pad(want[:rows].abs(), (0, pad)).view(rows, -1, 128).amax(2)
    tm = torch.nn.functional.pad(tol[:rows], (0, pad)).view(rows, -1, 128).amax(2)
    assert (hm - tm <= 448 * _pow2(k)).all() and ((hm + tm > 224 * _pow2(k)) | (k == -127)).all(), what
    return v


def _check_pass(case, x, ids, w, what):
    """The parts against their formulas, and the whole pass against the parts, bit for bit."""
    g, h = case.gate_up(x, ids)
    hv = _check_h(case, h, x, g, what + " h")
    y = efa.grouped_down(case.layer, h, ids, w, g)
    want, tol = case.exact_y(hv, ids, w, g)
    _within(y, want, tol, what + " y")
    assert (y.double() - want).norm() <= 2.0 ** -8 * want.norm(), what
    info = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    ws = case.layer.grouped_workspace(ids.shape[0])
    ws.fill_(255)  # whatever a workspace holds (NaN, -1) is not read
    whole = efa.expert_grouped(case.layer, x, ids, w, ws=ws, info=info)
    assert torch.equal(whole, y), what
    assert info[:2].tolist() == g.u_and_err.tolist() and int(info[2]) == 0
    return y


# --- grouping ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,m,N", [(1, 1, 1), (1, 8, 128), (3, 5, 7), (32, 8, 128), (257, 1, 3), (96, 6, 64),
                                   (4099, 3, 1000), (20000, 8, 128), (700, 256, 1024), (65536, 2, 2)])
@pytest.mark.parametrize("dirty", [False, True])
def test_group_slots_bit_for_bit(n, m, N, dirty):
    say("group", n, m, N, dirty)
    rng = np.random.default_rng(n * 31 + m)
    ids = np.argsort(rng.random((n, N)), axis=1)[:, :m].astype(np.int32) if n * N < 1 << 22 else \
        ((rng.integers(0, N, (n, 1)) + np.arange(m)) % N).astype(np.int32)
    if dirty:  # padding, ids out of range, repeated ids
        ids[rng.random((n, m)) < 0.2] = -1
        ids[0, 0] = N
        ids[n - 1, m - 1] = ids[n - 1, 0]
        ids[n // 2, 0] = np.iinfo(np.int32).max
    g = efa.group_slots(torch.from_numpy(ids).cuda(), N)
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < N)
    slots = np.nonzero(ok)[0]
    by = np.full(n * m, -1)
    by[:slots.size] = slots[np.argsort(flat[slots], kind="stable")]
    count = np.bincount(flat[slots], minlength=N)
    present = np.nonzero(count)[0]
    assert np.array_equal(g.count.cpu(), count)
    assert np.array_equal(g.offset.cpu(), np.concatenate([[0], np.cumsum(count)]))
    assert np.array_equal(g.slot_by_expert.cpu(), by)
    assert np.array_equal(g.distinct.cpu(), np.concatenate([present, np.full(N - present.size, -1)]))
    bad = slots.size < n * m or np.unique((slots // m) * N + flat[slots]).size < slots.size
    assert g.u_and_err.tolist() == [present.size, -5 if bad else 0]


@pytest.mark.parametrize("n,m,N", [(1, 1, 1), (32, 8, 128), (51, 5, 40)])
def test_group_slots_equals_route_group(n, m, N):
    ids, _ = _ids(n, n, m, N, zipf=0.7)
    ids[0, 0] = -3
    for a, b in zip(efa.group_slots(ids, N), efa.route_group(ids, N)):
        assert torch.equal(a, b)


def test_group_slots_equals_the_oracle():
    ids, _ = _ids(5, 500, 6, 64, zipf=1.0)
    st, *want, U = oracle.route_group(ids.cpu().numpy(), 64)
    g = efa.group_slots(ids, 64)
    for a, b in zip(g, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert g.u_and_err.tolist() == [U, st]


# --- block quantisation -----------------------------------------------------------------

def _quant_exact(v):
    """codes' values and exponents of rows (float64 [n][K]) by the definition."""
    n, K = v.shape
    fin = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).abs()
    vals, ks = torch.empty_like(v), []
    for c in range(0, K, 128):
        am = fin[:, c:c + 128].amax(1)
        k = torch.full((n,), -127, dtype=torch.int64)
        for j in range(-127, 121):
            k = torch.where(am > 448 * 2.0 ** (j - 1), torch.full_like(k, j), k)
        p = _pow2(k)[:, None]
        b = v[:, c:c + 128] / p
        e = torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6)))  # 8 significant bits: log2 is not near a whole number
        step = 2.0 ** (e - 3)
        vals[:, c:c + 128] = torch.where(torch.isfinite(b), torch.round(b / step) * step * p, torch.full_like(b, float("nan")))
        ks.append(k)
    return vals, torch.stack(ks, 1)


def _special_rows(K):
    x = _randn(3, 40, K) * torch.exp(2 * _randn(4, 40, 1))
    x[0] = 0
    x[1] = -0.0
    x[2] = 2.0 ** -133            # bf16's least value
    x[3] *= 2.0 ** -126
    x[4] = 448.0                  # the border of an exponent, and its neighbours in bf16
    x[5] = 450.0
    x[6] = 446.0
    x[7] = 3.3e38
    x[8, 0] = float("nan")
    x[9, K - 1] = float("inf")
    x[10, :] = float("-inf")
    x[11] = torch.arange(K) % 16 * 2.0 + 16  # halves of a code's step: ties
    x[12, 1:] *= 2.0 ** -20       # one large value: the rest below the least code
    return x.to(BF)


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 1408])
def test_quant_rows_bit_for_bit(K):
    say("quant", K)
    x = _special_rows(K)
    want, k = _quant_exact(x.double())
    q = efa.quant_rows(x.cuda())
    assert torch.equal(q.scale.cpu().long() - 127, k)
    got = _row_values(efa.Quantized(q.q.cpu(), q.scale.cpu()))
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    # and back: bf16 holds every value between its least and its largest one.  3.3e38 is
    # 248.2 * 2^120, and 256 * 2^120 after rounding to e4m3's steps of 16: bf16's next
    # value above its largest, which reads back as an infinity.
    back = efa.dequant_rows(q).cpu().double()
    held = (want.abs() >= 2.0 ** -126) & (want.abs() < 2.0 ** 128)
    assert torch.equal(back[held], want[held]) and torch.equal(back.isnan(), want.isnan())
    assert back[want.abs() == 2.0 ** 128].isinf().all()
    assert ((back - want).abs()[want.abs() < 2.0 ** -126] <= 2.0 ** -134).all()


@pytest.mark.parametrize("N,R,K", [(1, 16, 16), (3, 128, 128), (2, 272, 144), (2, 192, 400)])
def test_quant_weights_bit_for_bit(N, R, K):
    say("quant weights", N, R, K)
    w = (_randn(7, N, R, K) * 0.02 * torch.exp(_randn(8, N, R, 1))).to(BF)
    q, s = efa.quant_weights(w.cuda())
    q, s = q.cpu(), s.cpu()
    for r in range(0, R, 128):
        for c in range(0, K, 128):
            b = w[:, r:r + 128, c:c + 128].double()
            rr, cc = b.shape[1:]
            for e in range(N):  # one block as 128-wide rows that share the block's maximum
                rows = torch.zeros(rr, 128, dtype=torch.float64)
                rows[:, :cc] = b[e]
                am = rows.abs().max()
                k = int(torch.ceil(torch.log2(am / 448)))
                k += int(am > 448 * 2.0 ** k) - int(am <= 448 * 2.0 ** (k - 1))
                assert int(s[e, r // 128, c // 128]) - 127 == k
                v = b[e] / 2.0 ** k
                step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
                assert torch.equal(q[e, r:r + 128, c:c + 128].double(), torch.round(v / step) * step)


# --- products and passes ------------------------------------------------------------------

SHAPES = [  # N, m, d, d_ff, layout by type
    (1, 1, 16, 16, "plain"), (4, 2, 136, 72, "plain"), (8, 2, 64, 128, "tiled"), (5, 3, 400, 208, "plain"),
    (16, 4, 256, 192, "tiled"), (128, 8, 512, 256, "tiled"), (1024, 2, 64, 64, "tiled"), (8, 8, 192, 320, "plain"),
]


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("N,m,d,f,layout", SHAPES)
@pytest.mark.parametrize("n", [1, 2, 17, 300])
def test_pass(N, m, d, f, layout, n, typ):
    if typ == "fp8":
        d, f = -(-d // 16) * 16, -(-f // 16) * 16
    say("pass", N, m, d, f, layout, n, typ)
    case = Case(N, m, d, f, typ, layout, seed=n)
    x = _randn(50 + n, n, d).to(BF).cuda()
    ids, w = _ids(60 + n, n, m, N, zipf=1.0, pad=n // 4)
    _check_pass(case, x, ids, w, "pass")


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("n", [1, 3, 8, 40])
def test_small_8_bit_passes_sum_in_32_bits(n, layout):
    """Passes of few rows an expert widen the codes: their products carry no cut."""
    case = Case(64, 4, 1024, 640, "fp8", layout, seed=n)
    case.eps = lambda K: K * 2.0 ** -23
    x = (_randn(70 + n, n, 1024) * torch.exp(2 * _randn(71, 1, 1024))).to(BF).cuda()
    ids, w = _ids(72 + n, n, 4, 64, zipf=1.0)
    _check_pass(case, x, ids, w, "small")


COUNTS = [0, 1, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513, 0]


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("layout,d,f", [("plain", 272, 400), ("tiled", 128, 256), ("tiled", 320, 192),
                                        ("tiled", 1024, 512), ("plain", 2032, 144)])
def test_groups_of_every_size(layout, d, f, typ):
    say("groups", layout, d, f, typ)
    case = Case(len(COUNTS), 1, d, f, typ, layout, seed=3)
    ids = _ids_of_counts(COUNTS, 1)
    n = ids.shape[0]
    x = _randn(9, n, d).to(BF).cuda()
    w = _randn(10, n, 1).cuda()
    _check_pass(case, x, ids, w, "groups")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_every_row_on_one_expert(typ):
    case = Case(6, 1, 256, 384, typ, "tiled")
    n = 1500
    ids = torch.full((n, 1), 4, dtype=torch.int32, device="cuda")
    _check_pass(case, _randn(1, n, 256).to(BF).cuda(), ids, _randn(2, n, 1).cuda(), "one expert")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [5, 900])
def test_no_valid_id(typ, n):
    """Every slot padding: y zeros (or unchanged when accumulating), h untouched."""
    case = Case(8, 2, 128, 128, typ, "tiled")
    x = _randn(1, n, 128).to(BF).cuda()
    ids = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.full((n, 2), float("nan"), device="cuda")
    info = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = efa.expert_grouped(case.layer, x, ids, w, info=info)
    assert (y == 0).all() and info.tolist() == [0, -5, 0]
    y = _randn(2, n, 128).to(BF).cuda()
    was = y.clone()
    efa.expert_grouped(case.layer, x, ids, w, y=y, accumulate=True)
    assert torch.equal(y, was)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [6, 1000])
def test_rows_behind_the_last_group_are_left(typ, n):
    case = Case(8, 2, 128, 256, typ, "tiled")
    x = _randn(1, n, 128).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8, pad=n // 3)
    S = n * 2
    if typ == "fp8":
        out = efa.Quantized(torch.full((S, 256), 5.0, device="cuda").to(H8),
                            torch.full((S, 2), 9, dtype=torch.uint8, device="cuda"))
    else:
        out = torch.full((S, 256), 7.0, dtype=BF, device="cuda")
    g, h = case.gate_up(x, ids, out=out)
    rows = int(g.offset[-1])
    assert rows == (n - n // 3) * 2
    if typ == "fp8":
        assert (h.q[rows:].float() == 5).all() and (h.scale[rows:] == 9).all()
    else:
        assert (h[rows:] == 7).all()
    _check_h(case, h, x, g, "h")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [9, 700])
def test_nan_stays_in_its_token(typ, n):
    """A NaN or an infinity in one token's x, or in an expert's weights, reaches the
    tokens that use it and no other."""
    case = Case(8, 2, 256, 128, typ, "tiled")
    x = _randn(1, n, 256).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8)
    clean = efa.expert_grouped(case.layer, x, ids, w)
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[n // 2, 17] = bad
        y = efa.expert_grouped(case.layer, xb, ids, w)
        assert y[n // 2].isnan().any()
        keep = torch.arange(n, device="cuda") != n // 2
        assert torch.equal(y[keep], clean[keep])
    if typ == "bf16":
        W = [t.clone() for t in (case.layer.w_gate, case.layer.w_up, case.layer.w_down)]
        W[0][3] = float("nan")
        y = efa.expert_grouped(efa.Layer(*W, m=2, tiled=True), x, ids, w)
        hit = (ids == 3).any(1)
        assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_repeated_and_out_of_range_ids(typ):
    case = Case(8, 4, 128, 64, typ, "tiled")
    n = 40
    x = _randn(1, n, 128).to(BF).cuda()
    ids, w = _ids(2, n, 4, 8)
    ids[3] = ids[3, 0]              # one expert four times: counts four times
    ids[5, 1], ids[6, 2] = 8, -2147483648
    y = _check_pass(case, x, ids, w, "ids")
    one = efa.expert_grouped(case.layer, x[3:4].contiguous(), ids[3:4].contiguous(), w[3:4].contiguous())
    assert torch.equal(y[3], one[0]) or (y[3] - one[0]).abs().max() <= 2.0 ** -6 * one[0].abs().max()


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [7, 640])
def test_accumulate_and_always_on_experts(typ, n):
    """The recipe for always-on experts: a layer of their own with m = N and weights 1,
    accumulated onto the routed experts' y."""
    case, shared = Case(8, 2, 128, 256, typ, "tiled"), Case(2, 2, 128, 64, typ, "tiled", seed=20)
    x = _randn(1, n, 128).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8)
    y = efa.expert_grouped(case.layer, x, ids, w)
    routed = y.double()
    sids = torch.arange(2, dtype=torch.int32, device="cuda").repeat(n, 1).contiguous()
    ones = torch.ones(n, 2, device="cuda")
    out = efa.expert_grouped(shared.layer, x, sids, ones, y=y, accumulate=True)
    assert out is y
    g, h = shared.gate_up(x, sids)
    want, tol = shared.exact_y(_check_h(shared, h, x, g, "h"), sids, ones, g)
    _within(y, routed + want, tol + 2.0 ** -8 * (routed + want).abs() + 2.0 ** -8 * tol, "accumulated")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_layouts_agree(typ):
    """Plain and tiled copies of the same weights, small and large passes: the order of the
    sums may differ, the values agree to their bounds; one layout repeats bit for bit."""
    a, b = Case(8, 2, 256, 320, typ, "plain"), Case(8, 2, 256, 320, typ, "tiled")
    for n in (3, 800):
        x = _randn(1, n, 256).to(BF).cuda()
        ids, w = _ids(2, n, 2, 8, zipf=1.0)
        ya, yb = _check_pass(a, x, ids, w, "plain"), _check_pass(b, x, ids, w, "tiled")
        assert torch.equal(efa.expert_grouped(a.layer, x, ids, w), ya)
        assert torch.equal(efa.expert_grouped(b.layer, x, ids, w), yb)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [4, 600])
def test_agrees_with_the_verification_pass(typ, n):
    """The same weights through expert_dedup (n <= 64), fp32 y: within the roundings of h
    and y (bf16), or of 8-bit x, weights and h (2^-4 each, about 2^-5 on average)."""
    N, m, d, f = 8, 2, 256, 192
    W = [(_randn(5 + i, N, *s) * 0.05).to(BF).cuda() for i, s in enumerate(((f, d), (f, d), (d, f)))]
    plain = efa.Layer(*W, m=m)
    layer = (plain.fp8_copy() if typ == "fp8" else plain).tiled_copy()
    x = _randn(1, n, d).to(BF).cuda()
    ids, w = _ids(2, n, m, N)
    y = efa.expert_grouped(layer, x, ids, w).double()
    k = min(n, 64)
    ref = efa.expert_dedup(plain, x[:k], ids[:k], w[:k]).double()
    rel = float((y[:k] - ref).norm() / ref.norm())
    assert rel <= (2.0 ** -7 if typ == "bf16" else 2.0 ** -3), rel


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_a_larger_workspace_and_views(typ):
    """A workspace for more tokens serves fewer; x, ids and w may be rows of larger arrays."""
    case = Case(8, 2, 128, 128, typ, "tiled")
    big = 500
    ws = case.layer.grouped_workspace(big)
    x = _randn(1, big, 128).to(BF).cuda()
    ids, w = _ids(2, big, 2, 8)
    for n in (500, 33, 1):
        y = efa.expert_grouped(case.layer, x[-n:], ids[-n:], w[-n:], ws=ws)
        assert torch.equal(y, efa.expert_grouped(case.layer, x[-n:].clone(), ids[-n:].clone(), w[-n:].clone()))


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [3, 500])
def test_captured_and_replayed(typ, n):
    """Two graphs that share a workspace, replayed in turn with eager passes between."""
    case = Case(8, 2, 256, 128, typ, "tiled")
    ws = case.layer.grouped_workspace(n)
    x = _randn(1, n, 256).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8, pad=n // 4)
    w = w.nan_to_num()
    graphs, outs = [], []
    for _ in range(2):
        y = torch.empty(n, 256, dtype=BF, device="cuda")
        efa.expert_grouped(case.layer, x, ids, w, y=y, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            efa.expert_grouped(case.layer, x, ids, w, y=y, ws=ws)
        graphs.append(g)
        outs.append(y)
    for i in range(4):
        x.copy_(_randn(30 + i, n, 256).to(BF))
        ids.copy_(_ids(40 + i, n, 2, 8)[0])
        want = efa.expert_grouped(case.layer, x, ids, w)
        for g, y in zip(graphs, outs):
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_side_streams(typ):
    """Passes on two streams at once, each with what it allocates itself."""
    case = Case(8, 2, 256, 512, typ, "tiled")
    n = 900
    xs = [_randn(i, n, 256).to(BF).cuda() for i in range(2)]
    ids, w = _ids(2, n, 2, 8)
    want = [efa.expert_grouped(case.layer, x, ids, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(efa.expert_grouped(case.layer, xs[i], ids, w, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("layout,d,f", [("tiled", 512, 576), ("plain", 528, 640), ("plain", 784, 720),
                                        ("tiled", 896, 960), ("plain", 33040, 128), ("plain", 128, 33168)])
def test_contractions_of_every_length(layout, d, f, typ):
    """From four units of 128 bytes a tile, the fewest of the square tiles, to more scale
    bytes than a work group has threads."""
    say("lengths", layout, d, f, typ)
    counts = [300, 0, 41, 7]
    case = Case(len(counts), 1, d // (1 if typ == "fp8" else 2), f // (1 if typ == "fp8" else 2), typ, layout, seed=5)
    ids = _ids_of_counts(counts, 6)
    n = ids.shape[0]
    _check_pass(case, _randn(7, n, case.d).to(BF).cuda(), ids, _randn(8, n, 1).cuda(), "lengths")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_square_tiles_of_many_experts(typ):
    N, m, n = 1000, 3, 1500
    case = Case(N, m, 512, 528, typ, "plain", seed=4)
    ids, w = _ids(5, n, m, N, zipf=0.7, pad=11)
    _check_pass(case, _randn(6, n, 512).to(BF).cuda(), ids, w, "many experts")


def _gpu_layer(N, m, d, f, typ, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = [torch.randn(N, *s, generator=g, device="cuda", dtype=BF).mul_(0.05) for s in ((f, d), (f, d), (d, f))]
    layer = efa.Layer(*W, m=m)
    if typ == "fp8":
        layer = layer.fp8_copy()
    return layer, layer.tiled_copy() if layout == "tiled" else layer


def _columns(layer, which, e, cols):
    """Rows `cols` of expert e's matrix in 64 bits (plain layers)."""
    if isinstance(layer, efa.Fp8Layer):
        q, s = (layer.gate, layer.up, layer.down)[which]
        K = q.shape[2]
        return q[e, cols].double() * _pow2(s[e, cols // 128].long() - 127).repeat_interleave(128, dim=1)[:, :K]
    return (layer.w_gate, layer.w_up, layer.w_down)[which][e, cols].double()


def _check_sample(plain, x, ids, w, g, h, y, rows, hc, yc, fp8):
    """h at rows x hc against x, y at those rows' tokens x yc against h (m = 1: a token a row)."""
    token = g.slot_by_expert[rows].long()
    assert plain.m == 1
    xq = efa.quant_rows(x[token].contiguous()) if fp8 else x[token]
    xv = _row_values(xq) if fp8 else xq.double()
    hq = efa.Quantized(h.q[rows], h.scale[rows]) if fp8 else h[rows]
    hv = _row_values(hq) if fp8 else hq.double()
    cut = 7 * 2.0 ** -13 if fp8 else 0.0
    ex, eh = xv.shape[1] * 2.0 ** -23 + cut, hv.shape[1] * 2.0 ** -23 + cut
    for i in range(rows.numel()):
        e = int(ids[token[i], 0])
        W = [_columns(plain, k, e, hc) for k in (0, 1)]
        a, b = (xv[i] @ m_.T for m_ in W)
        da, db = (ex * (xv[i].abs() @ m_.abs().T) for m_ in W)
        s = a * torch.sigmoid(a)
        want = s * b
        tol = 1.1 * b.abs() * da + s.abs() * db + 1.1 * da * db + 2.0 ** -20 * want.abs()
        if fp8:
            step = _pow2(hq.scale[i, hc // 128].long() - 127) * 2.0 ** -10
            tol = tol + torch.maximum(2.0 ** -4 * (want.abs() + tol), step)
        else:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        _within(hv[i, hc], want, tol, "h %d" % i)
        D = _columns(plain, 2, e, yc)
        o = D @ hv[i]
        do = eh * (D.abs() @ hv[i].abs())
        wt = w[token[i], 0].double()
        tol = wt.abs() * (do + (2.0 ** -8 + 2.0 ** -22) * o.abs())
        want = wt * o
        _within(y[token[i], yc], want, tol + 2.0 ** -8 * (want.abs() + tol), "y %d" % i)


def _spread(n, k):
    return torch.linspace(0, n - 1, k, dtype=torch.float64, device="cuda").long().unique()


def _run_parts(layer, x, ids, w, fp8):
    g = efa.group_slots(ids, layer.N)
    h = efa.grouped_gate_up(layer, efa.quant_rows(x) if fp8 else x, g)
    return g, h, efa.grouped_down(layer, h, ids, w, g)


@pytest.mark.parametrize("typ,n", [("bf16", 140001), ("fp8", 270001)])
def test_x_beyond_31_bits(typ, n):
    """More than 2 GiB of x."""
    say("x beyond 31 bits", typ)
    d, f = 8192, 1040
    plain, layer = _gpu_layer(2, 1, d, f, typ, "plain", 1)
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=BF)
    ids = (torch.arange(n, device="cuda", dtype=torch.int32) % 2)[:, None].contiguous()
    w = torch.rand(n, 1, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    fp8 = typ == "fp8"
    g, h, y = _run_parts(layer, x, ids, w, fp8)
    _check_sample(plain, x, ids, w, g, h, y, _spread(n, 12), _spread(f, 40), _spread(d, 40), fp8)


@pytest.mark.parametrize("layout,d,f,typ", [("plain", 16384, 65272, "bf16"), ("tiled", 16384, 65248, "bf16"),
                                            ("plain", 16384, 65408, "bf16"), ("tiled", 16384, 65408, "bf16"),
                                            ("plain", 32752, 65536, "fp8"), ("tiled", 32640, 65472, "fp8")])
def test_matrices_of_31_bits(layout, d, f, typ):
    """Matrices of almost and of more than 2 GiB, less and more than a tile below it."""
    say("matrices of 31 bits", layout, d, f, typ)
    n = 300
    plain, layer = _gpu_layer(1, 1, d, f, typ, layout, 1)
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=BF)
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    w = torch.rand(n, 1, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    fp8 = typ == "fp8"
    g, h, y = _run_parts(layer, x, ids, w, fp8)
    _check_sample(plain, x, ids, w, g, h, y, _spread(n, 6), _spread(f, 60), _spread(d, 60), fp8)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
def test_a_million_rows(typ):
    """More thin tiles than one launch holds, and O and h beyond 32 bits."""
    say("a million rows", typ)
    n, d, f = (1 << 20) + 1, 64, 4096
    plain, layer = _gpu_layer(5, 1, d, f, typ, "tiled", 1)
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=BF)
    ids = torch.randint(0, 5, (n, 1), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda",
                        dtype=torch.int32)
    w = torch.rand(n, 1, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    fp8 = typ == "fp8"
    g, h, y = _run_parts(layer, x, ids, w, fp8)
    _check_sample(plain, x, ids, w, g, h, y, _spread(n, 40), _spread(f, 60), _spread(d, 60), fp8)
    assert torch.equal(efa.expert_grouped(layer, x, ids, w), y)


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [2, 700])
def test_captured_parts(typ, n):
    """Grouping, quantisation and the products captured one after the other, replayed on
    other values with eager calls between."""
    case = Case(8, 2, 256, 320, typ, "tiled")
    fp8 = typ == "fp8"
    x = _randn(1, n, 256).to(BF).cuda()
    ids, w = _ids(2, n, 2, 8)
    _run_parts(case.layer, x, ids, w, fp8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, h, y = _run_parts(case.layer, x, ids, w, fp8)
    for i in range(3):
        x.copy_(_randn(30 + i, n, 256).to(BF))
        ids.copy_(_ids(40 + i, n, 2, 8)[0])
        _, _, want = _run_parts(case.layer, x, ids, w, fp8)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_x_is_of_the_layers_type():
    x = _randn(1, 4, 64).to(BF).cuda()
    ids, _ = _ids(2, 4, 1, 2)
    for typ, xin in (("bf16", efa.quant_rows(x)), ("fp8", x), ("bf16", x.float())):
        case = Case(2, 1, 64, 64, typ)
        with pytest.raises(TypeError):
            efa.grouped_gate_up(case.layer, xin, efa.group_slots(ids, 2))


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [3, 400])
def test_many_slots_a_token(typ, n):
    """More slots a token than a wave has lanes, some of them empty."""
    N, m = 160, 130
    case = Case(N, m, 256, 208, typ, "plain", seed=n)
    ids, w = _ids(5, n, m, N)
    ids[n // 2, 1:129] = -1
    ids[0, :64] = N
    _check_pass(case, _randn(6, n, 256).to(BF).cuda(), ids, w, "many slots")


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [20, 1300])
def test_the_same_bits_every_time(typ, n):
    case = Case(32, 4, 512, 384, typ, "tiled")
    x = _randn(1, n, 512).to(BF).cuda()
    ids, w = _ids(2, n, 4, 32, zipf=1.0, pad=n // 9)
    first = efa.expert_grouped(case.layer, x, ids, w)
    for _ in range(8):
        assert torch.equal(efa.expert_grouped(case.layer, x, ids, w), first)


# --- the terms of a token's sum ---------------------------------------------------------

def _exact_sum(case, hv, ids, w, g, eps, rounding, block=0.0):
    """y and the bound of its error: sums of K products in fp32 (``eps`` of their
    magnitudes), each term rounded on its way to ``rounding`` of itself or ``block`` of the
    largest of its 64 columns, m weighted additions in fp32 (2^-22 a term), and one rounding
    to bf16."""
    at, slot = g.offset.tolist(), g.slot_by_expert.long()
    y = torch.zeros(ids.shape[0], case.d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e in range(case.N):
        s = slot[at[e]:at[e + 1]]
        h = hv[at[e]:at[e + 1]]
        o, mag = h @ case.W[2][e].T, h.abs() @ case.W[2][e].abs().T
        wt = w.reshape(-1)[s].double()[:, None]
        top = torch.nn.functional.pad(mag, (0, -case.d % 64)).view(mag.shape[0], -1, 64).amax(2) if s.numel() else mag
        top = top.repeat_interleave(64, dim=1)[:, :case.d]  # (a bound of the largest |o|)
        y.index_add_(0, s // case.m, wt * o)
        tol.index_add_(0, s // case.m, wt.abs() * (eps * mag + (rounding + case.m * 2.0 ** -22) * o.abs() + block * top))
    return y, tol + 2.0 ** -8 * (y.abs() + tol)


def _down_case(N, m, d, f, typ, layout, seed):
    """A layer whose experts differ in the sign of one column of W_down: two of them with
    weights 1 and -1 leave 2 w_c h_c of sums that are about sqrt(f) / 2 times as large.
    (A sign leaves a block's maximum, and so every code's magnitude, as it is.)"""
    case = Case(N, m, d, f, typ, layout, seed=seed)
    W = [(_randn(seed + i, *s) * 0.05).to(BF).repeat(N, 1, 1).cuda() for i, s in enumerate(((f, d), (f, d), (d, f)))]
    W[2][1::2, :, f // 3] *= -1
    layer = efa.Layer(*W, m=m)
    if case.fp8:
        layer = layer.fp8_copy()
        case.W = [_weight_values(*p) for p in (layer.gate, layer.up, layer.down)]
    else:
        case.W = [v.double() for v in W]
    case.layer = layer.tiled_copy() if layout == "tiled" else layer
    return case


def _cancelling(case, n, seed):
    """Every token on neighbouring experts with weights 1, -1, 1, ..., one h for all its slots."""
    first = torch.randint(0, case.N, (n, 1), generator=torch.Generator().manual_seed(seed))
    ids = ((first + torch.arange(case.m)) % case.N).to(torch.int32).cuda().contiguous()
    w = (1.0 - 2.0 * (torch.arange(case.m) % 2)).repeat(n, 1).cuda().contiguous()
    g = efa.group_slots(ids, case.N)
    h = _randn(seed + 1, n, case.f).to(BF).cuda()[g.slot_by_expert.long() // case.m].contiguous()
    hq = efa.quant_rows(h) if case.fp8 else h
    return ids, w, g, hq, _row_values(hq) if case.fp8 else h.double()


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("N,m,n", [(2, 2, 1), (2, 2, 15), (8, 4, 9), (128, 8, 1), (128, 8, 32)])
def test_terms_that_cancel(N, m, n, layout, typ):
    """Passes of few rows an expert hold the terms of a token's sum in fp32: y is rounded
    once, whatever the terms are next to it."""
    say("cancel", N, m, n, layout, typ)
    case = _down_case(N, m, 512, 768, typ, layout, seed=n)
    ids, w, g, h, hv = _cancelling(case, n, 80 + n)
    y = efa.grouped_down(case.layer, h, ids, w, g)
    want, tol = _exact_sum(case, hv, ids, w, g, 768 * 2.0 ** -23, 0.0)
    _within(y, want, tol, "y")
    # one rounding: at most 2^-8 of the norm, on average less than half of that
    assert (y.double() - want).norm() <= 2.0 ** -8 * want.norm()


# --- what the two kinds of tiles do with products of very different size ----------------

def _codes(values):
    return torch.tensor(values).to(H8).cuda()


def _group_case(small, at, n):
    """Down products whose contraction has three products that matter: 2^16, ``small`` (h's 2
    times small / 2) and -2^16, at the places ``at`` of consecutive k; output column r takes
    those of the r-th run of 24 k.  Scales are 1."""
    K, d = 1536, 64
    h, w = torch.zeros(K), torch.zeros(d, K)
    for r in range(d):
        for k, a, b in zip(at, (256.0, 2.0, -256.0), (256.0, small / 2, 256.0)):
            h[24 * r + k], w[r, 24 * r + k] = a, b
    one = torch.full((1, 1, 12), 127, dtype=torch.uint8, device="cuda")
    up = (torch.zeros(1, K, d, device="cuda").to(H8), one.view(1, 12, 1).contiguous())
    layer = efa.Fp8Layer(up, up, (_codes(w.tolist())[None].contiguous(), one), m=1)
    hq = efa.Quantized(_codes(h.repeat(n, 1).tolist()), torch.full((n, 12), 127, dtype=torch.uint8, device="cuda"))
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    return layer, hq, ids


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("n,square", [(1, False), (7, False), (15, False), (16, True), (300, True)])
@pytest.mark.parametrize("small,at", [(4.0, (0, 1, 2)), (4.0, (5, 0, 7)), (8.0, (0, 1, 2)), (4.0, (0, 8, 16)),
                                      (0.125, (3, 10, 20))])
def test_products_of_one_group_of_eight(small, at, n, square, layout):
    """2^16 + small - 2^16: ``small`` from thin tiles, whose products are summed in fp32.  The e4m3
    instruction of square tiles cuts each product to multiples of 2^-13 of its group's largest, 8
    here: 4 beside 2^16 is lost, 8 is kept, and so is 4 in a group of its own (of 0.125, the fp32 sum
    2^16 + 2^-3 holds all: 19 bits)."""
    say("group of eight", small, at, n)
    layer, h, ids = _group_case(small, at, n)
    layer = layer.tiled_copy() if layout == "tiled" else layer
    assert efa.grouped_square(layer, n, _abi.MOE_MAT_DOWN) is square
    y = efa.grouped_down(layer, h, ids, torch.ones(n, 1, device="cuda"), efa.group_slots(ids, 1))
    lost = square and small < 8.0 and max(at) < 8
    assert (y.double() == (0.0 if lost else small)).all(), y.unique()


@pytest.mark.parametrize("typ", ["bf16", "fp8"])
@pytest.mark.parametrize("n,square", [(3, False), (15, False), (200, True)])
@pytest.mark.parametrize("tiny", ["weights", "inputs"])
def test_the_least_values(tiny, n, square, typ):
    """Values down to bf16's least, 2^-133 (scale byte 0 where they are codes), next to values
    of about 2^120, so that the sums are ordinary numbers: none of their bits are lost."""
    say("least values", tiny, n, typ)
    N, d, f = 1, 512, 576
    ints = [torch.randint(-255, 256, s, generator=torch.Generator().manual_seed(i))
            for i, s in enumerate(((N, f, d), (N, f, d), (N, d, f), (n, d), (n, f)))]
    small = [(v.double() * 2.0 ** -133).float().to(BF) for v in ints]
    large = [(_randn(20 + i, *v.shape) * 2.0 ** 120).to(BF) for i, v in enumerate(ints)]
    W, (x, h) = (small[:3], large[3:]) if tiny == "weights" else (large[:3], small[3:])
    assert all(float(v.float().abs().max()) <= 2.0 ** -125 for v in small)
    case = Case(N, 1, d, f, typ)
    layer = efa.Layer(*(v.cuda() for v in W), m=1)
    if case.fp8:
        layer = layer.fp8_copy()
        case.W = [_weight_values(*p) for p in (layer.gate, layer.up, layer.down)]
        q = efa.quant_rows(small[3].cuda()).scale if tiny == "inputs" else layer.gate[1]
        assert (q == 0).all()
    else:
        case.W = [v.double().cuda() for v in W]
    case.layer = layer
    for mat in (_abi.MOE_MAT_GATE_UP, _abi.MOE_MAT_DOWN):
        assert efa.grouped_square(layer, n, mat) is square
    x, h = x.cuda(), h.cuda()
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    g, got = case.gate_up(x, ids)
    _check_h(case, got, x, g, "h")
    w = torch.ones(n, 1, device="cuda")
    hq = efa.quant_rows(h) if case.fp8 else h
    y = efa.grouped_down(layer, hq, ids, w, g)
    want, tol = _exact_sum(case, _row_values(hq) if case.fp8 else h.double(), ids, w, g, case.eps(f),
                           2.0 ** -8 if square else 0.0)
    assert want.abs().median() > 2.0 ** -10
    _within(y, want, tol, "y")


def test_more_rows_than_an_int_holds():
    """2^32 + 1 tokens, or 2^32 + 16 columns, are refused, not taken for one and sixteen."""
    ids = torch.empty((1 << 32) + 1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(_abi.MoeError):
        efa.group_slots(ids, 8)
    del ids
    x = torch.empty(1, (1 << 32) + 16, dtype=BF, device="cuda")
    with pytest.raises(_abi.MoeError):
        efa.quant_rows(x)
    with pytest.raises(_abi.MoeError):
        efa.quant_weights(x.view(1, 1, -1).expand(1, 1, -1))
    del x
    torch.cuda.empty_cache()
