"""The whole-layer pass (router, selection, routed and always-on experts) on the GPU against its
formulas in 64 bits.

Tolerances.  A logit is a sum of d products in fp32: off by at most dl = d * 2^-23 * sum|x w|.  A
score s moves by s * 2 dl (softmax: its own logit and the sum's; sigmoid: less), and by a few 2^-22
of the exponentials and the division; s + b is rounded once, 2^-24.  An expert is where it
may be if no other that comes later is larger by more than both errors.  Weights: 2 dl and
2^-20 relative, renormalised ones twice that.  y is, bit for bit, what the expert call gives for
the ids and weights handed back, rounded to the layer's type; and by itself within 2^-8 (bf16)
of the formula, relative to the magnitudes that are added up.
"""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


class Case:
    def __init__(self, N, m, d, f, typ=BF, layout="plain", shared=0, score="softmax", bias=False, renorm=True, scale=1.0,
                 seed=1, spread=1.0):
        self.N, self.m, self.d, self.f, self.typ = N, m, d, f, typ
        mk = lambda i, E: [(_randn(seed + i + k, E, *s) * 0.05).to(typ).cuda()  # noqa: E731
                           for k, s in enumerate(((f, d), (f, d), (d, f)))]
        self.W, self.S = mk(1, N), mk(11, shared) if shared else None
        layer = efa.Layer(*self.W, m=m, shared=tuple(self.S) if shared else None)
        self.layer = {"plain": lambda: layer, "packed": layer.packed_copy, "tiled": layer.tiled_copy}[layout]()
        self.wr = (_randn(seed + 20, N, d) * spread / d ** 0.5).to(typ).cuda()
        self.b = (_randn(seed + 21, N) * 0.1).cuda() if bias else None
        self.score, self.renorm, self.scale = score, renorm, scale
        self.router = efa.Router(self.wr, score=score, bias=self.b, renorm=renorm, scale=scale)

    def x(self, n, seed=5):
        return _randn(seed, n, self.d).to(self.typ).cuda()

    def scores(self, x):
        """(key, its error, scores) in float64."""
        l = x.double() @ self.wr.double().T
        dl = self.d * 2.0 ** -23 * (x.double().abs() @ self.wr.double().abs().T)
        s = l.softmax(1) if self.score == "softmax" else l.sigmoid()
        if self.b is None:
            return l, dl, s, dl
        ds = s * (2 * dl.amax(1, keepdim=True) + 2.0 ** -20)
        key = s + self.b.double()
        return key, ds + 2.0 ** -23 * key.abs(), s, dl

    def check_routing(self, x, ids, w):
        key, dk, s, dl = self.scores(x)
        n = x.shape[0]
        left = torch.ones_like(key, dtype=torch.bool)
        rows = torch.arange(n, device="cuda")
        for j in range(self.m):
            e = ids[:, j].long()
            assert (e >= 0).all() and (e < self.N).all()
            assert left[rows, e].all(), "an expert twice"
            left[rows, e] = False
            ahead = torch.where(left, key - dk, torch.full_like(key, -float("inf"))).amax(1)
            assert (key[rows, e] + dk[rows, e] >= ahead).all(), j
        v = torch.gather(s, 1, ids.long())
        tol = 2 * dl.amax(1, keepdim=True) + 2.0 ** -20
        if self.renorm:
            v, tol = v / v.sum(1, keepdim=True), 2 * tol
        v = v * self.scale
        assert ((w.double() - v).abs() <= tol * v.abs() + 1e-40).all()

    def exact(self, x, ids, w):
        """(y, magnitudes) in float64."""
        x = x.double()
        y = torch.zeros(x.shape[0], self.d, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        def ffn(x, gate, up, down):
            z = x @ gate.double().T
            h = z * z.sigmoid() * (x @ up.double().T)
            return h @ down.double().T, h.abs() @ down.double().abs().T
        for e in range(self.N):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                o, a = ffn(x[t], *(W[e] for W in self.W))
                wt = w[t, j].double()[:, None]
                y.index_add_(0, t, wt * o)
                mag.index_add_(0, t, wt.abs() * a)
        for e in range(0 if self.S is None else self.S[0].shape[0]):
            o, a = ffn(x, *(W[e] for W in self.S))
            y += o
            mag += a
        return y, mag


def _check(case, n, seed=5):
    x = case.x(n, seed)
    ids = torch.full((n, case.m), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n, case.m), 7.0, device="cuda")
    info = torch.full((3,), 9, dtype=torch.int32, device="cuda")
    ws = case.layer.pass_workspace(n)
    y = efa.layer_pass(case.layer, case.router, x, ids=ids, w=w, info=info, ws=ws)
    assert y.dtype is case.typ and y.shape == x.shape
    case.check_routing(x, ids, w)
    parts = efa.expert_dedup(case.layer, x, ids, w)
    assert torch.equal(parts.to(case.typ), y)
    assert info.tolist() == [torch.unique(ids).numel(), 0, 0]
    want, mag = case.exact(x, ids, w)
    # h as two bf16 (2^-17) or fp32; sums of d and of f products in fp32, far below
    tol = (2.0 ** -16 + (case.d + case.f) * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs() * (case.typ is BF) + 1e-30
    assert ((y.double() - want).abs() <= 1.01 * tol).all()
    # again, with the workspace as the call left it and without the outputs
    assert torch.equal(efa.layer_pass(case.layer, case.router, x, ws=ws), y)
    return x, y, ids, w


FORMS = [dict(), dict(renorm=False, scale=2.5), dict(score="sigmoid"), dict(score="sigmoid", bias=True, scale=16.0),
         dict(bias=True), dict(score="sigmoid", bias=True, renorm=False), dict(bias=True, renorm=False)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("n", [1, 2, 3, 16, 17, 33])
def test_forms(form, n):
    say("layer form", FORMS[form], n)
    _check(Case(40, 5, 256, 192, seed=form, **FORMS[form]), n)


@pytest.mark.parametrize("N,m,d,f,typ,layout,shared", [
    (1, 1, 8, 8, BF, "plain", 0), (3, 3, 40, 24, F32, "plain", 1), (8, 2, 4096, 64, BF, "tiled", 0),
    (16, 4, 256, 192, BF, "packed", 2), (70, 5, 200, 168, F32, "plain", 1), (128, 8, 2048, 96, BF, "tiled", 0),
    (129, 7, 136, 64, BF, "plain", 3), (256, 16, 512, 32, F32, "tiled", 0), (257, 9, 264, 40, BF, "plain", 0),
    (1024, 8, 2048, 8, BF, "plain", 0), (1024, 200, 64, 32, BF, "tiled", 0), (5, 5, 16384, 8, BF, "plain", 0)])
def test_shapes(N, m, d, f, typ, layout, shared):
    say("layer shape", N, m, d, f, typ, layout, shared)
    case = Case(N, m, d, f, typ, layout, shared, score="sigmoid" if N % 2 else "softmax", bias=N > 200)
    for n in (1, 2, 7, 64):
        if n * m + shared <= 256:
            _check(case, n, seed=n)


def test_a_token_alone_and_among_others():
    say("layer alone")
    case = Case(128, 8, 2048, 64, score="sigmoid", bias=True, layout="tiled")
    x, y, ids, w = _check(case, 32)
    for t in (0, 5, 16, 31):
        i1, w1 = torch.empty_like(ids[:1]), torch.empty_like(w[:1])
        y1 = efa.layer_pass(case.layer, case.router, x[t:t + 1].clone(), ids=i1, w=w1)
        assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])
        assert (y1[0].double() - y[t].double()).abs().max() <= 2.0 ** -7 * y[t].double().abs().max()


def test_equal_scores_take_the_lower_ids():
    say("layer ties")
    for N, kw in ((40, {}), (200, {}), (300, {}), (300, dict(score="sigmoid"))):
        case = Case(N, 6, 64, 32, **kw)
        case.wr[[3, 17, N - 1, 30]] = case.wr[11].clone()
        case.wr[[4, 7]] = 0
        case.router = efa.Router(case.wr, **kw)
        x = case.x(9)
        x = x[:1].repeat(9, 1)
        x[4:] *= -1
        ids = torch.empty(9, 6, dtype=torch.int32, device="cuda")
        w = torch.empty(9, 6, device="cuda")
        efa.layer_pass(case.layer, case.router, x, ids=ids, w=w)
        l = efa.router_topk(case.wr, x, 6).logits.double()
        case.check_routing(x, ids, w)
        for same in ([3, 11, 17, 30, N - 1], [4, 7]):
            for t in range(9):
                got = [e for e in ids[t].tolist() if e in same]
                assert got == same[:len(got)], (N, t, l[t])
    case = Case(30, 4, 64, 32)
    zero = efa.Router(torch.zeros_like(case.wr))
    ids = torch.empty(3, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(3, 4, device="cuda")
    efa.layer_pass(case.layer, zero, case.x(3), ids=ids, w=w)
    assert ids.tolist() == [[0, 1, 2, 3]] * 3 and (w == 0.25).all()


def test_sigmoids_too_small_for_fp32():
    say("layer small sigmoids")
    case = Case(12, 3, 64, 32, score="sigmoid")
    x = torch.ones(2, 64, dtype=BF, device="cuda")
    l = -150.0 - 4 * torch.arange(12).double()
    wr = (l[:, None] / 64).repeat(1, 64).to(BF).cuda()
    ids = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(2, 3, device="cuda")
    efa.layer_pass(case.layer, efa.Router(wr, score="sigmoid", scale=3.0), x, ids=ids, w=w)
    assert ids.tolist() == [[0, 1, 2]] * 2
    lk = (wr.double().sum(1))[:3]
    want = 3 * (lk - lk[0]).exp() / (lk - lk[0]).exp().sum()
    assert ((w.double() - want).abs() <= 2.0 ** -14 * want).all()  # logits near 150: 2^-16 in fp32
    efa.layer_pass(case.layer, efa.Router(wr, score="sigmoid", renorm=False), x, ids=ids, w=w)
    assert ids.tolist() == [[0, 1, 2]] * 2 and (w == 0).all()


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_nan(form):
    say("layer nan", FORMS[form])
    case = Case(20, 4, 64, 96, shared=1, **FORMS[form])
    x = case.x(6)
    x[2, 5] = float("nan")
    info = torch.zeros(3, dtype=torch.int32, device="cuda")
    ids = torch.empty(6, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(6, 4, device="cuda")
    y = efa.layer_pass(case.layer, case.router, x, ids=ids, w=w, info=info)
    assert (ids[2] == -1).all() and (w[2] == 0).all() and int(info[1]) == -5
    keep = [0, 1, 3, 4, 5]
    case.check_routing(x[keep], ids[keep], w[keep])
    assert torch.isnan(y[2]).all() and torch.isfinite(y[keep]).all()  # (the always-on expert's, of NaN)
    wr = case.wr.clone()
    wr[3] = float("nan")  # one expert's row: the others are as without it
    other = efa.Router(wr, score=case.score, bias=case.b, renorm=case.renorm, scale=case.scale)
    x = case.x(6)
    efa.layer_pass(case.layer, other, x, ids=ids, w=w)
    assert not (ids == 3).any()
    sub = [e for e in range(20) if e != 3]
    case.wr, case.N = case.wr[sub], 19
    case.b = None if case.b is None else case.b[sub]
    case.check_routing(x, torch.where(ids > 3, ids - 1, ids), w)


def test_accumulate():
    say("layer accumulate")
    for typ in (BF, F32):
        case = Case(16, 4, 128, 64, typ, shared=1)
        x = case.x(5)
        ids, w = torch.empty(5, 4, dtype=torch.int32, device="cuda"), torch.empty(5, 4, device="cuda")
        y0 = _randn(3, 5, 128).to(typ).cuda()
        y = efa.layer_pass(case.layer, case.router, x, y=y0.clone(), ids=ids, w=w, accumulate=True)
        assert torch.equal(y, efa.expert_dedup(case.layer, x, ids, w, y=y0.float(), accumulate=True).to(typ))


def test_one_workspace_for_every_length():
    say("layer lengths")
    case = Case(64, 4, 512, 128, shared=1)
    ws = case.layer.pass_workspace(40)
    for n in (40, 1, 17, 2, 33, 3, 16, 40):
        x = case.x(n, n)
        assert torch.equal(efa.layer_pass(case.layer, case.router, x, ws=ws), efa.layer_pass(case.layer, case.router, x))


def test_streams_and_graphs():
    say("layer streams and graphs")
    case = Case(64, 4, 512, 128, score="sigmoid", bias=True, layout="tiled")
    for n in (1, 2, 20):
        x = case.x(n)
        want = efa.layer_pass(case.layer, case.router, x)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        got = efa.layer_pass(case.layer, case.router, x, stream=st)
        st.synchronize()
        assert torch.equal(got, want)
        ws, y = case.layer.pass_workspace(n), torch.empty_like(want)
        ids = torch.empty(n, 4, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            efa.layer_pass(case.layer, case.router, x, y=y, ids=ids, ws=ws)
        for seed in range(4):
            x.copy_(case.x(n, seed + 40))
            graph.replay()
            i2 = torch.empty_like(ids)
            eager = efa.layer_pass(case.layer, case.router, x, ids=i2)
            torch.cuda.synchronize()
            assert torch.equal(y, eager) and torch.equal(ids, i2), (n, seed)


def test_two_layers_in_turn_then_a_prompt():
    """As a model runs them: two layers' passes one after the other on one stream, each with its workspace, and
    the same routing through the grouped calls in bf16 and int8."""
    say("layers in turn")
    a, b = Case(32, 4, 256, 128, seed=1), Case(32, 4, 256, 128, seed=50, score="sigmoid")
    wa, wb = a.layer.pass_workspace(8), b.layer.pass_workspace(8)
    x = a.x(8)
    ids, w = torch.empty(8, 4, dtype=torch.int32, device="cuda"), torch.empty(8, 4, device="cuda")
    for _ in range(3):
        y1 = efa.layer_pass(a.layer, a.router, x, ws=wa)
        y2 = efa.layer_pass(b.layer, b.router, y1, ids=ids, w=w, ws=wb)
    b.check_routing(y1, ids, w)
    want, mag = b.exact(y1, ids, w)
    assert ((y2.double() - want).abs() <= 2.0 ** -8 * (want.abs() + mag)).all()
    g = efa.expert_grouped(b.layer, y1, ids, w)
    assert ((g.double() - want).abs() <= 2.0 ** -6 * mag).all()  # (h in bf16 there)
    q = efa.expert_grouped(b.layer.int8_copy(), y1, ids, w).double()
    assert (q - want).norm() <= 0.035 * want.norm()


def test_refusals_on_the_device():
    case = Case(16, 4, 128, 64)
    x = case.x(5)
    bad = [dict(x=x.float()), dict(x=x[:, :64]), dict(x=x.t()), dict(x=x.cpu()), dict(y=torch.empty(5, 128, device="cuda")),
           dict(ids=torch.empty(5, 4, device="cuda")), dict(w=torch.empty(5, 3, device="cuda")),
           dict(info=torch.empty(2, dtype=torch.int32, device="cuda")), dict(router=case.wr), dict(layer=case.layer.desc()),
           dict(router=efa.Router(case.wr[:8].contiguous())), dict(router=efa.Router(case.wr.float())), dict(accumulate=True)]
    for kw in bad:
        a = dict(layer=case.layer, router=case.router, x=x)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            efa.layer_pass(**a)
    for kw in (dict(x=case.x(65)), dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        a = dict(layer=case.layer, router=case.router, x=x)
        a.update(kw)
        with pytest.raises(efa.MoeError):
            efa.layer_pass(**a)
    with pytest.raises(ValueError):
        efa.Router(case.wr, score="tanh")
    with pytest.raises(ValueError):
        efa.Router(case.wr, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        efa.Router(case.wr, bias=torch.zeros(16, device="cuda", dtype=BF))
