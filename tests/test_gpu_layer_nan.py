"""Tokens that the router of a whole-layer pass has no expert for: their y is NaN, as the formula's, with or without
always-on experts, and the other tokens' results are those of a pass without them."""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _layer(N, m, d, f, typ, shared, seed=3):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.05).to(typ).cuda()  # noqa: E731
    W = [mk(N, f, d), mk(N, f, d), mk(N, d, f)]
    S = (mk(shared, f, d), mk(shared, f, d), mk(shared, d, f)) if shared else None
    return efa.Layer(*W, m=m, shared=S), mk(N, d), (torch.randn(N, generator=g) * 0.1).cuda(), g


@pytest.mark.parametrize("typ", [BF, F32])
@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("n,bad", [(1, [0]), (2, [1]), (6, [2, 5]), (20, [0, 19]), (33, list(range(33))), (40, [17])])
def test_a_token_of_nan_has_a_y_of_nan(typ, shared, n, bad):
    say("layer nan token", typ, shared, n)
    layer, wr, b, g = _layer(20, 4, 64, 96, typ, shared)
    good = [t for t in range(n) if t not in bad]
    x = torch.randn(n, 64, generator=g).to(typ).cuda()
    for kw in (dict(), dict(score="sigmoid"), dict(score="sigmoid", bias=b, renorm=False), dict(bias=b)):
        router = efa.Router(wr, **kw)
        i0, w0 = torch.empty(n, 4, dtype=torch.int32, device="cuda"), torch.empty(n, 4, device="cuda")
        want = efa.layer_pass(layer, router, x, ids=i0, w=w0)
        xn = x.clone()
        xn[bad, 5] = float("nan")
        ids, w = torch.empty_like(i0), torch.empty_like(w0)
        info = torch.zeros(3, dtype=torch.int32, device="cuda")
        y = efa.layer_pass(layer, router, xn, ids=ids, w=w, info=info)
        assert torch.isnan(y[bad]).all(), kw
        assert (ids[bad] == -1).all() and (w[bad] == 0).all() and info[1:].tolist() == [-5, 0]
        assert int(info[0]) == torch.unique(ids[good]).numel()
        assert torch.equal(ids[good], i0[good]) and torch.equal(w[good], w0[good])
        ref = efa.expert_dedup(layer, xn, ids, w).to(typ)
        assert torch.equal(y[good], ref[good]) and torch.isfinite(y[good]).all()
        assert ((y - want)[good].float().abs() <= 2.0 ** -7 * want[good].float().abs() + 1e-5).all()
        # added to what is there
        y0 = torch.randn(n, 64, generator=g).to(typ).cuda()
        acc = efa.layer_pass(layer, router, xn, y=y0.clone(), accumulate=True)
        assert torch.isnan(acc[bad]).all() and torch.isfinite(acc[good]).all()


@pytest.mark.parametrize("n", [1, 5])
def test_fewer_candidates_than_slots(n):
    """Logits of some experts NaN: a token keeps those that are left, and only a slot without one is empty."""
    say("layer few candidates", n)
    layer, wr, _, g = _layer(6, 4, 64, 96, BF, 0)
    wr[[0, 2, 5]] = float("nan")
    x = torch.randn(n, 64, generator=g).to(BF).cuda()
    for kw in (dict(), dict(score="sigmoid"), dict(renorm=False)):
        ids, w = torch.empty(n, 4, dtype=torch.int32, device="cuda"), torch.empty(n, 4, device="cuda")
        info = torch.zeros(3, dtype=torch.int32, device="cuda")
        y = efa.layer_pass(layer, efa.Router(wr, **kw), x, ids=ids, w=w, info=info)
        assert (ids[:, :3].sort(1).values == torch.tensor([1, 3, 4], device="cuda")).all()
        assert (ids[:, 3] == -1).all() and (w[:, 3] == 0).all() and (w[:, :3] > 0).all() and int(info[1]) == -5
        assert torch.isfinite(y).all() and torch.equal(y, efa.expert_dedup(layer, x, ids, w).to(BF))


def test_ids_of_a_caller_add_nothing():
    """The expert calls by themselves are as they were: ids out of range add nothing, and y is 0 without a valid one."""
    layer, _, _, g = _layer(6, 2, 64, 96, F32, 0)
    x = torch.randn(3, 64, generator=g).cuda()
    ids = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    assert (efa.expert_dedup(layer, x, ids, w) == 0).all() and (efa.expert_perslot(layer, x, ids, w) == 0).all()
