"""Logits that are not finite in ``router_topk``, in both of its selection kernels (by rank up to 256 experts and 64
slots, else by rounds): a NaN logit is never selected and shifts no other, a slot left without a candidate gets id
-1 and weight 0."""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _want(logits, m):
    """(ids, weights in 64 bits) by the selection rule on one token's logits."""
    left = sorted((e for e in range(len(logits)) if logits[e] == logits[e]), key=lambda e: (-logits[e], e))[:m]
    z = torch.tensor([logits[e] for e in left], dtype=torch.float64)
    return left + [-1] * (m - len(left)), z.softmax(0).tolist() + [0.0] * (m - len(left))


@pytest.mark.parametrize("typ", [BF, F32])
@pytest.mark.parametrize("N,m,n", [(8, 2, 1), (8, 8, 5), (64, 6, 17), (256, 64, 3), (256, 65, 3), (257, 4, 2), (1024, 8, 7)])
def test_nan_logits_are_never_selected(typ, N, m, n):
    say("router nan", typ, N, m, n)
    g = torch.Generator().manual_seed(N + m)
    wr = (torch.randn(N, 64, generator=g) / 8).to(typ).cuda()
    x = torch.randn(n, 64, generator=g).to(typ).cuda()
    plain = efa.router_topk(wr, x, m)
    for bad in ([0], [N - 1, 3], list(range(0, N, 2)), list(range(N - 1)), list(range(N))):
        wb = wr.clone()
        wb[bad] = float("nan")
        xb = x.clone()
        if n > 2:
            xb[1, 7] = float("nan")  # a token without any logit
        out = efa.router_topk(wb, xb, m)
        logits = out.logits.cpu()
        keep = [e for e in range(N) if e not in set(bad)]
        rows = [t for t in range(n) if not (n > 2 and t == 1)]
        assert torch.isnan(logits[:, bad]).all()
        assert torch.equal(logits[rows][:, keep], plain.logits.cpu()[rows][:, keep])
        for t in range(n):
            ids, w = _want(logits[t].tolist(), m)
            assert out.ids[t].tolist() == ids, (t, len(bad))
            # the exponential, the sum and the division: a few 2^-23 each
            assert ((out.w[t].cpu().double() - torch.tensor(w)).abs() <= 2.0 ** -19 * torch.tensor(w)).all(), (t, len(bad))


@pytest.mark.parametrize("N", [40, 300])
def test_a_routed_pass_skips_what_has_no_expert(N):
    say("router nan pass", N)
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.05).to(BF).cuda()  # noqa: E731
    layer = efa.Layer(mk(N, 96, 64), mk(N, 96, 64), mk(N, 64, 96), m=4)
    wr, x = mk(N, 64), torch.randn(5, 64, generator=g).to(BF).cuda()
    want = efa.router_topk(wr, x, 4)
    y0 = efa.expert_dedup(layer, x, want.ids, want.w)
    x[3, 0] = float("nan")
    out = efa.router_topk(wr, x, 4)
    info = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = efa.expert_dedup(layer, x, out.ids, out.w, info=info)
    rest = [0, 1, 2, 4]
    assert out.ids[3].tolist() == [-1] * 4 and int(info[1]) == -5
    assert torch.equal(out.ids[rest], want.ids[rest]) and torch.equal(out.w[rest], want.w[rest])
    assert ((y - y0)[rest].abs() <= 2.0 ** -18 * (1 + y0[rest].abs())).all()  # (grouped otherwise: sums in another order)
