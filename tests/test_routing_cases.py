"""The check of a router's ids and weights by itself: it passes what fp32 gives for the right logits, and refuses logits
rounded to bf16, a chunk or a part of the contraction left out or met twice, and another token's logits."""
import pytest
import torch

from .routing_cases import FORMS, check, form, problem

N, M, TOKENS = 64, 6, 5


def _route(l, score="softmax", bias=None, renorm=True, scale=1.0):
    """ids and weights in fp32, from logits in fp32."""
    l = l.float()
    s = l.softmax(1) if score == "softmax" else l.sigmoid()
    key = l if bias is None else s + bias
    ids = torch.sort(-key, dim=1, stable=True).indices[:, :M]
    w = torch.gather(s, 1, ids)
    return ids.int(), (w / w.sum(1, keepdim=True) if renorm else w) * scale


@pytest.mark.parametrize("d", [2048, 4096, 16384])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_the_check(i, d):
    f = form(i, N)
    x, w, l = problem(N, d, TOKENS, d + i)
    assert torch.equal(x.bfloat16().double(), x) and torch.equal(w.bfloat16().double(), w)
    assert torch.equal((x.float() @ w.float().T).double(), l)  # in fp32 too, whatever its order
    check(*_route(l, **f), l, M, **f)
    part = d // 8
    wrong = {
        "bf16": l.bfloat16().double(),
        "a partial sum in bf16": x[:, :part] @ w[:, :part].T + (x[:, part:] @ w[:, part:].T).bfloat16().double(),
        "last chunk": x[:, :-8] @ w[:, :-8].T,
        "a part": x[:, part:] @ w[:, part:].T,
        "a part twice": l + x[:, :part] @ w[:, :part].T,
        "another token": l.roll(1, 0),
        "another expert": l.roll(1, 1),
    }
    for name, bad in wrong.items():
        with pytest.raises(AssertionError):
            check(*_route(bad, **f), l, M, **f)
            pytest.fail("not refused: " + name, pytrace=False)


def test_the_check_refuses_wrong_ties_and_weights():
    l = torch.zeros(1, 8, dtype=torch.float64)
    w = torch.full((1, 2), 0.5)
    check(torch.tensor([[0, 1]]), w, l, 2)
    for ids in ([[1, 0]], [[0, 2]]):
        with pytest.raises(AssertionError):
            check(torch.tensor(ids), w, l, 2)
    with pytest.raises(AssertionError):
        check(torch.tensor([[0, 1]]), w * (1 + 2.0 ** -16), l, 2)
