"""Routing problems whose logits are whole numbers of one power of two, so that fp32 holds every partial sum of them
exactly, in any order and grouping: a router's logits are then known to the last bit, and its ids, ties included, with them.

x and w are whole numbers up to 4 (w times 2^-k): products up to 16, sums of d <= 16384 of them below 2^18.

Tolerance of a weight, relative, in half steps of fp32 (2^-24): the difference l - top is exact; an exponential 4, in the
numerator and in the sum; the sum of N <= 1024 of them in a lane's 16 and six across lanes 22, a reciprocal or division
and the factor 2 each, once more where the selected are renormalised: below 64 together, 2^-18.
"""
import math

import torch

TOL = 2.0 ** -18


def problem(N, d, n, seed):
    """(x [n][d], w [N][d], logits [n][N]) in float64; bf16 and fp32 hold x and w exactly."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-4, 5, (n, d), generator=g).double()
    k = round(math.log2(20 / 3 * math.sqrt(d) / 1.5))  # logits of about 1.5
    w = torch.randint(-4, 5, (N, d), generator=g).double() * 2.0 ** -k
    return x, w, x @ w.T


def scores(l, score):
    return l.softmax(1) if score == "softmax" else l.sigmoid()


def check(ids, w, l, m, score="softmax", bias=None, renorm=True, scale=1.0):
    """ids and w of a router against logits l that it has to have met exactly.  With a bias the keys s + b are
    off by TOL s and one rounding, and an expert is right if no later one beats it by more."""
    ids, w, s = ids.cpu().long(), w.cpu().double(), scores(l, score)
    n, N = l.shape
    if bias is None:
        assert torch.equal(ids, torch.sort(-l, dim=1, stable=True).indices[:, :m]), "ids"
    else:
        key = s + bias.double()
        off = TOL * s + 2.0 ** -24 * key.abs()
        left = torch.ones_like(key, dtype=torch.bool)
        rows = torch.arange(n)
        for j in range(m):
            e = ids[:, j]
            assert ((e >= 0) & (e < N)).all() and left[rows, e.clamp(0, N - 1)].all(), "ids"
            left[rows, e] = False
            ahead = torch.where(left, key - off, torch.full_like(key, -math.inf)).amax(1)
            assert (key[rows, e] + off[rows, e] >= ahead).all(), "ids"
    v = torch.gather(s, 1, ids)
    if renorm:
        v = v / v.sum(1, keepdim=True)
    v = v * scale
    assert ((w - v).abs() <= TOL * v.abs()).all(), "weights: %.3g" % float(((w - v).abs() / v.abs()).max())


FORMS = [dict(), dict(renorm=False, scale=2.5), dict(score="sigmoid"), dict(score="sigmoid", bias=True, scale=2.5),
         dict(bias=True), dict(score="sigmoid", bias=True, renorm=False), dict(bias=True, renorm=False)]


def form(i, N):
    """Form i with its bias [N] float32."""
    f = dict(FORMS[i])
    if f.pop("bias", False):
        f["bias"] = torch.randn(N, generator=torch.Generator().manual_seed(N)) * 0.05
    return f
