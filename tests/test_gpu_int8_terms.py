"""Down products of int8 layers on square tiles: what a token's terms keep of their bits, whatever stands beside them.

A term w_tj s_h s_c sum goes from the product to the token's sum in fp16 as the whole number `sum` times a power of
two: half a step of fp16, 2^-11 of the term, at every scale of the row, of the column and of the columns beside it.
Around it fp32: the sum's conversion, two scales, the weight, 2^-24 each, and the m additions, 2^-24 of what is added
up each.  y is then rounded to bf16: 2^-8.
"""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say

pytestmark = pytest.mark.gpu

I8 = torch.int8


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _codes(g, *s):
    return torch.randint(-127, 128, s, generator=g, dtype=torch.int32).to(I8)


def _case(N, m, d, K, n, layout, ratios, seed=3):
    """(layer, h, ids, w, grouping) of n tokens, whose W_down has column c's scale at ratios[c % len(ratios)]."""
    g = _gen(seed)
    any_q = (torch.zeros(N, K, d, dtype=I8, device="cuda"), torch.ones(N, K, device="cuda"))
    wd = _codes(g, N, d, K)
    wd[:, 5::7, 1:] = 0  # columns whose sums are one product
    sd = torch.tensor(ratios, dtype=torch.float64).repeat(d // len(ratios) + 1)[:d] * (0.5 + torch.rand(N, d, generator=g).double())
    layer = efa.Int8Layer(any_q, any_q, (wd.cuda(), sd.float().cuda()), m=m)
    if layout == "tiled":
        layer = layer.tiled_copy()
    ids = torch.rand(n, N, generator=g).argsort(1)[:, :m].to(torch.int32).cuda().contiguous()
    w = torch.randn(n, m, generator=g).cuda()
    h = efa.Quantized(_codes(g, n * m, K).cuda(), torch.exp(torch.randn(n * m, generator=g)).cuda())
    return layer, wd.cuda(), sd.float().cuda(), h, ids, w, efa.group_slots(ids, N)


def _exact(wd, sd, h, ids, w, g):
    n, m = ids.shape
    row = torch.empty(n * m, dtype=torch.long, device="cuda")
    row[g.slot_by_expert.long()] = torch.arange(n * m, device="cuda")
    y = torch.zeros(n, sd.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for e in range(sd.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        r = row[t * m + j]
        o = (h.q[r].double() @ wd[e].double().T) * sd[e].double() * h.scale[r].double()[:, None] * w[t, j].double()[:, None]
        y.index_add_(0, t, o)
        mag.index_add_(0, t, o.abs())
    return y, mag


WIDE = [1.0, 2.0 ** -30, 2.0 ** -9, 2.0 ** 12, 2.0 ** -24, 2.0 ** -17, 2.0 ** -45, 2.0 ** -3]


@pytest.mark.parametrize("layout", ["plain", "tiled"])
@pytest.mark.parametrize("N,m,d,K,n", [(2, 1, 576, 512, 9000), (4, 3, 320, 1024, 3001), (2, 2, 1024, 14336, 700),
                                       (2, 1, 1024, 65536, 1200)])
@pytest.mark.parametrize("ratios", [[1.0], WIDE])
def test_terms_keep_eleven_bits(N, m, d, K, n, layout, ratios):
    say("int8 terms", N, m, d, K, n, layout, len(ratios))
    layer, wd, sd, h, ids, w, g = _case(N, m, d, K, n, layout, ratios)
    assert efa.grouped_square(layer, n, efa.MOE_MAT_DOWN)
    y = efa.grouped_down(layer, h, ids, w, g).double()
    want, mag = _exact(wd, sd, h, ids, w, g)
    tol = (2.0 ** -11 + (4 + m) * 2.0 ** -24) * 1.001 * mag  # (1.001: products of the errors)
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    over = (y - want).abs() - tol
    assert (over <= 0).all(), "column %d, %.3g of the terms" % (int(over.amax(0).argmax()),
                                                                float(((y - want).abs() / mag.clamp(min=1e-300)).max()))


def test_the_largest_codes_of_either_sign():
    """Codes of -128 too, which quantisation does not make: sums of 2^14 K, over the longest contraction 2^30."""
    say("int8 terms largest")
    N, d, K, n = 2, 1024, 65536, 1200
    wd = torch.full((N, d, K), -128, dtype=I8, device="cuda")
    sd = torch.full((N, d), 2.0 ** -6, device="cuda")
    any_q = (torch.zeros(N, K, d, dtype=I8, device="cuda"), torch.ones(N, K, device="cuda"))
    layer = efa.Int8Layer(any_q, any_q, (wd, sd), m=1)
    assert efa.grouped_square(layer, n, efa.MOE_MAT_DOWN)
    ids = (torch.arange(n, dtype=torch.int32, device="cuda") % 2)[:, None].contiguous()
    h = efa.Quantized(torch.full((n, K), -128, dtype=I8, device="cuda"), torch.full((n,), 2.0 ** -10, device="cuda"))
    y = efa.grouped_down(layer, h, ids, torch.ones(n, 1, device="cuda"), efa.group_slots(ids, N))
    assert (y == 2.0 ** 14).all()  # 2^30 2^-16, a power of two in every step
