"""The router of a whole-layer pass on logits that fp32 holds exactly (``routing_cases``): ids to the last tie and
weights to a few roundings, at widths where the contraction is cut into parts that meet in memory."""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say
from .routing_cases import FORMS, check, form, problem

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("N,m,d,typ", [
    (40, 5, 1024, BF), (64, 6, 2048, BF), (65, 3, 2056, BF), (128, 8, 2048, BF), (129, 8, 4104, BF), (256, 8, 7168, BF),
    (257, 8, 2048, BF), (384, 8, 7168, BF), (1024, 8, 4096, BF), (1021, 16, 8192, BF), (5, 5, 16384, BF), (16, 4, 16384, F32),
    (64, 6, 520, F32), (300, 16, 2048, F32), (1024, 8, 1032, F32)])
def test_ids_and_weights(N, m, d, typ):
    zero = lambda *s: torch.zeros(*s, dtype=typ, device="cuda")  # noqa: E731
    layer = efa.Layer(zero(N, 8, d), zero(N, 8, d), zero(N, d, 8), m=m)
    ws = layer.pass_workspace(256 // m if m > 4 else 64)
    for i in range(len(FORMS)):
        f = form(i, N)
        for n in (1, 2, 3, 4, 5, 8, 33):
            if n * m > 256:
                continue
            say("layer exact logits", N, m, d, typ, i, n)
            x, w, l = problem(N, d, n, 100 * i + n)
            dev = dict(f, bias=f["bias"].cuda()) if "bias" in f else f
            ids = torch.full((n, m), -7, dtype=torch.int32, device="cuda")
            wt = torch.full((n, m), 7.0, device="cuda")
            efa.layer_pass(layer, efa.Router(w.to(typ).cuda(), **dev), x.to(typ).cuda(), ids=ids, w=wt, ws=ws)
            check(ids, wt, l, m, **f)


@pytest.mark.parametrize("N", [16, 63, 64, 65, 128, 129, 256])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 6])
def test_selection_of_any_number(N, n):
    """By rounds or by rank, as the number of experts to take, the tokens and the experts have it."""
    zero = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    W = (zero(N, 8, 1024), zero(N, 8, 1024), zero(N, 1024, 8))
    for m in (1, 7, 8, 9, 12, 13, 16, 17, 18, 30, 31, 42, 43, 55, 56, 64, 65, 128, 256):
        if m > N or n * m > 256:
            continue
        layer = efa.Layer(*W, m=m)
        for i in (0, 2, 3):
            say("layer selection", N, n, m, i)
            f = form(i, N)
            x, w, l = problem(N, 1024, n, 10 * i + n)
            dev = dict(f, bias=f["bias"].cuda()) if "bias" in f else f
            ids = torch.full((n, m), -7, dtype=torch.int32, device="cuda")
            wt = torch.full((n, m), 7.0, device="cuda")
            efa.layer_pass(layer, efa.Router(w.to(BF).cuda(), **dev), x.to(BF).cuda(), ids=ids, w=wt)
            check(ids, wt, l, m, **f)
