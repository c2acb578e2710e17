"""Calls as a server makes them: passes of several lengths on several streams at once, each with its workspace, and
captured passes of several lengths that share one workspace and are replayed in turn, between eager ones.  Results are
bit for bit those of the calls one by one."""
import pytest
import torch

import expert_ffn_amd as efa

from .gpu_cases import say
from .test_gpu_int8 import Case, _check_pass, _ids, _randn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _layer():
    mk = lambda seed, *s: (_randn(seed, *s) * 0.05).to(BF).cuda()  # noqa: E731
    layer = efa.Layer(mk(1, 64, 128, 512), mk(2, 64, 128, 512), mk(3, 64, 512, 128), m=4)
    return layer, efa.Router(mk(4, 64, 512), score="sigmoid", bias=_randn(5, 64).cuda() * 0.1)


def _calls(kind, lengths):
    """(call(i, y, ws, stream), outputs one by one, workspace of n)"""
    if kind == "layer":
        layer, router = _layer()
        xs = [_randn(n, n, 512).to(BF).cuda() for n in lengths]
        call = lambda i, **kw: efa.layer_pass(layer, router, xs[i], **kw)  # noqa: E731
        space = layer.pass_workspace
    else:
        case = Case(16, 4, 576, 640)
        xs = [_randn(n, n, 576).to(BF).cuda() for n in lengths]
        routed = [_ids(n, n, 4, 16) for n in lengths]
        call = lambda i, **kw: efa.expert_grouped(case.layer, xs[i], *routed[i], **kw)  # noqa: E731
        space = case.layer.grouped_workspace
    return call, [call(i) for i in range(len(lengths))], space


@pytest.mark.parametrize("kind,lengths", [("layer", (1, 3, 20, 60)), ("int8", (9, 700, 40, 1300))])
def test_streams_at_once(kind, lengths):
    say("at once", kind)
    call, want, space = _calls(kind, lengths)
    streams = [torch.cuda.Stream() for _ in lengths]
    spaces = [space(n) for n in lengths]
    ys = [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            call(i, y=ys[i], ws=spaces[i], stream=st)
    torch.cuda.synchronize()
    for i in range(len(lengths)):
        assert torch.equal(ys[i], want[i]), lengths[i]


@pytest.mark.parametrize("kind,lengths", [("layer", (60, 1, 3, 20)), ("int8", (1300, 9, 40, 700))])
def test_captured_passes_that_share_a_workspace(kind, lengths):
    say("captured, one workspace", kind)
    call, want, space = _calls(kind, lengths)
    ws, ys, graphs = space(max(lengths)), [torch.empty_like(y) for y in want], []
    torch.cuda.synchronize()
    for i in range(len(lengths)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, y=ys[i], ws=ws)
    for r in range(4):
        for y in ys:
            y.zero_()
        for i in range(len(lengths)):
            graphs[(i + r) % len(lengths)].replay()
        assert torch.equal(call(r, ws=ws), want[r])
        torch.cuda.synchronize()
        for i in range(len(lengths)):
            assert torch.equal(ys[i], want[i]), (r, lengths[i])


@pytest.mark.parametrize("N,m,d,f,n", [(128, 100, 576, 640, 200), (128, 100, 576, 640, 3), (200, 130, 448, 512, 90),
                                       (70, 65, 256, 144, 300)])
def test_int8_passes_of_many_slots_a_token(N, m, d, f, n):
    """More slots a token than a wave has lanes, ids that are not valid and an id more than once among them."""
    say("int8 many slots", N, m, n)
    case = Case(N, m, d, f)
    ids, w = _ids(n, n, m, N)
    ids[:, m // 2] = -1
    ids[n // 2] = torch.randint(-5, N + 5, (m,), generator=torch.Generator().manual_seed(m)).int().cuda()
    _check_pass(case, _randn(3, n, d).to(BF).cuda(), ids, w, "slots %s" % ((N, m, d, f, n),))
