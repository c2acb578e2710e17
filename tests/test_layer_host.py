"""Refusals of the whole-layer pass on the host: every bad argument is answered before any launch
(the pointers are never followed)."""
import ctypes

import pytest
import torch

import expert_ffn_amd as efa
from expert_ffn_amd import _abi

OK = 0x10000  # 256-byte aligned, never followed
BIG = 1 << 40
INVAL, DTYPE, SPACE = _abi.MOE_E_INVAL, _abi.MOE_E_DTYPE, _abi.MOE_E_WORKSPACE


def _desc(**kw):
    d = dict(N=8, m=2, d_model=64, d_ff=128, dtype=_abi.MOE_BF16, flags=0, n_shared=0)
    d.update(kw)
    return _abi.LayerDesc(*(d[k] for k in ("N", "m", "d_model", "d_ff", "dtype", "flags", "n_shared")))


def _call(desc, n=4, score=0, **kw):
    a = dict(gate=OK, up=OK, down=OK, sg=OK, su=OK, sd=OK, wr=OK, bias=None, x=OK, y=OK, ids=None, w=None, info=None, ws=OK,
             size=BIG)
    a.update(kw)
    W = _abi.LayerWeights(a["gate"], a["up"], a["down"], a["sg"], a["su"], a["sd"])
    R = _abi.RouterDesc(a["wr"], a["bias"], score, 1, 1.0)
    return _abi.lib().moe_layer_pass(None if desc is None else ctypes.byref(desc), ctypes.byref(W), ctypes.byref(R), a["x"],
                                     n, a["y"], a["ids"], a["w"], a["info"], a["ws"], a["size"], None)


@pytest.mark.parametrize("change,n,want", [
    (dict(N=0), 4, INVAL), (dict(N=1025), 4, INVAL), (dict(m=0), 4, INVAL), (dict(m=9), 4, INVAL), (dict(), 0, INVAL),
    (dict(), -3, INVAL), (dict(), 65, INVAL), (dict(N=128, m=8), 33, INVAL), (dict(d_model=60), 4, DTYPE),
    (dict(d_ff=100), 4, DTYPE), (dict(dtype=_abi.MOE_FP8), 4, DTYPE), (dict(dtype=_abi.MOE_INT8), 4, DTYPE),
    (dict(dtype=3), 4, DTYPE), (dict(flags=8), 4, INVAL), (dict(flags=6), 4, INVAL), (dict(n_shared=17), 4, INVAL),
    (dict(n_shared=-1), 4, INVAL), (dict(d_model=16392), 4, INVAL), (dict(flags=_abi.MOE_FLAG_TILED, d_ff=144), 4, INVAL)])
def test_sizes(change, n, want):
    d = _desc(**change)
    assert _call(d, n) == want
    assert _abi.lib().moe_pass_workspace_bytes(ctypes.byref(d), n) == 0


def test_pointers_scores_and_workspace():
    d = _desc()
    L = _abi.lib()
    need = L.moe_pass_workspace_bytes(ctypes.byref(d), 4)
    assert need > L.moe_workspace_bytes(ctypes.byref(d), 4, 1)
    for name in ("gate", "up", "down", "wr", "x", "y", "ws"):
        assert _call(d, **{name: None}) == INVAL, name
        assert _call(d, **{name: OK + 8}) == INVAL, name
    for name in ("bias", "ids", "w", "info"):
        assert _call(d, **{name: OK + 2}) == INVAL, name
    for score in (-1, 2):
        assert _call(d, score=score) == INVAL
    sh = _desc(n_shared=1)
    for name in ("sg", "su", "sd"):
        assert _call(sh, **{name: None}) == INVAL and _call(sh, **{name: OK + 8}) == INVAL, name
    assert _call(d, size=256) == SPACE
    assert _call(None) == INVAL
    assert L.moe_pass_workspace_bytes(None, 4) == 0
    for kw in (dict(), dict(n_shared=2), dict(N=1024, m=4, d_model=2048), dict(N=128, m=4, d_model=2048, d_ff=768)):
        sizes = [L.moe_pass_workspace_bytes(ctypes.byref(_desc(**kw)), n) for n in range(1, 61)]
        assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:])), kw


def test_python_refuses():
    with pytest.raises(ValueError):
        efa.Router(torch.zeros(4, 8))  # not on the device
    with pytest.raises(ValueError):
        efa.Router(torch.zeros(4, 8), score="none")
    with pytest.raises(TypeError):
        efa.layer_pass(None, None, torch.zeros(1, 8))
    with pytest.raises(TypeError):
        efa.pass_workspace(3, 4)
