"""Refusals of the calls on 8-bit integers, on the host: every bad argument is answered before
any launch (the pointers are never followed)."""
import ctypes

import pytest
import torch

import expert_ffn_amd as efa
from expert_ffn_amd import _abi, grouped

OK = 0x10000  # 256-byte aligned, never followed
BIG = 1 << 40
INVAL, DTYPE, SPACE = _abi.MOE_E_INVAL, _abi.MOE_E_DTYPE, _abi.MOE_E_WORKSPACE


def _desc(**kw):
    d = dict(N=8, m=2, d_model=64, d_ff=128, dtype=_abi.MOE_INT8, flags=0, n_shared=0)
    d.update(kw)
    return _abi.LayerDesc(*(d[k] for k in ("N", "m", "d_model", "d_ff", "dtype", "flags", "n_shared")))


def _calls(desc, n, only=("gate_up", "down", "pass"), **kw):
    L = _abi.lib()
    a = dict(w=OK, s=OK, x=OK, xs=OK, h=OK, hs=OK, ids=OK, rw=OK, y=OK, off=OK, sbe=OK, ws=OK, size=BIG)
    a.update(kw)
    dp = ctypes.byref(desc) if desc is not None else None
    W = ctypes.byref(_abi.Int8Weights(a["w"], a["w"], a["w"], a["s"], a["s"], a["s"]))
    f = {
        "gate_up": lambda: L.moe_grouped_gate_up_int8(dp, W, a["x"], a["xs"], n, a["off"], a["sbe"], a["h"], a["hs"],
                                                      a["ws"], a["size"], None),
        "down": lambda: L.moe_grouped_down_int8(dp, W, a["h"], a["hs"], a["ids"], a["rw"], n, a["off"], a["sbe"], a["y"],
                                                a["ws"], a["size"], None),
        "pass": lambda: L.moe_expert_grouped_int8(dp, W, a["x"], a["ids"], a["rw"], n, a["y"], None, a["ws"], a["size"], None)}
    return {k: f[k]() for k in only}


@pytest.mark.parametrize("change,n,want", [
    (dict(N=0), 4, INVAL), (dict(N=1025), 4, INVAL), (dict(m=0), 4, INVAL), (dict(m=9), 4, INVAL),
    (dict(N=1024, m=257), 4, INVAL), (dict(), 0, INVAL), (dict(), -1, INVAL), (dict(), (1 << 21) + 1, INVAL),
    (dict(d_model=72), 4, DTYPE), (dict(d_ff=100), 4, DTYPE), (dict(d_model=0), 4, DTYPE), (dict(d_ff=-16), 4, DTYPE),
    (dict(d_model=65552), 4, INVAL), (dict(d_ff=65552), 4, INVAL), (dict(flags=8), 4, INVAL),
    (dict(flags=_abi.MOE_FLAG_WDOWN_PACKED), 4, INVAL), (dict(n_shared=1), 4, INVAL), (dict(n_shared=-1), 4, INVAL),
    (dict(flags=_abi.MOE_FLAG_TILED, d_model=80), 4, INVAL), (dict(flags=_abi.MOE_FLAG_TILED, d_ff=144), 4, INVAL),
    (dict(dtype=_abi.MOE_FP8), 4, DTYPE), (dict(dtype=_abi.MOE_BF16), 4, DTYPE), (dict(dtype=3), 4, DTYPE),
])
def test_sizes_and_flags(change, n, want):
    desc = _desc(**change)
    assert set(_calls(desc, n).values()) == {want}
    if desc.dtype == _abi.MOE_INT8:
        assert _abi.lib().moe_grouped_workspace_bytes(ctypes.byref(desc), n) == 0
        assert _abi.lib().moe_grouped_square(ctypes.byref(desc), n, 0) == want


def test_other_calls_refuse_the_type():
    L = _abi.lib()
    W = _abi.LayerWeights(OK, OK, OK)
    d = _desc()
    for f in (L.moe_expert_perslot, L.moe_expert_dedup):
        assert f(ctypes.byref(d), ctypes.byref(W), OK, OK, OK, 4, OK, None, OK, BIG, None) == DTYPE
    assert L.moe_expert_grouped(ctypes.byref(d), ctypes.byref(W), OK, OK, OK, 4, OK, None, OK, BIG, None) == DTYPE
    assert L.moe_workspace_bytes(ctypes.byref(d), 4, 0) == 0
    assert set(_calls(None, 4).values()) == {INVAL}


def test_pointers_and_workspace():
    d = _desc()
    L = _abi.lib()
    need = L.moe_grouped_workspace_bytes(ctypes.byref(d), 4)
    assert need > 0 and need % 256 == 0
    used = {"w": "gate_up down pass", "s": "gate_up down pass", "x": "gate_up pass", "xs": "gate_up", "h": "gate_up down",
            "hs": "gate_up down", "ids": "down pass", "rw": "down pass", "y": "down pass", "off": "gate_up down",
            "sbe": "gate_up down", "ws": "gate_up down pass"}
    used = {k: v.split() for k, v in used.items()}
    for name, where in used.items():
        assert set(_calls(d, 4, where, **{name: None}).values()) == {INVAL}, name
    for name, off in (("w", 8), ("x", 8), ("h", 8), ("y", 8), ("ws", 8), ("s", 2), ("xs", 2), ("hs", 2)):  # misaligned
        assert set(_calls(d, 4, used[name], **{name: OK + off}).values()) == {INVAL}, name
    assert set(_calls(d, 4, size=need - 1).values()) == {SPACE}
    sizes = [L.moe_grouped_workspace_bytes(ctypes.byref(d), n) for n in range(1, 300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("N,m,d,f", [(1, 1, 4096, 1024), (4, 2, 2048, 512), (8, 2, 576, 640), (128, 8, 2048, 768), (1024, 1, 16, 16), (8, 2, 4096, 14336)])
def test_a_longer_pass_needs_no_less(N, m, d, f):
    L = _abi.lib()
    desc = _desc(N=N, m=m, d_model=d, d_ff=f)
    sizes = [L.moe_grouped_workspace_bytes(ctypes.byref(desc), n) for n in list(range(1, 200)) + list(range(200, 9000, 61))]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_where_square_tiles_begin():
    """From 12 slots an expert, and in small layers from the rows x columns that make up for the compute units
    without a tile."""
    L = _abi.lib()
    for N, m, d, f, mat, first in ((128, 8, 2048, 768, 0, 12 * 128), (128, 8, 2048, 768, 1, 12 * 128),
                                   (16, 2, 1024, 512, 0, 2588), (16, 2, 1024, 512, 1, 2295), (1, 1, 4096, 1024, 0, 943)):
        desc = _desc(N=N, m=m, d_model=d, d_ff=f)
        n = -(-first // m)
        assert [L.moe_grouped_square(ctypes.byref(desc), k, mat) for k in (n - 1, n)] == [0, 1], (N, d, f, mat)
    # contractions of up to three units never
    assert L.moe_grouped_square(ctypes.byref(_desc(N=1, m=1, d_model=384, d_ff=4096)), 1 << 20, 0) == 0


def test_rows():
    L = _abi.lib()
    for f, order in ((L.moe_quant_rows_int8, lambda x, q, s, r, K: (x, r, K, q, s)),
                     (L.moe_dequant_rows_int8, lambda x, q, s, r, K: (q, s, r, K, x))):
        for bad, want in (((None, OK, OK, 4, 64), INVAL), ((OK, None, OK, 4, 64), INVAL), ((OK, OK, None, 4, 64), INVAL),
                          ((OK + 2, OK, OK, 4, 64), INVAL), ((OK, OK + 8, OK, 4, 64), INVAL), ((OK, OK, OK + 2, 4, 64), INVAL),
                          ((OK, OK, OK, 0, 64), INVAL), ((OK, OK, OK, (1 << 26) + 1, 64), INVAL), ((OK, OK, OK, -1, 64), INVAL),
                          ((OK, OK, OK, 4, 65552), INVAL), ((OK, OK, OK, 4, 8), DTYPE), ((OK, OK, OK, 4, 24), DTYPE),
                          ((OK, OK, OK, 4, 0), DTYPE), ((OK, OK, OK, 4, -16), DTYPE)):
            assert f(*order(*bad), None) == want, bad


def test_tiled_copies():
    L = _abi.lib()
    for kw in (dict(d_model=80), dict(d_ff=144), dict(d_model=0)):
        assert L.moe_pack_tiled(ctypes.byref(_desc(**kw)), OK, OK + (1 << 30), 0, None) == INVAL
    assert L.moe_pack_tiled(ctypes.byref(_desc()), OK, OK + 16, 0, None) == INVAL  # overlapping
    assert L.moe_pack_tiled(ctypes.byref(_desc()), OK, OK + (1 << 30), 2, None) == INVAL


def test_python_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        efa.quant_rows(x, dtype=torch.int8)  # not on the device
    for bad in (torch.uint8, torch.bfloat16, torch.float8_e5m2):
        with pytest.raises(TypeError):
            efa.quant_rows(x, dtype=bad)
        with pytest.raises(TypeError):
            efa.quant_weights(x, dtype=bad)
    with pytest.raises(ValueError):
        efa.dequant_rows(efa.Quantized(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)))
    with pytest.raises(ValueError):
        efa.Int8Layer((x, x), (x, x), (x, x, x), m=1)
    with pytest.raises(TypeError):
        grouped._check_codes(torch.float16)
