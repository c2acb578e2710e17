"""Refusals of the grouped calls, on the host: every bad argument is answered before any
launch (the pointers are never followed)."""
import ctypes

import pytest
import torch

import expert_ffn_amd as efa
from expert_ffn_amd import _abi, grouped

OK = 0x10000  # 256-byte aligned, never followed
BIG = 1 << 40


def _desc(**kw):
    d = dict(N=8, m=2, d_model=64, d_ff=128, dtype=_abi.MOE_BF16, flags=0, n_shared=0)
    d.update(kw)
    return _abi.LayerDesc(*(d[k] for k in ("N", "m", "d_model", "d_ff", "dtype", "flags", "n_shared")))


def _calls(desc, n, only=("gate_up", "down", "pass"), **kw):
    """The statuses of the entry points that take a descriptor of this type (those of
    ``only``, each of which has to refuse the arguments)."""
    L = _abi.lib()
    a = dict(w=OK, s=OK, x=OK, xs=OK, h=OK, hs=OK, ids=OK, rw=OK, y=OK, off=OK, sbe=OK, ws=OK, size=BIG)
    a.update(kw)
    dp = ctypes.byref(desc) if desc is not None else None
    if desc is not None and desc.dtype == _abi.MOE_FP8:
        W = _abi.Fp8Weights(a["w"], a["w"], a["w"], a["s"], a["s"], a["s"])
        f = {
            "gate_up": lambda: L.moe_grouped_gate_up_fp8(dp, ctypes.byref(W), a["x"], a["xs"], n, a["off"], a["sbe"],
                                                         a["h"], a["hs"], a["ws"], a["size"], None),
            "down": lambda: L.moe_grouped_down_fp8(dp, ctypes.byref(W), a["h"], a["hs"], a["ids"], a["rw"], n, a["off"],
                                                   a["sbe"], a["y"], a["ws"], a["size"], None),
            "pass": lambda: L.moe_expert_grouped_fp8(dp, ctypes.byref(W), a["x"], a["ids"], a["rw"], n, a["y"], None,
                                                     a["ws"], a["size"], None)}
    else:
        W = _abi.LayerWeights(a["w"], a["w"], a["w"])
        f = {
            "gate_up": lambda: L.moe_grouped_gate_up(dp, ctypes.byref(W), a["x"], n, a["off"], a["sbe"], a["h"],
                                                     a["ws"], a["size"], None),
            "down": lambda: L.moe_grouped_down(dp, ctypes.byref(W), a["h"], a["ids"], a["rw"], n, a["off"], a["sbe"],
                                               a["y"], a["ws"], a["size"], None),
            "pass": lambda: L.moe_expert_grouped(dp, ctypes.byref(W), a["x"], a["ids"], a["rw"], n, a["y"], None,
                                                 a["ws"], a["size"], None)}
    return {k: f[k]() for k in only}


INVAL, DTYPE, SPACE = _abi.MOE_E_INVAL, _abi.MOE_E_DTYPE, _abi.MOE_E_WORKSPACE


@pytest.mark.parametrize("dtype", [_abi.MOE_BF16, _abi.MOE_FP8])
@pytest.mark.parametrize("change,n,want", [
    (dict(N=0), 4, INVAL), (dict(N=1025), 4, INVAL), (dict(m=0), 4, INVAL), (dict(m=9), 4, INVAL),
    (dict(N=1024, m=257), 4, INVAL), (dict(), 0, INVAL), (dict(), -1, INVAL), (dict(), (1 << 21) + 1, INVAL),
    (dict(d_model=60), 4, DTYPE), (dict(d_ff=100), 4, DTYPE), (dict(d_model=0), 4, DTYPE), (dict(d_ff=-16), 4, DTYPE),
    (dict(d_model=65552), 4, INVAL), (dict(d_ff=65552), 4, INVAL), (dict(flags=8), 4, INVAL),
    (dict(flags=_abi.MOE_FLAG_WDOWN_PACKED), 4, INVAL), (dict(n_shared=1), 4, INVAL), (dict(n_shared=-1), 4, INVAL),
    (dict(flags=_abi.MOE_FLAG_TILED, d_model=80), 4, INVAL), (dict(flags=_abi.MOE_FLAG_TILED, d_ff=144), 4, INVAL),
])
def test_sizes_and_flags(dtype, change, n, want):
    desc = _desc(dtype=dtype, **change)
    assert set(_calls(desc, n).values()) == {want}
    assert _abi.lib().moe_grouped_workspace_bytes(ctypes.byref(desc), n) == 0


def test_types():
    L = _abi.lib()
    for dtype in (_abi.MOE_F32, 3, 7, -1):
        assert set(_calls(_desc(dtype=dtype), 4).values()) == {DTYPE}
        assert L.moe_grouped_workspace_bytes(ctypes.byref(_desc(dtype=dtype)), 4) == 0
    assert set(_calls(None, 4).values()) == {INVAL}
    assert L.moe_grouped_workspace_bytes(None, 4) == 0
    # 8-bit rows are whole 16-byte pieces
    assert set(_calls(_desc(dtype=_abi.MOE_FP8, d_model=72), 4).values()) == {DTYPE}
    # the calls on verification passes do not take 8-bit layers
    W = _abi.LayerWeights(OK, OK, OK)
    d8 = _desc(dtype=_abi.MOE_FP8)
    for f in (L.moe_expert_perslot, L.moe_expert_dedup):
        assert f(ctypes.byref(d8), ctypes.byref(W), OK, OK, OK, 4, OK, None, OK, BIG, None) == DTYPE
    assert L.moe_workspace_bytes(ctypes.byref(d8), 4, 0) == 0


@pytest.mark.parametrize("dtype", [_abi.MOE_BF16, _abi.MOE_FP8])
def test_pointers_and_workspace(dtype):
    d = _desc(dtype=dtype)
    need = _abi.lib().moe_grouped_workspace_bytes(ctypes.byref(d), 4)
    assert need > 0 and need % 256 == 0
    used = {"w": "gate_up down pass", "x": "gate_up pass", "h": "gate_up down", "ids": "down pass", "rw": "down pass",
            "y": "down pass", "off": "gate_up down", "sbe": "gate_up down", "ws": "gate_up down pass"}
    if dtype == _abi.MOE_FP8:
        used.update(s="gate_up down pass", xs="gate_up", hs="gate_up down")
    used = {k: v.split() for k, v in used.items()}
    for name, where in used.items():
        assert set(_calls(d, 4, where, **{name: None}).values()) == {INVAL}, name
    for name in ("w", "x", "h", "y", "ws"):  # misaligned
        assert set(_calls(d, 4, used[name], **{name: OK + 8}).values()) == {INVAL}, name
    assert set(_calls(d, 4, used["ws"], size=need - 1).values()) == {SPACE}
    sizes = [_abi.lib().moe_grouped_workspace_bytes(ctypes.byref(d), n) for n in range(1, 300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_group_and_quant_refusals():
    L = _abi.lib()
    five = (OK,) * 5
    for n, m, N in ((0, 1, 8), (1, 0, 8), (1, 9, 8), (1, 1, 0), (1, 1, 1025), (1, 257, 1024), ((1 << 22) + 1, 1, 8)):
        assert L.moe_group_slots(OK, n, m, N, *five, OK, BIG, None) == INVAL
        assert L.moe_group_workspace_bytes(n, m, N) == 0
    need = L.moe_group_workspace_bytes(4096, 8, 128)
    assert L.moe_group_slots(OK, 1 << 19, 8, 128, *five, OK, 64, None) == SPACE
    assert L.moe_group_slots(OK, 4096, 8, 128, *five, OK + 16, need, None) == INVAL
    assert L.moe_group_slots(OK, 4096, 8, 128, *five, None, need, None) == INVAL
    for i in range(5):
        assert L.moe_group_slots(OK, 4, 2, 8, *(None if j == i else OK for j in range(5)), OK, BIG, None) == INVAL
    assert L.moe_group_slots(None, 4, 2, 8, *five, OK, BIG, None) == INVAL
    for f in (L.moe_quant_rows, L.moe_dequant_rows):
        order = (lambda x, q, s, r, K: (x, r, K, q, s)) if f is L.moe_quant_rows else (lambda x, q, s, r, K: (q, s, r, K, x))
        for bad, want in (((None, OK, OK, 4, 64), INVAL), ((OK, None, OK, 4, 64), INVAL), ((OK, OK, None, 4, 64), INVAL),
                          ((OK + 2, OK, OK, 4, 64), INVAL), ((OK, OK + 8, OK, 4, 64), INVAL), ((OK, OK, OK, 0, 64), INVAL),
                          ((OK, OK, OK, (1 << 22) + 1, 64), INVAL), ((OK, OK, OK, 4, 65552), INVAL),
                          ((OK, OK, OK, 4, 0), DTYPE), ((OK, OK, OK, 4, 24), DTYPE), ((OK, OK, OK, 4, -16), DTYPE)):
            assert f(*order(*bad), None) == want, bad
    for args, want in (((None, 1, 16, 16, OK, OK), INVAL), ((OK, 1, 16, 16, None, OK), INVAL),
                       ((OK, 1, 16, 16, OK, None), INVAL), ((OK, 0, 16, 16, OK, OK), INVAL),
                       ((OK, 1025, 16, 16, OK, OK), INVAL), ((OK, 1, 24, 16, OK, OK), DTYPE),
                       ((OK, 1, 16, 8, OK, OK), DTYPE), ((OK, 1, 65552, 16, OK, OK), INVAL),
                       ((OK + 8, 1, 16, 16, OK, OK), INVAL)):
        assert L.moe_quant_weights(*args, None) == want, args
    # tiling of codes: whole steps of 64
    for kw in (dict(d_model=96), dict(d_ff=32), dict(d_model=0)):
        assert L.moe_pack_tiled(ctypes.byref(_desc(dtype=_abi.MOE_FP8, **kw)), OK, OK + (1 << 30), 0, None) == INVAL


def test_python_refusals_without_a_gpu():
    """Tensors that are not on a device, of another type or class."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        efa.quant_rows(x)
    with pytest.raises(ValueError):
        efa.quant_weights(x[None])
    with pytest.raises(ValueError):
        efa.group_slots(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(TypeError):
        efa.dequant_rows(x)
    with pytest.raises(TypeError):
        efa.expert_grouped(object(), x, None, None)
    with pytest.raises(_abi.MoeError):
        efa.group_workspace(0, 1, 8, device="cpu")
    with pytest.raises(ValueError):
        efa.Fp8Layer((torch.zeros(2, 16, 16),), (x, x), (x, x), m=1)
    assert grouped._blocks(128) == 1 and grouped._blocks(129) == 2


@pytest.mark.parametrize("dtype", [_abi.MOE_BF16, _abi.MOE_FP8])
def test_a_longer_pass_needs_no_less(dtype):
    """The workspace of n tokens serves fewer, also where the grouping takes fewer and
    longer chunks for more slots (from 8193 and 65537 slots on)."""
    d = _desc(N=1024, m=1, d_model=16, d_ff=16, dtype=dtype)
    ns = [1, 2, 8191, 8192, 8193, 65535, 65536, 65537, 70000, 131072, 131073, 262144, 262145, 1 << 22]
    sizes = [_abi.lib().moe_grouped_workspace_bytes(ctypes.byref(d), n) for n in ns]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), sizes


@pytest.mark.parametrize("dtype", [_abi.MOE_BF16, _abi.MOE_FP8])
@pytest.mark.parametrize("N,m,d,f", [(2, 2, 512, 768), (64, 4, 1024, 640), (128, 8, 2048, 768), (8, 2, 4096, 14336)])
def test_a_longer_pass_needs_no_less_where_tiles_change(N, m, d, f, dtype):
    """Also where a longer pass takes other tiles, which hold their terms in other types."""
    desc = _desc(N=N, m=m, d_model=d, d_ff=f, dtype=dtype)
    sizes = [_abi.lib().moe_grouped_workspace_bytes(ctypes.byref(desc), n) for n in range(1, 24 * N // m + 24)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_which_tiles():
    """moe_grouped_square: square tiles from 8, 12 or 16 rows an expert, by type and tiles, for
    contractions of more than 384 bytes and matrices of 31 bits."""
    L = _abi.lib()

    def square(n, mat, **kw):
        return L.moe_grouped_square(ctypes.byref(_desc(**kw)), n, mat)
    G, D = _abi.MOE_MAT_GATE_UP, _abi.MOE_MAT_DOWN
    few = dict(N=8, m=2, d_model=512, d_ff=512)        # fewer tiles than two a compute unit
    many = dict(N=1000, m=2, d_model=512, d_ff=528)
    for dtype, least in ((_abi.MOE_BF16, 8), (_abi.MOE_FP8, 12)):
        for mat in (G, D):
            assert square(63, mat, dtype=dtype, **few) == 0 and square(64, mat, dtype=dtype, **few) == 1
            n = least * 1000 // 2
            assert square(n - 1, mat, dtype=dtype, **many) == 0 and square(n, mat, dtype=dtype, **many) == 1
    for dtype, es in ((_abi.MOE_BF16, 2), (_abi.MOE_FP8, 1)):
        short = dict(N=8, m=2, dtype=dtype, d_model=384 // es, d_ff=400 // es)
        assert square(4000, G, **short) == 0 and square(4000, D, **short) == 1
    assert square(4000, G, N=1, m=1, dtype=_abi.MOE_BF16, d_model=16384, d_ff=65408) == 0
    for bad in (dict(N=0), dict(m=9), dict(n_shared=1), dict(flags=8)):
        assert square(4, G, **{"dtype": _abi.MOE_BF16, **bad}) == INVAL
    assert square(0, G, dtype=_abi.MOE_BF16) == INVAL and square(4, 2, dtype=_abi.MOE_BF16) == INVAL
    assert square(4, G, dtype=_abi.MOE_F32) == DTYPE and square(4, G, dtype=_abi.MOE_BF16, d_ff=100) == DTYPE
    assert L.moe_grouped_square(None, 4, G) == INVAL


def test_sizes_beyond_an_int_are_refused():
    """A size that C's int does not hold is not taken for what its lowest bits say."""
    for n, m, N in (((1 << 32) + 1, 1, 8), (1, (1 << 32) + 1, 8), (1, 1, (1 << 32) + 8), (1 - (1 << 32), 1, 8)):
        with pytest.raises(_abi.MoeError):
            efa.group_workspace(n, m, N, device="cpu")

    class Stub(efa.Fp8Layer):  # a layer that needs no memory
        def __init__(self):
            self.N, self.m, self.d, self.d_ff, self.tiled = 8, 2, 64, 128, False

        device = torch.device("cpu")
    for n in ((1 << 32) + 1, 1 - (1 << 32)):
        with pytest.raises(_abi.MoeError):
            Stub().grouped_workspace(n)
        with pytest.raises(_abi.MoeError):
            efa.grouped_square(Stub(), n, _abi.MOE_MAT_DOWN)
    assert Stub().grouped_workspace(1).numel() > 0 and efa.grouped_square(Stub(), 1, _abi.MOE_MAT_DOWN) is False
