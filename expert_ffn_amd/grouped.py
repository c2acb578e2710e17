"""The expert operation on grouped rows: passes of any length, in bf16 or with 8-bit
weights, e4m3 or int8 (argument marshalling of the grouped calls of ``include/moe_expert.h``).

Every call runs on ``stream`` (default: the current stream of its tensors' device), with
that device current.  Outputs and workspaces that are not given are allocated for that
stream.
"""
import contextlib
import ctypes
from collections import namedtuple

import torch

from . import _abi
from ._abi import check, lib
from .ops import Grouping, Layer, _check_dev

# e4m3 codes [rows][K] and their scale bytes [rows][ceil(K/128)]: code * 2^(byte - 127); or int8
# codes [rows][K] and float32 scales [rows]: code * scale
Quantized = namedtuple("Quantized", ["q", "scale"])

_INT_MAX = (1 << 31) - 1
_NO_GUARD = contextlib.nullcontext()
_BF16, _F32, _I32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_I8 = torch.int8
_SUFFIX = {_BF16: "", _E4M3: "_fp8", _I8: "_int8"}  # of the calls on rows of this type


def _blocks(v):
    return -(-v // 128)


def _int(v):
    """A size as an argument of a call: one that C's int does not hold goes as the largest that
    it does, which every call refuses."""
    return v if -1 << 31 <= v <= _INT_MAX else _INT_MAX


def _guard(dev):
    return _NO_GUARD if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


# The current stream's handle; torch.cuda.current_stream(dev).cuda_stream makes a stream object first, 2 us of a
# call's 8.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on(dev, stream):
    if stream is None:
        return _current(dev.index)
    if stream.device != dev:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, dev))
    return stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):  # memory of the stream that the call runs on
        return torch.empty(shape, dtype=dtype, device=dev)


def _check(name, t, dtype, shape, dev):
    """One tensor of a call: contiguous, of this type, shape and device.  Small calls are
    bound by the host, so what is right is found right in one expression."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor, got %s" % (name, type(t).__name__))
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    _check_dev(name, t, dtype, shape)
    raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _ws(ws, desc, n, dev, stream):
    """Workspace of a grouped call (its size is checked by the call itself)."""
    if ws is None:
        nb = lib().moe_grouped_workspace_bytes(ctypes.byref(desc), _int(n))
        if nb == 0:
            raise _abi.MoeError("moe_grouped_workspace_bytes", _abi.MOE_E_INVAL)
        return _empty(nb, _U8, dev, stream)
    if not (ws.dtype is _U8 and ws.device == dev and ws.is_contiguous()):
        _check_dev("ws", ws, _U8)
        raise ValueError("ws is on %s, expected %s" % (ws.device, dev))
    return ws


def _check_codes(codes):
    if codes is not _E4M3 and codes is not _I8:
        raise TypeError("codes are float8_e4m3fn or int8, not %s" % (codes,))


def _scales(codes, rows, K):
    """(type, shape) of the scales of rows of codes."""
    return (_U8, (rows, _blocks(K))) if codes is _E4M3 else (_F32, (rows,))


def _new_quantized(codes, rows, K, dev, stream):
    typ, shape = _scales(codes, rows, K)
    return Quantized(_empty((rows, K), codes, dev, stream), _empty(shape, typ, dev, stream))


def _check_quantized(name, v, codes, rows, K, dev):
    if not isinstance(v, Quantized):
        raise TypeError("%s must be Quantized (codes and scales), got %s" % (name, type(v).__name__))
    typ, shape = _scales(codes, rows, K)
    return _check(name + ".q", v.q, codes, (rows, K), dev), _check(name + ".scale", v.scale, typ, shape, dev)


def _check_grouping(g, n, m, N, dev):
    if not isinstance(g, Grouping):
        raise TypeError("grouping must be Grouping, got %s" % type(g).__name__)
    return (_check("count", g.count, _I32, (N,), dev), _check("offset", g.offset, _I32, (N + 1,), dev),
            _check("slot_by_expert", g.slot_by_expert, _I32, (n * m,), dev),
            _check("distinct", g.distinct, _I32, (N,), dev), _check("u_and_err", g.u_and_err, _I32, (2,), dev))


class _CodesLayer:
    """8-bit weights of one MoE layer: each matrix a pair (codes, scales)."""

    def __init__(self, gate, up, down, m, tiled=False):
        for name, pair in (("gate", gate), ("up", up), ("down", down)):
            if len(pair) != 2:
                raise ValueError("%s must be (codes, %s)" % (name, self._what))
        N, d_ff, d = gate[0].shape
        self.N, self.m, self.d, self.d_ff = N, int(m), d, d_ff
        self.tiled = bool(tiled)
        for name, (q, s), (R, K) in (("gate", gate, (d_ff, d)), ("up", up, (d_ff, d)), ("down", down, (d, d_ff))):
            _check_dev("w_" + name, q, self.codes)
            _check("w_" + name, q, self.codes, (N, R, K), gate[0].device)
            _check("s_" + name, s, *self._scales(N, R, K), gate[0].device)
        self.gate, self.up, self.down = tuple(gate), tuple(up), tuple(down)
        self._weights = self._struct(*(m_[i].data_ptr() for i in (0, 1) for m_ in (self.gate, self.up, self.down)))

    @property
    def device(self):
        return self.gate[0].device

    @property
    def expert_bytes(self):
        return 3 * self.d * self.d_ff + sum(p[1][0].numel() * p[1].element_size() for p in (self.gate, self.up, self.down))

    def desc(self, accumulate=False):
        """The layer's descriptor (``moe_layer_desc``)."""
        flags = (_abi.MOE_FLAG_ACCUMULATE if accumulate else 0) | (_abi.MOE_FLAG_TILED if self.tiled else 0)
        return _abi.LayerDesc(self.N, self.m, self.d, self.d_ff, self._code, flags, 0)

    def tiled_copy(self, stream=None):
        """The same layer with the codes copied into the tiled layout by
        ``moe_pack_tiled`` (scales shared)."""
        if self.tiled:
            return self
        desc, dev = self.desc(), self.device

        def tl(pair, mat):
            out = _empty(pair[0].shape, self.codes, dev, stream)
            with _guard(dev):
                check("moe_pack_tiled", lib().moe_pack_tiled(ctypes.byref(desc), pair[0].data_ptr(), out.data_ptr(),
                                                             mat, _on(dev, stream)))
            return out, pair[1]
        G, D = _abi.MOE_MAT_GATE_UP, _abi.MOE_MAT_DOWN
        return type(self)(tl(self.gate, G), tl(self.up, G), tl(self.down, D), self.m, tiled=True)

    def grouped_workspace(self, n):
        """Workspace of the grouped calls on this layer for passes of up to n tokens."""
        return grouped_workspace(self, n)


class Fp8Layer(_CodesLayer):
    """8-bit weights of one MoE layer: each matrix a pair (codes float8_e4m3fn, scale
    bytes uint8), W_gate and W_up [N][d_ff][d] with [N][d_ff/128][d/128] scales, W_down
    [N][d][d_ff] with [N][d/128][d_ff/128] (sizes rounded up), as ``Layer.fp8_copy``
    makes them; with ``tiled`` the codes are in the layout of ``moe_pack_tiled``."""

    codes, _code, _what, _struct = _E4M3, _abi.MOE_FP8, "scale bytes", _abi.Fp8Weights

    @staticmethod
    def _scales(N, R, K):
        return _U8, (N, _blocks(R), _blocks(K))


class Int8Layer(_CodesLayer):
    """8-bit integer weights of one MoE layer: each matrix a pair (codes int8, scales
    float32 of its output channels), W_gate and W_up [N][d_ff][d] with [N][d_ff] scales,
    W_down [N][d][d_ff] with [N][d], as ``Layer.int8_copy`` makes them; with ``tiled`` the
    codes are in the layout of ``moe_pack_tiled``."""

    codes, _code, _what, _struct = _I8, _abi.MOE_INT8, "scales", _abi.Int8Weights

    @staticmethod
    def _scales(N, R, K):
        return _F32, (N, R)


def quant_weights(w, stream=None, dtype=_E4M3):
    """bf16 matrices [N][R][K] to (codes, scales): with float8_e4m3fn scale bytes
    [N][R/128][K/128], one power of two for each block of 128 x 128 (``moe_quant_weights``);
    with int8 float32 [N][R], one for each row (``moe_quant_rows_int8``)."""
    _check_codes(dtype)
    _check_dev("w", w, _BF16)
    if w.dim() != 3:
        raise ValueError("w must be [N][R][K], got %s" % (tuple(w.shape),))
    N, R, K = w.shape
    dev = w.device
    q = _empty((N, R, K), dtype, dev, stream)
    if dtype is _I8:
        s = _empty((N, R), _F32, dev, stream)
        with _guard(dev):
            check("moe_quant_rows_int8", lib().moe_quant_rows_int8(w.data_ptr(), N * R, _int(K), q.data_ptr(),
                                                                   s.data_ptr(), _on(dev, stream)))
        return q, s
    s = _empty((N, _blocks(R), _blocks(K)), _U8, dev, stream)
    with _guard(dev):
        check("moe_quant_weights", lib().moe_quant_weights(w.data_ptr(), _int(N), _int(R), _int(K), q.data_ptr(),
                                                           s.data_ptr(), _on(dev, stream)))
    return q, s


def _codes_copy(cls, layer, stream):
    if layer.dtype != torch.bfloat16 or layer.packed or layer.tiled:
        raise ValueError("%s takes plain bf16 weights (tile the copy)" % ("fp8_copy" if cls is Fp8Layer else "int8_copy"))
    if layer.shared is not None:
        raise ValueError("copy the routed and the shared experts as layers of their own (without_shared)")
    return cls(*(quant_weights(w, stream, cls.codes) for w in (layer.w_gate, layer.w_up, layer.w_down)), m=layer.m)


def fp8_copy(layer, stream=None):
    """``layer`` (plain bf16 weights) with 8-bit weights in plain layout."""
    return _codes_copy(Fp8Layer, layer, stream)


def int8_copy(layer, stream=None):
    """``layer`` (plain bf16 weights) with int8 weights in plain layout."""
    return _codes_copy(Int8Layer, layer, stream)


def quant_rows(x, out=None, stream=None, dtype=_E4M3):
    """Rows of bf16 values [rows][K] to ``Quantized``: with float8_e4m3fn one power of two
    for each block of 128 along a row (``moe_quant_rows``), with int8 one scale for each
    row (``moe_quant_rows_int8``)."""
    _check_codes(dtype)
    _check_dev("x", x, _BF16)
    if x.dim() != 2:
        raise ValueError("x must be [rows][K], got %s" % (tuple(x.shape),))
    rows, K = x.shape
    dev = x.device
    if out is None:
        out = _new_quantized(dtype, rows, K, dev, stream)
    q, s = _check_quantized("out", out, dtype, rows, K, dev)
    name = "moe_quant_rows" if dtype is _E4M3 else "moe_quant_rows_int8"
    with _guard(dev):
        check(name, getattr(lib(), name)(x.data_ptr(), rows, _int(K), q, s, _on(dev, stream)))
    return out


def dequant_rows(v, out=None, stream=None):
    """The bf16 values that ``Quantized`` rows stand for (``moe_dequant_rows``,
    ``moe_dequant_rows_int8``)."""
    if not isinstance(v, Quantized) or v.q.dim() != 2:
        raise TypeError("dequant_rows takes Quantized rows")
    rows, K = v.q.shape
    dev, codes = v.q.device, v.q.dtype
    _check_dev("v.q", v.q)
    _check_codes(codes)
    q, s = _check_quantized("v", v, codes, rows, K, dev)
    if out is None:
        out = _empty((rows, K), _BF16, dev, stream)
    x = _check("out", out, _BF16, (rows, K), dev)
    name = "moe_dequant_rows" if codes is _E4M3 else "moe_dequant_rows_int8"
    with _guard(dev):
        check(name, getattr(lib(), name)(q, s, rows, _int(K), x, _on(dev, stream)))
    return out


def group_workspace(n, m, N, device="cuda"):
    """Workspace of ``group_slots`` for n tokens of m slots and N experts."""
    nb = lib().moe_group_workspace_bytes(_int(int(n)), _int(int(m)), _int(int(N)))
    if nb == 0:
        raise _abi.MoeError("moe_group_workspace_bytes", _abi.MOE_E_INVAL)
    return torch.empty(nb, dtype=torch.uint8, device=device)


def group_slots(ids, N, out=None, ws=None, stream=None):
    """``route_group`` for any number of slots (``moe_group_slots``): ids int32 [n][m];
    ids outside [0, N) take no part."""
    _check_dev("ids", ids, _I32)
    if ids.dim() != 2:
        raise ValueError("ids must be [n][m], got %s" % (tuple(ids.shape),))
    n, m = ids.shape
    N, dev = int(N), ids.device
    if n * m > _INT_MAX or N > _INT_MAX:  # (neither n nor m is more than their product, or one is 0)
        raise _abi.MoeError("moe_group_slots", _abi.MOE_E_INVAL)
    if ws is None:
        nb = lib().moe_group_workspace_bytes(n, m, N)
        if nb == 0:
            raise _abi.MoeError("moe_group_workspace_bytes", _abi.MOE_E_INVAL)
        ws = _empty(nb, _U8, dev, stream)
    if out is None:
        out = Grouping(*(_empty(k, _I32, dev, stream) for k in (N, N + 1, n * m, N, 2)))
    ptrs = _check_grouping(out, n, m, N, dev)
    wsp = _check("ws", ws, _U8, ws.shape, dev)
    with _guard(dev):
        check("moe_group_slots", lib().moe_group_slots(ids.data_ptr(), n, m, N, *ptrs, wsp, ws.numel(),
                                                       _on(dev, stream)))
    return out


def _kind(layer):
    """(type of the layer's rows: bf16, or of its codes; its device); refuses what the
    grouped calls do not take."""
    if isinstance(layer, _CodesLayer):
        return layer.codes, layer.device
    if not isinstance(layer, Layer):
        raise TypeError("layer must be Layer, Fp8Layer or Int8Layer, got %s" % type(layer).__name__)
    if layer.dtype != _BF16:
        raise TypeError("grouped calls take bf16 or 8-bit weights, got %s" % layer.dtype)
    if layer.packed:
        raise ValueError("grouped calls take plain or tiled weights, not a packed W_down")
    if layer.n_shared:
        raise ValueError("run the shared experts as a layer of their own with m = N and accumulate=True "
                         "(and the routed ones from without_shared())")
    return _BF16, layer.w_gate.device


def grouped_workspace(layer, n):
    """Workspace of the grouped calls for passes of up to n tokens."""
    _, dev = _kind(layer)
    return _ws(None, layer.desc(), int(n), dev, None)


def grouped_square(layer, n, mat):
    """Whether passes of n tokens take square tiles for ``mat`` (MOE_MAT_GATE_UP or
    MOE_MAT_DOWN); thin ones otherwise (``moe_grouped_square``, host only)."""
    _kind(layer)
    v = lib().moe_grouped_square(ctypes.byref(layer.desc()), _int(int(n)), _int(int(mat)))
    if v < 0:
        raise _abi.MoeError("moe_grouped_square", v)
    return bool(v)


def grouped_gate_up(layer, x, grouping, out=None, ws=None, stream=None):
    """h [n*m][d_ff] in row order (``moe_grouped_gate_up``): bf16 from bf16 x [n][d], or
    with 8-bit weights ``Quantized`` from ``Quantized`` x (``quant_rows`` with the layer's
    type of codes).  Rows from offset[N] on are left as they were."""
    typ, dev = _kind(layer)
    codes = typ is not _BF16
    if isinstance(x, Quantized) != codes:
        raise TypeError("x must be %s for this layer" % ("Quantized (quant_rows)" if codes else "a bf16 tensor"))
    n = (x.q if codes else x).shape[0]
    S, d, f = n * layer.m, layer.d, layer.d_ff
    _, offset, slots, _, _ = _check_grouping(grouping, n, layer.m, layer.N, dev)
    desc, name = layer.desc(), "moe_grouped_gate_up" + _SUFFIX[typ]
    if codes:
        xs = _check_quantized("x", x, typ, n, d, dev)
        if out is None:
            out = _new_quantized(typ, S, f, dev, stream)
        hs = _check_quantized("out", out, typ, S, f, dev)
    else:
        xs = (_check("x", x, _BF16, (n, d), dev),)
        if out is None:
            out = _empty((S, f), _BF16, dev, stream)
        hs = (_check("out", out, _BF16, (S, f), dev),)
    ws = _ws(ws, desc, n, dev, stream)
    with _guard(dev):
        check(name, getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(layer._weights), *xs, _int(n), offset, slots,
                                         *hs, ws.data_ptr(), ws.numel(), _on(dev, stream)))
    return out


def _check_y(layer, y, n, dev, accumulate, stream):
    if y is None:
        if accumulate:
            raise ValueError("accumulate=True needs y")
        y = _empty((n, layer.d), _BF16, dev, stream)
    return y, _check("y", y, _BF16, (n, layer.d), dev)


def grouped_down(layer, h, ids, w, grouping, y=None, ws=None, accumulate=False, stream=None):
    """y [n][d] bf16: the down products of h's rows, summed over each token's slots with
    the routing weights w (``moe_grouped_down``); ``accumulate`` adds to y."""
    typ, dev = _kind(layer)
    n, m, f = ids.shape[0], layer.m, layer.d_ff
    idp, wp = _check("ids", ids, _I32, (n, m), dev), _check("w", w, _F32, (n, m), dev)
    _, offset, slots, _, _ = _check_grouping(grouping, n, m, layer.N, dev)
    y, yp = _check_y(layer, y, n, dev, accumulate, stream)
    desc, name = layer.desc(accumulate), "moe_grouped_down" + _SUFFIX[typ]
    hs = (_check("h", h, _BF16, (n * m, f), dev),) if typ is _BF16 else _check_quantized("h", h, typ, n * m, f, dev)
    ws = _ws(ws, desc, n, dev, stream)
    with _guard(dev):
        check(name, getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(layer._weights), *hs, idp, wp, _int(n), offset, slots,
                                         yp, ws.data_ptr(), ws.numel(), _on(dev, stream)))
    return y


def expert_grouped(layer, x, ids, w, y=None, ws=None, info=None, accumulate=False, stream=None):
    """A whole pass of any length: grouping, gate/up and down (``moe_expert_grouped``, or
    ``moe_expert_grouped_fp8`` for an ``Fp8Layer`` and ``moe_expert_grouped_int8`` for an
    ``Int8Layer``, which quantise x first).  x and y
    bf16 [n][d]; ids outside [0, N) add nothing; ``info`` int32 [3]: U, ids status, 0."""
    typ, dev = _kind(layer)
    n, m = x.shape[0], layer.m
    xp = _check("x", x, _BF16, (n, layer.d), dev)
    idp, wp = _check("ids", ids, _I32, (n, m), dev), _check("w", w, _F32, (n, m), dev)
    y, yp = _check_y(layer, y, n, dev, accumulate, stream)
    infop = None if info is None else _check("info", info, _I32, (3,), dev)
    desc, name = layer.desc(accumulate), "moe_expert_grouped" + _SUFFIX[typ]
    ws = _ws(ws, desc, n, dev, stream)
    with _guard(dev):
        check(name, getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(layer._weights), xp, idp, wp, _int(n), yp,
                                         infop, ws.data_ptr(), ws.numel(), _on(dev, stream)))
    return y
