"""A whole MoE layer on the tokens of a verification pass: router, selection, routed and
always-on experts (argument marshalling of ``moe_layer_pass`` in ``include/moe_expert.h``).
"""
import ctypes

import torch

from . import _abi
from ._abi import check, lib
from .grouped import _check, _empty, _guard, _int, _on
from .ops import Layer, _check_dev

_SCORES = {"softmax": _abi.MOE_SCORE_SOFTMAX, "sigmoid": _abi.MOE_SCORE_SIGMOID}


class Router:
    """The router of a layer: W_r [N][d] of the layer's type; ``score`` "softmax" or
    "sigmoid" of the logits; ``bias`` float32 [N], added to the scores for the selection
    alone; ``renorm``: the selected experts' weights are divided by their sum; ``scale``: a
    factor of the weights."""

    def __init__(self, w, score="softmax", bias=None, renorm=True, scale=1.0):
        if score not in _SCORES:
            raise ValueError("score must be one of %s, got %r" % (sorted(_SCORES), score))
        _check_dev("w", w)
        if w.dim() != 2:
            raise ValueError("w must be [N][d], got %s" % (tuple(w.shape),))
        if bias is not None:
            _check("bias", bias, torch.float32, (w.shape[0],), w.device)
        self.w, self.bias, self.score, self.renorm, self.scale = w, bias, score, bool(renorm), float(scale)
        self._desc = _abi.RouterDesc(w.data_ptr(), None if bias is None else bias.data_ptr(), _SCORES[score],
                                     int(self.renorm), self.scale)


def _check_layer(layer):
    if not isinstance(layer, Layer):
        raise TypeError("layer must be Layer, got %s" % type(layer).__name__)
    return layer.w_gate.device


def pass_workspace(layer, n, stream=None):
    """Zero-filled workspace of ``layer_pass`` for passes of up to n tokens."""
    dev = _check_layer(layer)
    nb = lib().moe_pass_workspace_bytes(ctypes.byref(layer.desc()), _int(int(n)))
    if nb == 0:
        raise _abi.MoeError("moe_pass_workspace_bytes", _abi.MOE_E_INVAL)
    if stream is None:
        return torch.zeros(nb, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.zeros(nb, dtype=torch.uint8, device=dev)


def layer_pass(layer, router, x, y=None, ids=None, w=None, info=None, ws=None, accumulate=False, stream=None):
    """y [n][d] of the layer for x [n][d], both of the layer's type (``moe_layer_pass``): at
    most 64 tokens and 256 slots.  ``ids`` int32 [n][m] and ``w`` float32 [n][m] receive the
    routing where given, ``info`` int32 [3] U, ids status and sync status; ``ws`` comes
    from ``pass_workspace`` (one call at a time).  A token all of whose logits are NaN gets ids -1,
    weights 0 and a y of NaN.  Runs on ``stream`` (default: the current
    stream of the layer's device)."""
    dev = _check_layer(layer)
    if not isinstance(router, Router):
        raise TypeError("router must be Router, got %s" % type(router).__name__)
    _check("router.w", router.w, layer.dtype, (layer.N, layer.d), dev)
    n = x.shape[0]
    xp = _check("x", x, layer.dtype, (n, layer.d), dev)
    if y is None:
        if accumulate:
            raise ValueError("accumulate=True needs y")
        y = _empty((n, layer.d), layer.dtype, dev, stream)
    yp = _check("y", y, layer.dtype, (n, layer.d), dev)
    idp = None if ids is None else _check("ids", ids, torch.int32, (n, layer.m), dev)
    wp = None if w is None else _check("w", w, torch.float32, (n, layer.m), dev)
    infop = None if info is None else _check("info", info, torch.int32, (3,), dev)
    if ws is None:
        ws = pass_workspace(layer, n, stream)
    wsp = _check("ws", ws, torch.uint8, ws.shape, dev)
    desc = layer.desc(accumulate)
    with _guard(dev):
        check("moe_layer_pass", lib().moe_layer_pass(ctypes.byref(desc), ctypes.byref(layer._weights),
                                                     ctypes.byref(router._desc), xp, _int(n), yp, idp, wp, infop, wsp,
                                                     ws.numel(), _on(dev, stream)))
    return y
