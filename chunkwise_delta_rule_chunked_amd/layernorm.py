"""Binding of include/delta_layernorm.h: the layer norm of the residual stream, with the dropout of its
branch, and dropout alone.  Marshals and checks arguments as block.py does.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import BF16, _check, load_library
from .block import _arg, _bytes_of, _f32, _on, _opt, _out, _raw, _rows, _workspace

_lib = None


class Dropout(ctypes.Structure):
    """delta_dropout"""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("step", ctypes.c_void_p)]


def _load():
    """libdelta.so with the argument types of delta_layernorm.h declared."""
    global _lib
    if _lib is None:
        lib = load_library()
        P, I, F, Z, R = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
        for name, args in {
            "delta_layer_dropout": [R, I, I] + [P] * 5,
            "delta_layer_layernorm": [R, I, I, F] + [P] * 8,
            "delta_layer_layernorm_bwd_workspace_bytes": [R, I, I, P],
            "delta_layer_layernorm_bwd": [R, I, I, F] + [P] * 10 + [Z, P],
        }.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _dropout(p, seed, offset, device):
    """(the call's delta_dropout, whether anything is dropped)."""
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1], got %r" % (p,))
    step = None
    if isinstance(offset, torch.Tensor):
        step, offset = _arg(offset, "offset", torch.Size(()), torch.int64, device), 0
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset must be in [0, 2^64)")
    return Dropout(p, seed, offset, step), round(p * 65536) != 0


def layer_dropout(x, residual=None, *, p: float, seed: int, offset=0, y=None, stream=None):
    """dropout(x) + residual (delta_layer_dropout): a value is dropped with probability p (to the nearest 65536th)
    and else divided by 1 - p.  The mask comes from (seed, offset) and the value's row and channel alone and is
    never stored: the gradient of x is the same call on y's gradient, without a residual.  `offset` is a number, or
    an int64 GPU scalar that the kernel reads (advance it in a captured graph, and each replay has a mask of its
    own).  Pass y=x or y=residual to work in place."""
    rows, width, code = _rows(x, "x")
    dev, shp = x.device, x.shape
    drop, _ = _dropout(p, seed, offset, dev)
    with _on(dev, stream):
        px, pr = _arg(x, "x", shp, x.dtype, dev), _opt(residual, "residual", shp, x.dtype, dev)
        y, py = _out(y, "y", shp, x.dtype, dev, x)
        rc = _load().delta_layer_dropout(rows, width, code, ctypes.byref(drop), px, pr, py, _raw(dev))
    _check(rc, "delta_layer_dropout")
    return y


def layer_layernorm(x, weight, bias=None, residual=None, *, eps: float = 1e-5, p: float = 0.0, seed: int = 0, offset=0,
                    sum=None, y=None, stream=None):
    """s = dropout(x) + residual (rounded to x's type) and y = (s - mean) / sqrt(var + eps) * weight + bias over the
    last dimension (delta_layer_layernorm); weight and bias [width] fp32, p, seed and offset as layer_dropout's.
    Returns (s, y); without a residual and with p = 0 s is x itself.  Pass sum=residual to update the residual
    stream in place."""
    rows, width, code = _rows(x, "x")
    dev, shp = x.device, x.shape
    drop, drops = _dropout(p, seed, offset, dev)
    with _on(dev, stream):
        px, pr = _arg(x, "x", shp, x.dtype, dev), _opt(residual, "residual", shp, x.dtype, dev)
        pw, pb, ps = _arg(weight, "weight", (width,), _f32, dev), _opt(bias, "bias", (width,), _f32, dev), None
        own = residual is not None or drops
        if own:
            sum, ps = _out(sum, "sum", shp, x.dtype, dev, x)
        y, py = _out(y, "y", shp, x.dtype, dev, x)
        rc = _load().delta_layer_layernorm(rows, width, code, eps, ctypes.byref(drop), px, pr, pw, pb, ps, py, _raw(dev))
    _check(rc, "delta_layer_layernorm")
    return (sum if own else x), y


@functools.lru_cache(maxsize=1024)
def layernorm_bwd_workspace_bytes(rows, width, dtype=BF16) -> int:
    """Workspace of layer_layernorm_bwd for this shape (none is used without dweight and dbias)."""
    return _bytes_of(_load(), "delta_layer_layernorm_bwd_workspace_bytes", rows, width, dtype)


def layer_layernorm_bwd(dy, s, weight, dsum=None, *, eps: float = 1e-5, p: float = 0.0, seed: int = 0, offset=0,
                        want_dweight: bool = True, want_dbias: bool = True, grads=None, workspace=None, stream=None):
    """Backward pass of layer_layernorm (delta_layer_layernorm_bwd) from its s, with the forward pass's p, seed and
    offset; dsum is the gradient that reaches s past the norm (None for zero).  Returns a dict: dresidual and dx in
    s's type (dx through the dropout; the same tensor where p = 0), dweight and dbias [width] fp32 (None unless
    wanted).  `grads` may hold preallocated outputs under the same names."""
    rows, width, code = _rows(s, "s")
    dev, shp = s.device, s.shape
    drop, drops = _dropout(p, seed, offset, dev)
    g = {"dresidual": None, "dx": None, "dweight": None, "dbias": None}
    unknown = set(grads or ()) - set(g)
    if unknown:
        raise ValueError("grads has names that are none of %s: %s" % (", ".join(g), ", ".join(map(str, unknown))))
    g.update(grads or {})
    with _on(dev, stream):
        pdy, ps = _arg(dy, "dy", shp, s.dtype, dev), _arg(s, "s", shp, s.dtype, dev)
        pw, pds = _arg(weight, "weight", (width,), _f32, dev), _opt(dsum, "dsum", shp, s.dtype, dev)
        pdx = pdw = pdb = None
        if not drops and g["dx"] is not None and g["dresidual"] is not None and g["dx"] is not g["dresidual"]:
            raise ValueError("with p = 0 dx is dresidual: give one tensor for both, or one of them")
        if not drops and g["dresidual"] is None:
            g["dresidual"] = g["dx"]
        g["dresidual"], pdr = _out(g["dresidual"], "dresidual", shp, s.dtype, dev, s)
        if drops:
            g["dx"], pdx = _out(g["dx"], "dx", shp, s.dtype, dev, s)
        else:
            g["dx"] = g["dresidual"]
        if g["dweight"] is not None or want_dweight:
            g["dweight"], pdw = _out(g["dweight"], "dweight", (width,), _f32, dev, weight)
        if g["dbias"] is not None or want_dbias:
            g["dbias"], pdb = _out(g["dbias"], "dbias", (width,), _f32, dev, weight)
        need = 0 if pdw is None and pdb is None else layernorm_bwd_workspace_bytes(rows, width, code)
        ws, nws, keep = _workspace(workspace, need, dev)
        rc = _load().delta_layer_layernorm_bwd(rows, width, code, eps, ctypes.byref(drop), pdy, ps, pw, pds, pdr, pdx, pdw, pdb,
                                               ws, nws, _raw(dev))
    _check(rc, "delta_layer_layernorm_bwd")
    return g
