"""Binding of include/delta_linear.h: linear attention with a decay for each head, forward and backward over a
sequence and for one token.  Marshals and checks arguments as block.py does.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import BF16, _check, load_library, make_shape
from .block import _arg, _bytes_of, _code, _f32, _on, _opt, _out, _raw, _workspace

GATE_NONE, GATE_TOKEN, GATE_HEAD = 0, 1, 2  # include/delta_linear.h: DELTA_LIN_GATE_*
_lib = None


def _load():
    """libdelta.so with the argument types of delta_linear.h declared."""
    global _lib
    if _lib is None:
        lib = load_library()
        P, I, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        for name, args in {
            "delta_fwd_lin_workspace_bytes": [P, I, P], "delta_fwd_lin": [P, I, I] + [P] * 8 + [Z, P],
            "delta_bwd_lin_workspace_bytes": [P, I, I, P], "delta_bwd_lin": [P, I, I] + [P] * 13 + [Z, P],
            "delta_decode_lin": [P, I, I] + [P] * 7,
        }.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=1024)
def _plan(B, L, Hk, H, dk, dv, code, scale):
    """The shape as the library takes it (the structure and a reference to it), and the forward pass's workspace."""
    sh = make_shape(B, L, H, dk, dv, 1, 64, code, scale)
    ref = ctypes.byref(sh)
    return ref, _bytes_of(_load(), "delta_fwd_lin_workspace_bytes", ref, Hk)


def lin_workspace_bytes(B, L, Hk, H, dk, dv, dtype=BF16) -> int:
    """Workspace of fwd_lin for this shape."""
    return _plan(B, L, Hk, H, dk, dv, dtype, 1.0)[1]


@functools.lru_cache(maxsize=1024)
def bwd_lin_workspace_bytes(B, L, Hk, H, dk, dv, dtype=BF16, gate=GATE_TOKEN) -> int:
    """Workspace of bwd_lin for this shape (gate: 0 none, or no dg_log wanted, 1 [B, L, H], 2 [H])."""
    return _bytes_of(_load(), "delta_bwd_lin_workspace_bytes", _plan(B, L, Hk, H, dk, dv, dtype, 1.0)[0], Hk, gate)


def _inputs(q, k, v, g_log, scale):
    """Shapes, plan, gate kind and pointers of what every call takes."""
    code = _code(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, L, Hk, dk]")
    B, L, Hk, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v must be [B, L, H, dv]")
    H, dv = v.shape[2:]
    if Hk == 0 or H % Hk:
        raise ValueError("v's heads (%d) must be a multiple of q's (%d)" % (H, Hk))
    dev = q.device
    ptrs = [_arg(q, "q", q.shape, q.dtype, dev), _arg(k, "k", q.shape, q.dtype, dev), _arg(v, "v", (B, L, H, dv), q.dtype, dev)]
    gate = GATE_NONE
    if g_log is not None:
        if not isinstance(g_log, torch.Tensor) or g_log.dim() not in (1, 3):
            raise ValueError("g_log must be [B, L, H], [H] or None")
        gate = GATE_TOKEN if g_log.dim() == 3 else GATE_HEAD
        ptrs.append(_arg(g_log, "g_log", (B, L, H) if gate == GATE_TOKEN else (H,), _f32, dev))
    else:
        ptrs.append(None)
    return (B, L, Hk, H, dk, dv), code, _plan(B, L, Hk, H, dk, dv, code, float(scale)), gate, ptrs


def fwd_lin(q, k, v, g_log=None, S0=None, *, scale: float = 1.0, O=None, S_final=None, want_state: bool = True,
            workspace=None, stream=None):
    """Linear attention with a decay for each head over a sequence (delta_fwd_lin): S_t = exp(g_t) S_{t-1} +
    k_t v_t^T, o_t = scale S_t^T q_t.  q, k [B,L,Hk,dk] and v [B,L,H,dv] (bf16 or fp32; H a multiple of Hk,
    consecutive value heads sharing a query and key head), g_log fp32: [B,L,H], [H] for fixed decays, or None;
    S0 [B,H,dk,dv] fp32 or None.  Returns (O, S_final); S_final is None if want_state is False and no buffer is
    given.  Pass S_final=S0 to update the state in place."""
    (B, L, Hk, H, dk, dv), code, (ref, need), gate, ptrs = _inputs(q, k, v, g_log, scale)
    dev, sshp = q.device, (B, H, dk, dv)
    with _on(dev, stream):
        p0, ps = _opt(S0, "S0", sshp, _f32, dev), None
        O, po = _out(O, "O", v.shape, q.dtype, dev, v)
        if S_final is not None or want_state:
            S_final, ps = _out(S_final, "S_final", sshp, _f32, dev, v if S0 is None else S0)
        ws, nws, keep = _workspace(workspace, need, dev)
        rc = _load().delta_fwd_lin(ref, Hk, gate, *ptrs, p0, po, ps, ws, nws, _raw(dev))
    _check(rc, "delta_fwd_lin")
    return O, S_final


def bwd_lin(q, k, v, g_log, S0, dO, dS_final=None, *, scale: float = 1.0, want_dg_log: bool = True, want_dS0: bool = True,
            grads=None, workspace=None, stream=None):
    """Backward pass of fwd_lin for the same arguments (delta_bwd_lin); dO has v's shape and type, dS_final
    [B,H,dk,dv] fp32 may be None for zero.  Returns a dict: dq, dk, dv in the inputs' type (dq and dk summed over
    the heads that share them), dg_log fp32 like g_log (None without gates or unless want_dg_log), dS0 fp32 (None
    unless want_dS0).  With dg_log the workspace holds a state for each chunk, and bf16 dq and dk are formed from
    states that are as good as float32 (else rounded to bf16): their last bits differ.  `grads` may hold preallocated
    outputs under the same names."""
    dims, code, (ref, _), gate, ptrs = _inputs(q, k, v, g_log, scale)
    B, L, Hk, H, dk, dv = dims
    dev, sshp = q.device, (B, H, dk, dv)
    g = {"dq": None, "dk": None, "dv": None, "dg_log": None, "dS0": None}
    unknown = set(grads or ()) - set(g)
    if unknown:
        raise ValueError("grads has names that are none of %s: %s" % (", ".join(g), ", ".join(map(str, unknown))))
    g.update(grads or {})
    if g_log is None and g["dg_log"] is not None:
        raise ValueError("dg_log needs g_log")
    with _on(dev, stream):
        p0, pd, ps = _opt(S0, "S0", sshp, _f32, dev), _arg(dO, "dO", v.shape, q.dtype, dev), _opt(dS_final, "dS_final", sshp, _f32, dev)
        outs = []
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            g[name], p = _out(g[name], name, like.shape, q.dtype, dev, like)
            outs.append(p)
        pg = p00 = None
        if g_log is not None and (g["dg_log"] is not None or want_dg_log):
            g["dg_log"], pg = _out(g["dg_log"], "dg_log", g_log.shape, _f32, dev, g_log)
        if g["dS0"] is not None or want_dS0:
            g["dS0"], p00 = _out(g["dS0"], "dS0", sshp, _f32, dev, v)
        ws, nws, keep = _workspace(workspace, bwd_lin_workspace_bytes(*dims, code, gate if pg else GATE_NONE), dev)
        rc = _load().delta_bwd_lin(ref, Hk, gate, *ptrs, p0, pd, ps, *outs, pg, p00, ws, nws, _raw(dev))
    _check(rc, "delta_bwd_lin")
    return g


def decode_lin(q, k, v, g_log, S, *, scale: float = 1.0, O=None, stream=None):
    """One token of linear attention (delta_decode_lin): q, k [B,1,Hk,dk], v [B,1,H,dv], g_log [B,1,H], [H] or
    None, S [B,H,dk,dv] fp32 updated in place.  Returns O [B,1,H,dv]."""
    (B, L, Hk, H, dk, dv), code, (ref, _), gate, ptrs = _inputs(q, k, v, g_log, scale)
    if L != 1:
        raise ValueError("decode_lin takes one token: q must be [B, 1, Hk, dk]")
    dev = q.device
    with _on(dev, stream):
        ps = _arg(S, "S", (B, H, dk, dv), _f32, dev)
        O, po = _out(O, "O", v.shape, q.dtype, dev, v)
        rc = _load().delta_decode_lin(ref, Hk, gate, *ptrs, ps, po, _raw(dev))
    _check(rc, "delta_decode_lin")
    return O
