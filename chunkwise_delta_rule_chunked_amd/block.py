"""Binding of include/delta_block.h: the gated linear recurrence, the RMS norm of the residual
stream and gradient clipping.

As the rest of the package it only marshals arguments, and it checks every tensor's shape, type
and device before the library sees a pointer.  Work goes to the device the tensors are on,
whichever is current: to that device's current stream, or to `stream`.  Outputs and workspaces
that the caller does not pass are allocated on the stream that the work runs on.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools

import torch

from . import BF16, F32, _check, load_library, make_shape

GLR_CHUNK = 64  # include/delta_block.h: DELTA_GLR_CHUNK
INPUT_GATES = {"none": 0, "complement": 1, "norm": 2}

_f32 = torch.float32
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
_lib = None


def _load():
    """libdelta.so with the argument types of delta_block.h declared."""
    global _lib
    if _lib is None:
        lib = load_library()
        P, S, I, F, Z = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        R = ctypes.c_int64
        for name, args in {
            "delta_fwd_glr_workspace_bytes": [S, P], "delta_fwd_glr": [S, I] + [P] * 7 + [Z, P],
            "delta_bwd_glr_workspace_bytes": [S, P], "delta_bwd_glr": [S, I] + [P] * 9 + [Z, P],
            "delta_decode_glr": [S, I] + [P] * 5,
            "delta_layer_rmsnorm": [R, I, I, F] + [P] * 6,
            "delta_layer_rmsnorm_quant": [R, I, I, F, I] + [P] * 7,
            "delta_layer_rmsnorm_bwd_workspace_bytes": [R, I, I, P],
            "delta_layer_rmsnorm_bwd": [R, I, I, F] + [P] * 7 + [Z, P],
            "delta_grad_norm_workspace_bytes": [I, P, P],
            "delta_grad_norm": [I] + [P] * 5 + [Z, P],
            "delta_clip_grads": [I] + [P] * 3 + [F, F] + [P] * 3 + [Z, P],
        }.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


_here = contextlib.nullcontext()


def _on(device, stream):
    """Context in which `device` is current and `stream` (None, a torch stream or a raw handle) its
    current stream."""
    if stream is None:
        return _here if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _raw(device):
    # the handle of torch.cuda.current_stream(device) without building the stream object (2 us)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _code(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    return code


def _arg(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device.index:
        raise ValueError("%s must be a GPU tensor on %s" % (name, device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _opt(t, *spec):
    """As _arg; None: NULL."""
    return None if t is None else _arg(t, *spec)


def _out(t, name, shape, dtype, device, like):
    """(tensor, pointer) of an output: the given one, checked, or a new one made from the checked input
    `like` (quicker than from a device, and most so where the shape is the same)."""
    if t is None:
        t = torch.empty_like(like, dtype=dtype) if like.shape == shape else like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _arg(t, name, shape, dtype, device)


def _workspace(given, need, device):
    """(pointer, bytes, tensor to keep alive) of a workspace of at least `need` bytes."""
    if given is None:
        if need == 0:
            return None, 0, None
        given = torch.empty(need, dtype=torch.uint8, device=device)
    elif not isinstance(given, torch.Tensor) or given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on %s" % device)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _gate(name):
    try:
        return INPUT_GATES[name]
    except (KeyError, TypeError):
        raise ValueError("input_gate must be one of %s, got %r" % (", ".join(INPUT_GATES), name)) from None


def _bytes_of(lib, fn, *args):
    """The size that a workspace function of the loaded library gives."""
    n = ctypes.c_size_t(0)
    _check(getattr(lib, fn)(*args, ctypes.byref(n)), fn)
    return n.value


def _bytes(fn, *args):
    return _bytes_of(_load(), fn, *args)


@functools.lru_cache(maxsize=1024)
def _glr_plan(B, L, H, dv, code):
    """The shape as the library takes it, and its workspaces forward and backward: what a size alone
    says."""
    sh = make_shape(B, L, H, 16, dv, 1, 64, code)
    ref = ctypes.byref(sh)
    return ref, _bytes("delta_fwd_glr_workspace_bytes", ref), _bytes("delta_bwd_glr_workspace_bytes", ref)


def _glr_shape(x):
    code = _code(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, L, H, dv]")
    return x.shape, _glr_plan(*x.shape, code)


def glr_workspace_bytes(B, L, H, dv, dtype=BF16) -> int:
    """Workspace of fwd_glr for this shape."""
    return _glr_plan(B, L, H, dv, dtype)[1]


def bwd_glr_workspace_bytes(B, L, H, dv, dtype=BF16) -> int:
    """Workspace of bwd_glr for this shape."""
    return _glr_plan(B, L, H, dv, dtype)[2]


def fwd_glr(x, g_log, h0=None, *, input_gate: str = "none", O=None, h_final=None, states=None,
            want_state: bool = True, want_states: bool = False, workspace=None, stream=None):
    """Gated linear recurrence over a sequence (delta_fwd_glr): h_t = a_t h_{t-1} + w_t x_t per
    channel, a = exp(g_log), w = 1 ("none"), 1 - a ("complement") or sqrt(1 - a^2) ("norm").
    x [B,L,H,dv] (bf16 or fp32), g_log [B,L,H,dv] fp32 (-inf: hard reset), h0 [B,H,dv] fp32 or None.
    Returns (O, h_final, states); h_final is None if want_state is False and no buffer is given,
    states (the states before tokens 0, 64, ..., [B,ceil(L/64),H,dv] fp32, what bwd_glr takes) None
    unless want_states or a buffer is given.  Pass h_final=h0 to update the state in place."""
    shp, (ref, need, _) = _glr_shape(x)
    B, L, H, dv = shp
    gate, dev, sshp = _gate(input_gate), x.device, (B, H, dv)
    with _on(dev, stream):
        px, pg = _arg(x, "x", shp, x.dtype, dev), _arg(g_log, "g_log", shp, _f32, dev)
        p0, ph, ps = _opt(h0, "h0", sshp, _f32, dev), None, None
        O, po = _out(O, "O", shp, x.dtype, dev, x)
        if h_final is not None or want_state:
            h_final, ph = _out(h_final, "h_final", sshp, _f32, dev, x)
        if states is not None or want_states:
            states, ps = _out(states, "states", (B, -(-L // GLR_CHUNK), H, dv), _f32, dev, x)
        ws, nws, keep = _workspace(workspace, need, dev)
        rc = _load().delta_fwd_glr(ref, gate, px, pg, p0, po, ph, ps, ws, nws, _raw(dev))
    _check(rc, "delta_fwd_glr")
    return O, h_final, states


def bwd_glr(x, g_log, states, dO, dh_final=None, *, input_gate: str = "none", want_dh0: bool = True, grads=None,
            workspace=None, stream=None):
    """Backward pass of fwd_glr (delta_bwd_glr) from the same x and g_log and the states it wrote;
    dO has x's shape and type, dh_final [B,H,dv] fp32 may be None for zero.  Returns a dict of
    float32 gradients dx, dg_log and dh0 (None unless want_dh0); `grads` may hold preallocated
    outputs under the same names."""
    shp, (ref, _, need) = _glr_shape(x)
    B, L, H, dv = shp
    gate, dev, sshp = _gate(input_gate), x.device, (B, H, dv)
    g = {"dx": None, "dg_log": None, "dh0": None}
    g.update(grads or {})
    with _on(dev, stream):
        px, pg = _arg(x, "x", shp, x.dtype, dev), _arg(g_log, "g_log", shp, _f32, dev)
        ps = _arg(states, "states", (B, -(-L // GLR_CHUNK), H, dv), _f32, dev)
        pd, ph, p0 = _arg(dO, "dO", shp, x.dtype, dev), _opt(dh_final, "dh_final", sshp, _f32, dev), None
        g["dx"], pdx = _out(g["dx"], "dx", shp, _f32, dev, g_log)
        g["dg_log"], pdg = _out(g["dg_log"], "dg_log", shp, _f32, dev, g_log)
        if g["dh0"] is not None or want_dh0:
            g["dh0"], p0 = _out(g["dh0"], "dh0", sshp, _f32, dev, x)
        ws, nws, keep = _workspace(workspace, need, dev)
        rc = _load().delta_bwd_glr(ref, gate, px, pg, ps, pd, ph, pdx, pdg, p0, ws, nws, _raw(dev))
    _check(rc, "delta_bwd_glr")
    return g


def decode_glr(x, g_log, h, *, input_gate: str = "none", O=None, stream=None):
    """One token of the gated linear recurrence (delta_decode_glr): x [B,1,H,dv], g_log [B,1,H,dv]
    fp32, h [B,H,dv] fp32 updated in place.  Returns O [B,1,H,dv]."""
    shp, (ref, _, _) = _glr_shape(x)
    B, L, H, dv = shp
    if L != 1:
        raise ValueError("decode_glr takes one token: x must be [B, 1, H, dv]")
    gate, dev = _gate(input_gate), x.device
    with _on(dev, stream):
        px, pg = _arg(x, "x", shp, x.dtype, dev), _arg(g_log, "g_log", shp, _f32, dev)
        ph = _arg(h, "h", (B, H, dv), _f32, dev)
        O, po = _out(O, "O", shp, x.dtype, dev, x)
        rc = _load().delta_decode_glr(ref, gate, px, pg, ph, po, _raw(dev))
    _check(rc, "delta_decode_glr")
    return O


def _rows(x, name):
    code = _code(x, name)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("%s must be [..., width]" % name)
    width = x.shape[-1]
    return x.numel() // width, width, code


def layer_rmsnorm(x, weight, residual=None, *, eps: float = 1e-6, sum=None, y=None, stream=None):
    """s = x + residual (rounded to x's type) and y = s / sqrt(mean(s^2) + eps) * weight over the last
    dimension (delta_layer_rmsnorm); weight [width] fp32.  Returns (s, y); without a residual s is x
    itself.  Pass sum=residual to update the residual stream in place."""
    rows, width, code = _rows(x, "x")
    dev, shp = x.device, x.shape
    with _on(dev, stream):
        px, pr, pw = _arg(x, "x", shp, x.dtype, dev), _opt(residual, "residual", shp, x.dtype, dev), \
            _arg(weight, "weight", (width,), _f32, dev)
        ps = None
        if residual is not None:
            sum, ps = _out(sum, "sum", shp, x.dtype, dev, x)
        y, py = _out(y, "y", shp, x.dtype, dev, x)
        rc = _load().delta_layer_rmsnorm(rows, width, code, eps, px, pr, pw, ps, py, _raw(dev))
    _check(rc, "delta_layer_rmsnorm")
    return (x if residual is None else sum), y


def layer_rmsnorm_quant(x, weight, residual=None, *, eps: float = 1e-6, group: int = 128, sum=None, y8=None, scale=None,
                        stream=None):
    """layer_rmsnorm with its output in 8 bits (delta_layer_rmsnorm_quant): y ~ y8 * scale, y8 in
    torch.float8_e4m3fn, scale [..., ceil(width/group)] fp32 per `group` channels (128, or 0 for one
    per row: [..., 1]).  Returns (s, y8, scale)."""
    rows, width, code = _rows(x, "x")
    dev, shp = x.device, x.shape
    if group not in (0, 128):
        raise ValueError("group must be 0 (one scale per row) or 128, got %r" % (group,))
    sshp = shp[:-1] + (-(-width // group) if group else 1,)
    with _on(dev, stream):
        px, pr, pw = _arg(x, "x", shp, x.dtype, dev), _opt(residual, "residual", shp, x.dtype, dev), \
            _arg(weight, "weight", (width,), _f32, dev)
        ps = None
        if residual is not None:
            sum, ps = _out(sum, "sum", shp, x.dtype, dev, x)
        y8, py = _out(y8, "y8", shp, torch.float8_e4m3fn, dev, x)
        scale, pc = _out(scale, "scale", sshp, _f32, dev, x)
        rc = _load().delta_layer_rmsnorm_quant(rows, width, code, eps, group, px, pr, pw, ps, py, pc, _raw(dev))
    _check(rc, "delta_layer_rmsnorm_quant")
    return (x if residual is None else sum), y8, scale


@functools.lru_cache(maxsize=1024)
def rmsnorm_bwd_workspace_bytes(rows, width, dtype=BF16) -> int:
    """Workspace of layer_rmsnorm_bwd for this shape (none is used without dweight)."""
    return _bytes("delta_layer_rmsnorm_bwd_workspace_bytes", rows, width, dtype)


def layer_rmsnorm_bwd(dy, s, weight, dsum=None, *, eps: float = 1e-6, want_dweight: bool = True, dx=None, dweight=None,
                      workspace=None, stream=None):
    """Backward pass of layer_rmsnorm (delta_layer_rmsnorm_bwd) from its s; dsum is the gradient that
    reaches s past the norm (None for zero).  Returns (dx, dweight): dx, in s's type, is the gradient
    of x and of residual alike; dweight [width] fp32 is None unless want_dweight."""
    rows, width, code = _rows(s, "s")
    dev, shp = s.device, s.shape
    with _on(dev, stream):
        pdy, ps, pw = _arg(dy, "dy", shp, s.dtype, dev), _arg(s, "s", shp, s.dtype, dev), \
            _arg(weight, "weight", (width,), _f32, dev)
        pds, pdw = _opt(dsum, "dsum", shp, s.dtype, dev), None
        dx, pdx = _out(dx, "dx", shp, s.dtype, dev, s)
        if dweight is not None or want_dweight:
            dweight, pdw = _out(dweight, "dweight", (width,), _f32, dev, weight)
        need = 0 if pdw is None else rmsnorm_bwd_workspace_bytes(rows, width, code)
        ws, nws, keep = _workspace(workspace, need, dev)
        rc = _load().delta_layer_rmsnorm_bwd(rows, width, code, eps, pdy, ps, pw, pds, pdx, pdw, ws, nws, _raw(dev))
    _check(rc, "delta_layer_rmsnorm_bwd")
    return dx, dweight


def _grad_table(grads, dev, what):
    """Host arrays describing the tensors of a sequence or dict (Nones left out), all on device `dev` or,
    where that is None, on the first one's."""
    ts = [t for t in (grads.values() if isinstance(grads, dict) else grads) if t is not None]
    if not ts:
        raise ValueError("no %ss given" % what)
    if dev is None:
        _code(ts[0], "%s 0" % what)
        dev = ts[0].device
    T = torch.Tensor  # map over its methods and no ctypes arrays: this is most of a call on many tensors
    if set(map(T.get_device, ts)) != {dev.index} or not all(map(T.is_contiguous, ts)):
        raise ValueError("every %s must be a contiguous GPU tensor on %s" % (what, dev))
    codes = [_DTYPES.get(t.dtype) for t in ts]
    if None in codes:
        raise TypeError("every %s must be bfloat16 or float32" % what)
    return dev, len(ts), array.array("q", map(T.numel, ts)), array.array("i", codes), array.array("Q", map(T.data_ptr, ts))


def _outs_of(grads, out):
    """The outputs of the gradients that are not None, in the gradients' order: a dict's by name, a
    sequence's by place."""
    if isinstance(grads, dict):
        if not isinstance(out, dict) or out.keys() != grads.keys():
            raise ValueError("out must be a dict with the gradients' names")
        pairs = [(g, out[k]) for k, g in grads.items()]
    else:
        out = out if isinstance(out, dict) else list(out)
        if isinstance(out, dict) or len(out) != len(grads):
            raise ValueError("out must be a sequence as long as the gradients")
        pairs = list(zip(grads, out))
    outs = [o for g, o in pairs if g is not None]
    if any(o is None for o in outs):
        raise ValueError("out must have a tensor for every gradient")
    return outs


def _host(a):
    """Address of a host array (of its elements; the caller keeps it alive)."""
    return None if a is None else a.buffer_info()[0]


def _norm_or_clip(grads, clip, max_norm, eps, out, norm, workspace, stream):
    if not isinstance(grads, (dict, list, tuple)):
        grads = list(grads)
    dev, n, sizes, codes, ptrs = _grad_table(grads, None, "gradient")
    outs = None
    if out is not None:
        _, _, osizes, ocodes, outs = _grad_table(_outs_of(grads, out), dev, "output")
        if osizes != sizes or ocodes != codes:
            raise ValueError("out must match the gradients one by one in size and type")
    lib, hp, hs, hc = _load(), _host(ptrs), _host(sizes), _host(codes)
    with _on(dev, stream):
        if norm is None:
            norm = torch.empty((), dtype=_f32, device=dev)
        pn = _arg(norm, "norm", torch.Size(()), _f32, dev)
        ws, nws, keep = _workspace(workspace, _bytes("delta_grad_norm_workspace_bytes", n, hs), dev)
        if clip:
            rc = lib.delta_clip_grads(n, hp, hs, hc, max_norm, eps, _host(outs), pn, ws, nws, _raw(dev))
        else:
            rc = lib.delta_grad_norm(n, hp, hs, hc, pn, ws, nws, _raw(dev))
    _check(rc, "delta_clip_grads" if clip else "delta_grad_norm")
    return norm


def grad_norm(grads, *, norm=None, workspace=None, stream=None):
    """Global 2-norm of a sequence or dict of gradients (bf16 or fp32, Nones left out), as a float32
    scalar on the device (delta_grad_norm)."""
    return _norm_or_clip(grads, False, 0.0, 0.0, None, norm, workspace, stream)


def clip_grads(grads, max_norm: float, *, eps: float = 1e-6, out=None, norm=None, workspace=None, stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global 2-norm
    (delta_clip_grads): in place, or into `out` (tensors like the gradients: for a dict one with the same
    names, for a sequence one as long, read only where there is a gradient).  Returns the norm before
    clipping, a float32 scalar on the device."""
    return _norm_or_clip(grads, True, float(max_norm), float(eps), out, norm, workspace, stream)
