"""Block operators on torch tensors: the binding of mv_linear, mv_linear_backward,
mv_activation_backward, mv_norm and mv_norm_backward (``include/mv.h``).

    n, r = norm(y, weight, residual=r, gate=gate, ...)   # after a branch, before the next
    grads = norm_backward(dn, y, weight, dr=dr, ...)
    y = linear(x, w, bias, act="gelu", residual=r)       # dense layer, router's logits
    dz = activation_backward(dy, z, act="gelu")
    dx, dw, dbias = linear_backward(dz, x, w)

They stand around :mod:`.moe`'s operators: ``linear`` makes the logits that
:func:`.moe.route` takes and ``linear_backward`` takes what
:func:`.moe.route_backward` gives on to the router's weights and its input;
``norm`` gives :func:`.moe.experts` its x and takes up its y.  Calls, streams,
outputs, workspaces and errors are as there: enqueued on ``stream`` (default:
the current one of the inputs' device) without waiting, outputs and workspaces
from torch's allocator, nothing recorded for autograd, ValueError for malformed
arguments, :class:`.mv.MVError` for what the library refuses, no CPU fallback.
A product whose kernel waited two seconds in vain (a broken device, or one that was
stopped) is incomplete, and only :func:`gave_up` tells.
"""
from __future__ import annotations

import ctypes as C
from collections import namedtuple

import torch

from . import mv
from .moe import _DTYPES, _On, _choice, _descriptor, _raw_stream, _tensor, _u64, _vp

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_HALVES = (torch.float16, torch.bfloat16)
_current_device = torch._C._cuda_getDevice
_MAX_SCALE = torch.finfo(torch.float32).max        # the descriptors hold it in 32 bits

LinearDesc, _linear_desc = _descriptor(
    "LinearDesc", "tokens:Q cols:Q rows:Q x_stride:Q w_stride:Q residual_stride:Q dtype:I out_dtype:I "
    "bias_dtype:I act:I scale:f x:P w:P bias:P residual:P y:P z:P")
LinearGradDesc, _linear_grad_desc = _descriptor(
    "LinearGradDesc", "tokens:Q cols:Q rows:Q x_stride:Q w_stride:Q dz_stride:Q dtype:I dz_dtype:I "
    "dz:P x:P w:P dx:P dw:P dbias:P")
ActGradDesc, _act_grad_desc = _descriptor(
    "ActGradDesc", "tokens:Q cols:Q dy_stride:Q z_stride:Q dtype:I act:I scale:f dy:P z:P dz:P")

NormDesc, _norm_desc = _descriptor(
    "NormDesc", "tokens:Q hidden:Q gates:Q y_stride:Q residual_stride:Q dtype:I param_dtype:I kind:I "
    "alpha:f eps:f y:P residual:P weight:P bias:P post:P post_bias:P gate:P")
NormGradDesc, _norm_grad_desc = _descriptor(
    "NormGradDesc", "dn_stride:Q dr_stride:Q dn:P dr:P dy:P dresidual:P dweight:P dbias:P dpost:P dpost_bias:P dgate:P")

KINDS = {"rms": 0, "layer": 1}
MAX_HIDDEN = 16384
NormGrads = namedtuple("NormGrads", "dy dresidual dweight dbias dpost dpost_bias dgate")
_lib = None


def _library() -> C.CDLL:
    """libmv.so, its block operators declared (descriptors by address)."""
    global _lib
    if _lib is None:
        lib = mv.library()
        for f in ("mv_linear", "mv_linear_backward"):
            getattr(lib, f).argtypes = [_vp, _vp, _u64, _vp]
            getattr(lib, f + "_workspace_bytes").argtypes = [_vp, C.POINTER(_u64)]
        lib.mv_activation_backward.argtypes = [_vp, _vp]
        lib.mv_norm.argtypes = [_vp, _vp, _vp, _vp]
        lib.mv_norm_backward_workspace_bytes.argtypes = [_vp, _vp, C.POINTER(_u64)]
        lib.mv_norm_backward.argtypes = [_vp, _vp, _vp, _u64, _vp]
        lib.mv_block_status.argtypes = [C.POINTER(C.c_uint32)]
        _lib = lib
    return _lib


def _run(name: str, desc: bytes, dev):
    """One enqueued call on the current stream of ``dev``; without a workspace
    first, as small sizes need none."""
    lib = _lib or _library()
    call, stream = getattr(lib, name), _raw_stream(dev.index)
    rc = call(desc, 0, 0, stream)
    if rc == mv.MV_ENOMEM:
        need = _u64()
        rc = getattr(lib, name + "_workspace_bytes")(desc, C.byref(need))
        if rc == mv.MV_OK:
            ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
            rc = call(desc, ws.data_ptr(), need.value, stream)
    if rc != mv.MV_OK:
        raise mv.MVError(rc, name)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _apart(t, rows: int, cols: int) -> int:
    """How far the rows of ``t`` (or None) lie apart; of one row, its columns."""
    return cols if rows < 2 or t is None else t.stride(0)


def _scale(name: str, v: float):
    if not abs(v) <= _MAX_SCALE:
        raise ValueError(f"{name} is {v}")


def linear(x, w, bias=None, *, act: str = "none", residual=None, scale: float = 1.0,
           out_dtype=None, keep: bool = False, stream=None):
    """y = residual + scale * act(x w^T + bias), [tokens, rows] of ``out_dtype``.

    ``x`` [tokens, cols] and ``w`` [rows, cols] are float16 or bfloat16, both
    alike; their rows may lie apart, and rows that are not 16-byte aligned cost a
    copy.  ``bias`` [rows] is of their type or float32, ``residual`` [tokens,
    rows] (rows may lie apart) of ``out_dtype``: x's type (the default) or
    float32.  ``act`` is "none", "relu", "gelu", "gelu_tanh" (gelu in its
    hyperbolic-tangent form) or "silu".  With ``keep`` the result is (y, z), z
    the pre-activations x w^T + bias in x's type, as
    :func:`activation_backward` takes them.
    """
    _tensor("x", x, _HALVES, (None, None), rows_apart=True)
    tokens, cols = x.shape
    dev, dt = x.device, x.dtype
    _tensor("w", w, (dt,), (None, cols), dev, rows_apart=True)
    rows = w.shape[0]
    if not cols:
        raise ValueError("a product of no columns")
    out = dt if out_dtype is None else out_dtype
    if out is not dt and out is not torch.float32:
        raise ValueError(f"out_dtype is {dt} or torch.float32, not {out}")
    if bias is not None:
        _tensor("bias", bias, (dt, torch.float32), (rows,), dev)
    if residual is not None:
        _tensor("residual", residual, (out,), (tokens, rows), dev, rows_apart=True)
    a = _choice("act", act, ACTS)
    _scale("scale", scale)
    if stream is not None or dev.index != _current_device():
        with _On(dev, stream, (x, w, bias, residual)):
            return _linear(x, w, bias, residual, tokens, cols, rows, dt, out, a, scale, keep, dev)
    return _linear(x, w, bias, residual, tokens, cols, rows, dt, out, a, scale, keep, dev)


def _linear(x, w, bias, residual, tokens, cols, rows, dt, out, act, scale, keep, dev):
    y = torch.empty((tokens, rows), dtype=out, device=dev)
    z = torch.empty((tokens, rows), dtype=dt, device=dev) if keep else None
    if tokens and rows:
        _run("mv_linear", _linear_desc(
            tokens, cols, rows, _apart(x, tokens, cols), _apart(w, rows, cols), _apart(residual, tokens, rows),
            _DTYPES[dt], _DTYPES[out], _DTYPES[dt if bias is None else bias.dtype], act, scale,
            x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(z)), dev)
    return (y, z) if keep else y


def linear_backward(dz, x, w, *, dx: bool = True, dw: bool = True, bias: bool = False, stream=None):
    """Gradients of z = x w^T + bias, given z's: (dx, dw, dbias), of x's type.

    ``dz`` [tokens, rows] is of x's type, or float32 where that is bfloat16 (each
    value then counts to 2^-17 of itself, and times an infinity is a NaN); its
    rows may lie apart.  ``dx = dz w`` [tokens, cols], ``dw = dz^T x`` [rows,
    cols] and, with ``bias``, ``dbias`` [rows], the sum over the tokens; None
    for what is not asked for.  A gradient at the output of :func:`linear` goes
    through :func:`activation_backward` first; the residual's is that gradient
    itself.
    """
    _tensor("x", x, _HALVES, (None, None), rows_apart=True)
    tokens, cols = x.shape
    dev, dt = x.device, x.dtype
    _tensor("w", w, (dt,), (None, cols), dev, rows_apart=True)
    rows = w.shape[0]
    if not cols:
        raise ValueError("a product of no columns")
    _tensor("dz", dz, (dt, torch.float32) if dt is torch.bfloat16 else (dt,), (tokens, rows), dev, rows_apart=True)
    if stream is not None or dev.index != _current_device():
        with _On(dev, stream, (dz, x, w)):
            return _linear_backward(dz, x, w, tokens, cols, rows, dt, dx, dw, bias, dev)
    return _linear_backward(dz, x, w, tokens, cols, rows, dt, dx, dw, bias, dev)


def _linear_backward(dz, x, w, tokens, cols, rows, dt, dx, dw, bias, dev):
    gx = torch.empty((tokens, cols), dtype=dt, device=dev) if dx else None
    gw = torch.empty((rows, cols), dtype=dt, device=dev) if dw else None
    gb = torch.empty((rows,), dtype=dt, device=dev) if bias else None
    if not rows:
        if dx:
            gx.zero_()
        return gx, gw, gb
    _run("mv_linear_backward", _linear_grad_desc(
        tokens, cols, rows, _apart(x, tokens, cols), _apart(w, rows, cols), _apart(dz, tokens, rows), _DTYPES[dt], _DTYPES[dz.dtype],
        dz.data_ptr(), x.data_ptr(), w.data_ptr(), _ptr(gx), _ptr(gw), _ptr(gb)), dev)
    return gx, gw, gb


def activation_backward(dy, z, *, act: str, scale: float = 1.0, stream=None):
    """dz = scale * dy * act'(z): a gradient at :func:`linear`'s y, taken to its z.

    ``dy`` and ``z`` [tokens, cols] (float32, float16 or bfloat16, both alike;
    rows may lie apart), ``act`` and ``scale`` as there.
    """
    _tensor("z", z, _DTYPES, (None, None), rows_apart=True)
    tokens, cols = z.shape
    _tensor("dy", dy, (z.dtype,), (tokens, cols), z.device, rows_apart=True)
    a = _choice("act", act, ACTS)
    _scale("scale", scale)
    dev = z.device
    if stream is not None or dev.index != _current_device():
        with _On(dev, stream, (dy, z)):
            return _activation_backward(dy, z, tokens, cols, a, scale, dev)
    return _activation_backward(dy, z, tokens, cols, a, scale, dev)


def _activation_backward(dy, z, tokens, cols, act, scale, dev):
    dz = torch.empty((tokens, cols), dtype=z.dtype, device=dev)
    rc = (_lib or _library()).mv_activation_backward(_act_grad_desc(
        tokens, cols, _apart(dy, tokens, cols), _apart(z, tokens, cols), _DTYPES[z.dtype], act, scale, dy.data_ptr(), z.data_ptr(),
        dz.data_ptr()), _raw_stream(dev.index))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, "mv_activation_backward")
    return dz


def norm(y, weight, bias=None, *, residual=None, alpha: float = 1.0, post=None, post_bias=None,
         gate=None, kind: str = "rms", eps: float = 1e-6, stream=None):
    """The norms after a branch and before the next one: (n, r), [tokens, hidden] of ``y``'s type.

        u = N(y) * post + post_bias       (y without post)
        r = alpha * residual + gate * u   (without what is None)
        n = N(r) * weight + bias

    ``y`` [tokens, hidden] (float32, float16 or bfloat16) is what the branch
    gave, ``residual`` the stream beside it (y's type; the rows of both may lie
    apart).  N divides by the root mean square ("rms") or takes the mean off
    first ("layer"); ``eps`` is added to the mean square.  The parameters
    ``weight``, ``bias``, ``post``, ``post_bias`` [hidden] and ``gate`` are all
    of y's type or all float32.  ``gate`` is [hidden], or [gates, hidden] where
    gates divides tokens: each row for as many tokens in a row.  r is the new
    stream; n is normed from r before its rounding.  Without residual, post and
    gate there is no new stream, and r is ``y`` itself.
    """
    tokens, hidden, gates, k, params, dev = _norm_checks(y, weight, bias, residual, alpha, post, post_bias, gate, kind, eps)
    if stream is not None or dev.index != _current_device():
        with _On(dev, stream, (y, weight, bias, residual, post, post_bias, gate)):
            return _norm(y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates, k, params, eps, dev)
    return _norm(y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates, k, params, eps, dev)


def _norm_checks(y, weight, bias, residual, alpha, post, post_bias, gate, kind, eps):
    _tensor("y", y, _DTYPES, (None, None), rows_apart=True)
    tokens, hidden = y.shape
    dev = y.device
    if not 1 <= hidden <= MAX_HIDDEN:
        raise ValueError(f"hidden is 1 to {MAX_HIDDEN}, not {hidden}")
    _tensor("weight", weight, (y.dtype, torch.float32), (hidden,), dev)
    params = weight.dtype
    if bias is not None:
        _tensor("bias", bias, (params,), (hidden,), dev)
    if residual is not None:
        _tensor("residual", residual, (y.dtype,), (tokens, hidden), dev, rows_apart=True)
    if post is not None:
        _tensor("post", post, (params,), (hidden,), dev)
    if post_bias is not None:
        if post is None:
            raise ValueError("post_bias needs post")
        _tensor("post_bias", post_bias, (params,), (hidden,), dev)
    gates = 1
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 1:
            _tensor("gate", gate, (params,), (hidden,), dev)
        else:
            _tensor("gate", gate, (params,), (None, hidden), dev)
            gates = gate.shape[0]
        if gates < 1 or tokens % gates:
            raise ValueError(f"{gates} gates do not divide {tokens} tokens evenly")
    _scale("alpha", alpha)
    if not 0.0 <= eps <= _MAX_SCALE:
        raise ValueError(f"eps is {eps}")
    return tokens, hidden, gates, _choice("kind", kind, KINDS), params, dev


def _norm(y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates, kind, params, eps, dev):
    n = torch.empty((tokens, hidden), dtype=y.dtype, device=dev)
    same = residual is None and post is None and gate is None
    r = y if same else torch.empty((tokens, hidden), dtype=y.dtype, device=dev)
    rc = (_lib or _library()).mv_norm(_norm_desc(
        tokens, hidden, gates, _apart(y, tokens, hidden), _apart(residual, tokens, hidden), _DTYPES[y.dtype],
        _DTYPES[params], kind, alpha, eps, y.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), _ptr(post),
        _ptr(post_bias), _ptr(gate)), n.data_ptr(), 0 if same else r.data_ptr(), _raw_stream(dev.index))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, "mv_norm")
    return n, r


def norm_backward(dn, y, weight, bias=None, *, dr=None, residual=None, alpha: float = 1.0, post=None,
                  post_bias=None, gate=None, kind: str = "rms", eps: float = 1e-6, stream=None):
    """Gradients of :func:`norm`'s n and r, given ``dn`` and (unless None) ``dr``.

    The other arguments are norm's.  The result is a NormGrads (dy, dresidual,
    dweight, dbias, dpost, dpost_bias, dgate): of y's type the first two, of the
    parameters' type the others, each like what it is the gradient of and None
    where that is None.  The statistics are computed again, so norm keeps none.
    ``dn`` and ``dr`` [tokens, hidden] are of y's type; their rows may lie apart.
    """
    tokens, hidden, gates, k, params, dev = _norm_checks(y, weight, bias, residual, alpha, post, post_bias, gate, kind, eps)
    _tensor("dn", dn, (y.dtype,), (tokens, hidden), dev, rows_apart=True)
    if dr is not None:
        _tensor("dr", dr, (y.dtype,), (tokens, hidden), dev, rows_apart=True)
    if stream is not None or dev.index != _current_device():
        with _On(dev, stream, (dn, dr, y, weight, bias, residual, post, post_bias, gate)):
            return _norm_backward(dn, dr, y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates,
                                  k, params, eps, dev)
    return _norm_backward(dn, dr, y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates, k,
                          params, eps, dev)


def _norm_backward(dn, dr, y, weight, bias, residual, alpha, post, post_bias, gate, tokens, hidden, gates, kind, params,
                   eps, dev):
    def like(p, dtype, *shape):
        return None if p is None else torch.empty(shape, dtype=dtype, device=dev)

    g = NormGrads(like(y, y.dtype, tokens, hidden), like(residual, y.dtype, tokens, hidden), like(weight, params, hidden),
                  like(bias, params, hidden), like(post, params, hidden), like(post_bias, params, hidden),
                  None if gate is None else like(gate, params, *gate.shape))
    d = _norm_desc(
        tokens, hidden, gates, _apart(y, tokens, hidden), _apart(residual, tokens, hidden), _DTYPES[y.dtype],
        _DTYPES[params], kind, alpha, eps, y.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), _ptr(post),
        _ptr(post_bias), _ptr(gate))
    e = _norm_grad_desc(_apart(dn, tokens, hidden), _apart(dr, tokens, hidden), dn.data_ptr(), _ptr(dr), *map(_ptr, g))
    lib, need = _lib or _library(), _u64()
    rc = lib.mv_norm_backward_workspace_bytes(d, e, C.byref(need))
    if rc == mv.MV_OK:
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        rc = lib.mv_norm_backward(d, e, _ptr(ws), need.value, _raw_stream(dev.index))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, "mv_norm_backward")
    return g


def gave_up() -> int:
    """How many waits of the products' kernels ran into their limit on the
    current device: not 0 only if it is broken, or stopped for seconds.  Waits for the device."""
    n = C.c_uint32()
    rc = (_lib or _library()).mv_block_status(C.byref(n))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, "mv_block_status")
    return n.value
