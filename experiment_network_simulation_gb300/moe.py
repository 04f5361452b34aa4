"""Routed-expert operators on torch tensors: the binding of mv_route,
mv_route_backward, mv_exchange and mv_experts (``include/mv.h``).

    ids, weights = route(logits, topk, ...)          # the router
    dlogits = route_backward(logits, ids, dweights)  # its gradient
    load, sent = exchange(ids, place, ranks)         # tokens from rank to rank
    y = experts(x, ids, weights, w13, s13, w2, s2)   # the chosen experts' products

``sent`` times the bytes of a token is the byte matrix that
:func:`.inputs.moe_workload` makes an all-to-all of.  Every call is enqueued
on ``stream`` (default: the current one of the inputs' device) and returns
without waiting; outputs and workspaces come from torch's allocator on that
stream, and nothing is recorded for autograd.  Malformed arguments raise
ValueError, what the library refuses :class:`.mv.MVError`.  There is no CPU
fallback: tensors have to be on a CUDA device.
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

from . import mv

SOFTMAX, SIGMOID = 0, 1
_SCORES = {"softmax": SOFTMAX, "sigmoid": SIGMOID}
_RULES = {"max": 0, "top2": 1}
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MAX_EXPERTS, MAX_TOPK, MAX_GROUPS, MAX_RANKS = 1024, 32, 32, 8192
_MAX_SCALE = torch.finfo(torch.float32).max        # the descriptors hold it in 32 bits

_vp, _u64 = C.c_void_p, C.c_uint64
_raw_stream = torch._C._cuda_getCurrentRawStream


def _descriptor(name: str, fields: str):
    """A mv_*_desc of ``include/mv.h`` as a ctypes structure (Q, I, f: 64-, 32-bit
    and float fields, P: pointers), and its packer: filling a structure field
    by field costs a call of these microseconds."""
    types = {"Q": _u64, "I": C.c_uint32, "f": C.c_float, "P": _vp}
    pairs = [f.split(":") for f in fields.split()]
    cls = type(name, (C.Structure,), {"_fields_": [(n, types[t]) for n, t in pairs]})
    packer = struct.Struct("@" + "".join(t for _, t in pairs))
    assert packer.size <= C.sizeof(cls) < packer.size + 8          # C pads the end
    return cls, packer.pack


RouteDesc, _route_desc = _descriptor(
    "RouteDesc", "tokens:Q row_stride:Q experts:I topk:I groups:I top_groups:I dtype:I scores:I "
    "group_rule:I renorm:I scale:f logits:P bias:P ids:P weights:P")
RouteGradDesc, _route_grad_desc = _descriptor(
    "RouteGradDesc", "tokens:Q row_stride:Q experts:I topk:I dtype:I scores:I renorm:I scale:f "
    "logits:P ids:P dweights:P dlogits:P")
ExchangeDesc, _exchange_desc = _descriptor(
    "ExchangeDesc", "batches:Q tokens:Q topk:I experts:I sources:I ranks:I once:I ids:P place:P "
    "starts:P load:P sent:P")
ExpertsDesc, _experts_desc = _descriptor(
    "ExpertsDesc", "tokens:Q row_stride:Q topk:I experts:I hidden:I inner:I group:I dtype:I x:P "
    "ids:P weights:P w13:P s13:P w2:P s2:P y:P")

_lib = None


def _library() -> C.CDLL:
    """libmv.so, its routed-expert calls declared (descriptors by address)."""
    global _lib
    if _lib is None:
        lib = mv.library()
        for f in ("mv_route", "mv_route_backward", "mv_exchange"):
            getattr(lib, f).argtypes = [_vp, _vp]
        lib.mv_experts_workspace_bytes.argtypes = [_vp, C.POINTER(_u64)]
        lib.mv_experts.argtypes = [_vp, _vp, _u64, _vp]
        for f in ("mv_route", "mv_route_backward", "mv_exchange", "mv_experts_workspace_bytes",
                  "mv_experts"):
            getattr(lib, f).restype = C.c_int
        _lib = lib
    return _lib


def _call(name: str, desc: bytes, index: int):
    """One enqueued call on the current stream of device ``index``."""
    rc = getattr(_lib or _library(), name)(desc, _raw_stream(index))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, name)


def _tensor(name: str, t, dtype, shape, device=None, rows_apart: bool = False):
    """Check one argument: type, device, shape (None: any size), dense layout."""
    if (t.__class__ is torch.Tensor and t.is_cuda and t.dtype in dtype and t.is_contiguous()
            and t.dim() == len(shape) and (device is None or t.device == device)):
        for s, n in zip(shape, t.shape):
            if s is not None and s != n:
                break
        else:
            return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is a torch tensor, not {type(t).__name__}")
    if not t.is_cuda:
        raise RuntimeError(f"{name} is on {t.device}; the operators need a CUDA device, "
                           "there is no CPU fallback")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype not in dtype:
        raise ValueError(f"{name} is {t.dtype}, not {' or '.join(str(d) for d in dtype)}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not "
                         f"({', '.join('any' if s is None else str(s) for s in shape)})")
    if rows_apart:
        if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{name}'s rows are not dense and apart (strides {t.stride()})")
    elif not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous (strides {t.stride()})")


def _stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


class _On:
    """The device and the stream of one call that are not the current ones."""

    def __init__(self, device, stream, inputs):
        self.stack = [torch.cuda.device(device)]
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, not on {device}")
            self.stack.append(torch.cuda.stream(stream))
            if stream != torch.cuda.current_stream(device):
                for t in inputs:
                    if t is not None:
                        t.record_stream(stream)

    def __enter__(self):
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


def _elsewhere(device, stream) -> bool:
    """Whether a call is not for the current device and stream."""
    return stream is not None or device.index != torch.cuda.current_device()


def _choice(what: str, value, table: dict) -> int:
    if value not in table:
        raise ValueError(f"{what} is one of {', '.join(table)}, not {value!r}")
    return table[value]


def route(logits, topk: int, *, scores: str = "softmax", bias=None, groups: int = 1,
          top_groups: int = 1, group_rule: str = "max", renorm: bool = True, scale: float = 1.0,
          stream=None):
    """Choose ``topk`` experts for every token: (ids int32, weights float32), [tokens, topk].

    ``logits`` [tokens, experts] (float32, float16 or bfloat16; rows may lie
    apart).  Experts are ordered by their ``scores`` ("softmax" or "sigmoid")
    plus ``bias`` (float32 [experts]), within the ``top_groups`` of ``groups``
    equal groups that have the greatest value: their best expert's ("max") or
    the sum of their two best ("top2").  Equal values go to the lowest index.
    The weights are the chosen experts' scores, without the bias, divided by
    their sum if ``renorm``, times ``scale``.  An expert whose logit or bias is
    -inf or NaN is closed (by the bias: for the choice alone, its share of the
    softmax stays its own); slots that no open expert is left for hold id -1
    and weight 0.
    """
    _tensor("logits", logits, _DTYPES, (None, None), rows_apart=True)
    tokens, n = logits.shape
    if not 1 <= n <= MAX_EXPERTS:
        raise ValueError(f"{n} experts: 1 to {MAX_EXPERTS} are taken")
    if not 1 <= groups <= MAX_GROUPS or n % groups:
        raise ValueError(f"{groups} groups: at most {MAX_GROUPS}, and {n} experts divide into them evenly")
    if not 1 <= top_groups <= groups:
        raise ValueError(f"top_groups is 1 to {groups}, not {top_groups}")
    most = min(MAX_TOPK, top_groups * (n // groups))
    if not 1 <= topk <= most:
        raise ValueError(f"topk is 1 to {most}, not {topk}")
    if not abs(scale) <= _MAX_SCALE:
        raise ValueError(f"scale is {scale}")
    s, r = _choice("scores", scores, _SCORES), _choice("group_rule", group_rule, _RULES)
    if bias is not None:
        _tensor("bias", bias, (torch.float32,), (n,), logits.device)
    dev = logits.device
    if _elsewhere(dev, stream):
        with _On(dev, stream, (logits, bias)):
            return _route(logits, tokens, n, topk, s, bias, groups, top_groups, r, renorm, scale, dev)
    return _route(logits, tokens, n, topk, s, bias, groups, top_groups, r, renorm, scale, dev)


def _route(logits, tokens, n, topk, s, bias, groups, top_groups, r, renorm, scale, dev):
    ids = torch.empty((tokens, topk), dtype=torch.int32, device=dev)
    weights = torch.empty((tokens, topk), dtype=torch.float32, device=dev)
    _call("mv_route", _route_desc(
        tokens, _stride(logits), n, topk, groups, top_groups, _DTYPES[logits.dtype], s, r,
        bool(renorm), scale, logits.data_ptr(), 0 if bias is None else bias.data_ptr(),
        ids.data_ptr(), weights.data_ptr()), dev.index)
    return ids, weights


def route_backward(logits, ids, dweights, *, scores: str = "softmax", renorm: bool = True,
                   scale: float = 1.0, stream=None):
    """Gradient of :func:`route`'s weights: dlogits, like ``logits`` and dense.

    ``ids`` are route's for these logits, ``dweights`` (float32) the weights'
    gradient.  The choice of experts and the bias have no gradient.
    """
    _tensor("logits", logits, _DTYPES, (None, None), rows_apart=True)
    tokens, n = logits.shape
    if not 1 <= n <= MAX_EXPERTS:
        raise ValueError(f"{n} experts: 1 to {MAX_EXPERTS} are taken")
    _tensor("ids", ids, (torch.int32,), (tokens, None), logits.device)
    topk = ids.shape[1]
    if not 1 <= topk <= min(MAX_TOPK, n):
        raise ValueError(f"topk is 1 to {min(MAX_TOPK, n)}, not {topk}")
    _tensor("dweights", dweights, (torch.float32,), (tokens, topk), logits.device)
    if not abs(scale) <= _MAX_SCALE:
        raise ValueError(f"scale is {scale}")
    s = _choice("scores", scores, _SCORES)
    dev = logits.device
    if _elsewhere(dev, stream):
        with _On(dev, stream, (logits, ids, dweights)):
            return _route_backward(logits, tokens, n, topk, ids, dweights, s, renorm, scale, dev)
    return _route_backward(logits, tokens, n, topk, ids, dweights, s, renorm, scale, dev)


def _route_backward(logits, tokens, n, topk, ids, dweights, s, renorm, scale, dev):
    out = torch.empty((tokens, n), dtype=logits.dtype, device=dev)
    _call("mv_route_backward", _route_grad_desc(
        tokens, _stride(logits), n, topk, _DTYPES[logits.dtype], s, bool(renorm), scale,
        logits.data_ptr(), ids.data_ptr(), dweights.data_ptr(), out.data_ptr()), dev.index)
    return out


def exchange(ids, place, ranks: int, *, sources: int | None = None, starts=None,
             once: bool = True, stream=None):
    """Count an expert-parallel exchange: (load [experts], sent [sources, ranks]), int32.

    ``ids`` int32 [tokens, topk], or [batches, tokens, topk] for as many
    independent exchanges (both results then get that dimension).  Tokens lie
    by source rank: equal shares of ``sources`` (default: ``ranks``), or
    ``starts`` (ascending int64 [sources + 1], on the device; tokens outside
    them count nowhere).  ``place`` int32 [experts] is the rank an expert lives
    on.  ``sent[s, d]`` counts the tokens of s with an expert on d, or without
    ``once`` every one of their experts there; ``load[e]`` the slots that hold
    e.  Ids outside [0, experts) are empty slots.
    """
    if isinstance(ids, torch.Tensor) and ids.dim() == 2:
        _tensor("ids", ids, (torch.int32,), (None, None))
        batches, (tokens, topk), lead = 1, ids.shape, ()
    else:
        _tensor("ids", ids, (torch.int32,), (None, None, None))
        batches, tokens, topk = ids.shape
        lead = (batches,)
    _tensor("place", place, (torch.int32,), (None,), ids.device)
    n = place.shape[0]
    if not 1 <= n <= MAX_EXPERTS:
        raise ValueError(f"{n} experts: 1 to {MAX_EXPERTS} are taken")
    if not 1 <= topk <= MAX_TOPK:
        raise ValueError(f"topk is 1 to {MAX_TOPK}, not {topk}")
    if not 1 <= ranks <= MAX_RANKS:
        raise ValueError(f"ranks is 1 to {MAX_RANKS}, not {ranks}")
    if starts is not None:
        _tensor("starts", starts, (torch.int64,), (None,), ids.device)
        if not (starts.shape[0] >= 2 and sources in (None, starts.shape[0] - 1)):
            raise ValueError(f"starts holds {starts.shape[0]} offsets, not one more than the sources")
        sources = starts.shape[0] - 1
    else:
        sources = ranks if sources is None else sources
        if not (sources >= 1 and tokens % sources == 0):
            raise ValueError(f"{tokens} tokens do not divide evenly over {sources} sources; give starts")
    dev = ids.device
    if _elsewhere(dev, stream):
        with _On(dev, stream, (ids, place, starts)):
            return _exchange(ids, lead, batches, tokens, topk, place, n, starts, sources, ranks, once, dev)
    return _exchange(ids, lead, batches, tokens, topk, place, n, starts, sources, ranks, once, dev)


def _exchange(ids, lead, batches, tokens, topk, place, n, starts, sources, ranks, once, dev):
    load = torch.empty((*lead, n), dtype=torch.int32, device=dev)
    sent = torch.empty((*lead, sources, ranks), dtype=torch.int32, device=dev)
    _call("mv_exchange", _exchange_desc(
        batches, tokens, topk, n, sources, ranks, bool(once), ids.data_ptr(), place.data_ptr(),
        0 if starts is None else starts.data_ptr(), load.data_ptr(), sent.data_ptr()), dev.index)
    return load, sent


def experts(x, ids, weights, w13, s13, w2, s2, *, stream=None):
    """The chosen experts' products, [tokens, hidden] of ``x``'s type:
    sum over a token's slots of weight * W2 (silu(W1 x) * (W3 x)).

    ``x`` [tokens, hidden] (float16 or bfloat16; rows may lie apart by a
    multiple of 8), ``ids`` int32 and ``weights`` float32 [tokens, topk].
    ``w13`` uint8 [experts, 2 * inner, hidden / 2] holds W1's rows, then W3's,
    two 4-bit numbers to a byte (the even column in the low half), ``s13``
    [experts, 2 * inner, hidden / group] their scales in ``x``'s type:
    W = (q - 8) * scale.  ``w2`` [experts, hidden, inner / 2] and ``s2``
    [experts, hidden, inner / group] likewise, group 32, 64 or 128.  Ids
    outside [0, experts) add nothing (experts of other ranks).
    """
    _tensor("x", x, (torch.float16, torch.bfloat16), (None, None), rows_apart=True)
    tokens, hidden = x.shape
    dev = x.device
    _tensor("w13", w13, (torch.uint8,), (None, None, None), dev)
    n, inner2 = w13.shape[0], w13.shape[1]
    inner = inner2 // 2
    if not 1 <= n <= MAX_EXPERTS:
        raise ValueError(f"{n} experts: 1 to {MAX_EXPERTS} are taken")
    if not (hidden >= 32 and inner2 >= 64 and inner2 % 2 == 0 and 2 * w13.shape[2] == hidden):
        raise ValueError(f"w13 has shape {tuple(w13.shape)}, not [experts, 2 * inner, {hidden} / 2]")
    _tensor("s13", s13, (x.dtype,), (n, inner2, None), dev)
    group = hidden // s13.shape[2] if s13.shape[2] else 0
    if not (group in (32, 64, 128) and hidden == group * s13.shape[2] and inner % group == 0):
        raise ValueError(f"s13 has shape {tuple(s13.shape)}: a scale stands for 32, 64 or 128 of {hidden} columns, "
                         f"and {inner} inner rows divide by that too")
    _tensor("w2", w2, (torch.uint8,), (n, hidden, inner // 2), dev)
    _tensor("s2", s2, (x.dtype,), (n, hidden, inner // group), dev)
    _tensor("ids", ids, (torch.int32,), (tokens, None), dev)
    topk = ids.shape[1]
    if not 1 <= topk <= MAX_TOPK:
        raise ValueError(f"topk is 1 to {MAX_TOPK}, not {topk}")
    _tensor("weights", weights, (torch.float32,), (tokens, topk), dev)
    if _elsewhere(dev, stream):
        with _On(dev, stream, (x, ids, weights, w13, s13, w2, s2)):
            return _experts(x, tokens, topk, n, hidden, inner, group, ids, weights, w13, s13, w2, s2, dev)
    return _experts(x, tokens, topk, n, hidden, inner, group, ids, weights, w13, s13, w2, s2, dev)


def _experts(x, tokens, topk, n, hidden, inner, group, ids, weights, w13, s13, w2, s2, dev):
    lib, need = _lib or _library(), _u64()
    y = torch.empty((tokens, hidden), dtype=x.dtype, device=dev)
    d = _experts_desc(tokens, _stride(x), topk, n, hidden, inner, group, _DTYPES[x.dtype],
                      x.data_ptr(), ids.data_ptr(), weights.data_ptr(), w13.data_ptr(),
                      s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), y.data_ptr())
    rc = lib.mv_experts_workspace_bytes(d, C.byref(need))
    if rc == mv.MV_OK:
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        rc = lib.mv_experts(d, ws.data_ptr(), need.value, _raw_stream(dev.index))
    if rc != mv.MV_OK:
        raise mv.MVError(rc, "mv_experts")
    return y
