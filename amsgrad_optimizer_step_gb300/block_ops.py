"""Binding of the residual blocks' operators (``include/fa_block_ops.h``).

Dropout from a counter-based generator, the join of a block's output to the residual stream
with the norms behind and before it, and the router of gated experts with its balance loss:
each function marshals torch tensors into the C call of the same name, as ``model_ops``
does.  Outputs and scratch are the caller's; the ``*_buffers`` helpers make them.
``layers`` has the same operators with autograd.  The RUDA documentation pages cover the
optimizer only and have no counterpart to these.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import FaDropoutKey, FaJoin, FaJoinGradient, FaRouter, FaRouting, check
from .model_ops import _FLOATS, _code, _matrix, _rows, _stream, _vector

__all__ = [
    "fa_dropout", "fa_block_join", "fa_block_join_scratch", "fa_block_join_gradient", "fa_route",
    "fa_route_scratch", "fa_route_gradient", "Dropout", "Join", "join_scratch", "RouteBuffers",
    "route_buffers",
]

_U64 = (1 << 64) - 1
_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


# A generation step's call is bound by the host: what a tensor is asked is asked once, and in the
# order in which it is usually right; a refusal's message is built on the way out.

def _mat(name: str, t: torch.Tensor, shape, dtype) -> tuple[int, int]:
    """Pointer and row distance of a matrix of this shape and type, with adjacent elements in a
    row."""
    if t.dtype is dtype and t.is_contiguous() and t.shape == shape:
        return t.data_ptr(), shape[1]
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    return t.data_ptr(), _rows(name, t, shape)


def _mat_or_none(name: str, t: Optional[torch.Tensor], shape, dtype) -> tuple[Optional[int], int]:
    if t is None:
        return None, shape[1]
    if t.dtype is dtype and t.is_contiguous() and t.shape == shape:
        return t.data_ptr(), shape[1]
    return _mat(name, t, shape, dtype)


def _vec_or_none(name: str, t: Optional[torch.Tensor], n: int, dtype) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    return _vector(name, t, n, dtype)


# ---- dropout -----------------------------------------------------------------------

class Dropout(NamedTuple):
    """Which elements a dropout keeps: the same record drops the same places of a matrix of as
    many columns, in every call and on every layout (see fa_dropout_key)."""
    p: float
    seed: int = 0
    offset: int = 0  # the call's own
    counter: Optional[torch.Tensor] = None  # int64 [1] on the device, added to offset


def _key(drop: Dropout) -> FaDropoutKey:
    p, seed, offset, counter = drop
    return FaDropoutKey(p, seed & _U64, offset & _U64, _vec_or_none("counter", counter, 1, _I64))


def fa_dropout(x: torch.Tensor, out: torch.Tensor, drop: Dropout, stream=None) -> None:
    """out = x with elements dropped and the others multiplied by 1 / (1 - p); its gradient is
    the same call on the output's.  out may be x itself."""
    rows, cols = shape = _matrix("x", x)
    dtype = x.dtype
    ptr, ld = _mat("x", x, shape, dtype)
    to, to_ld = _mat("out", out, shape, dtype)
    check("fa_dropout", _lib.load().fa_dropout(
        rows, cols, ptr, ld, _code("x", x, _FLOATS), ctypes.byref(_key(drop)), to, to_ld,
        _stream(stream)))


# ---- the join of a block to the residual stream ------------------------------------------

class Join(NamedTuple):
    """The constants of a join (see fa_join)."""
    post_norm: bool = True
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    eps: float = 1e-6
    weight_offset: float = 0.0
    dropout: Optional[Dropout] = None


_JOIN = Join()


def _join_record(j: Join, shape, dtype, stream_dtype, branch, post_weight, pre_weight, gate):
    """The C record (which keeps the key it points to), and the weights' type."""
    rows, cols = shape
    some = post_weight if post_weight is not None else pre_weight if pre_weight is not None else gate
    wdtype = dtype if some is None else some.dtype
    post_norm, residual_scale, branch_scale, eps, weight_offset, drop = j
    y, y_ld = _mat_or_none("branch", branch, shape, dtype)
    w1 = _vec_or_none("post_weight", post_weight, cols, wdtype)
    w2 = _vec_or_none("pre_weight", pre_weight, cols, wdtype)
    g, g_ld, groups = None, cols, 1
    if gate is not None:
        groups = _matrix("gate", gate)[0]
        g, g_ld = _mat("gate", gate, (groups, cols), wdtype)
    codes = _FLOATS.get
    record = FaJoin(rows, cols, codes(dtype, -1), codes(stream_dtype, -1), codes(wdtype, -1),
                    bool(post_norm), y, y_ld, w1, w2, g, g_ld, groups, residual_scale,
                    branch_scale, eps, weight_offset)
    if drop is not None:
        record.key = _key(drop)
        record.dropout = ctypes.addressof(record.key)
    return record, wdtype


def fa_block_join(join: Optional[Join], residual: torch.Tensor, branch: Optional[torch.Tensor],
                  out: Optional[torch.Tensor], normed: Optional[torch.Tensor] = None,
                  post_rstd: Optional[torch.Tensor] = None,
                  pre_rstd: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None,
                  pre_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = residual_scale * residual + branch_scale * gate * dropout(norm(branch)), and normed
    = the norm of out as it is stored.  The rstd vectors keep what the gradient takes.  out may
    be the residual itself.  The branch's type is normed's too (without a branch normed's own)."""
    shape = _matrix("residual", residual)
    typed = branch if branch is not None else normed if normed is not None else residual
    dtype, stream_dtype = typed.dtype, residual.dtype
    record, _ = _join_record(join or _JOIN, shape, dtype, stream_dtype, branch, post_weight,
                             pre_weight, gate)
    r, r_ld = _mat("residual", residual, shape, stream_dtype)
    o, o_ld = _mat_or_none("out", out, shape, stream_dtype)
    n, n_ld = _mat_or_none("normed", normed, shape, dtype)
    check("fa_block_join", _lib.load().fa_block_join(
        ctypes.byref(record), r, r_ld, o, o_ld, n, n_ld,
        _vec_or_none("post_rstd", post_rstd, shape[0], _F32),
        _vec_or_none("pre_rstd", pre_rstd, shape[0], _F32), _stream(stream)))


def fa_block_join_scratch(rows: int, cols: int, groups: int) -> int:
    """Bytes of scratch fa_block_join_gradient needs (groups: the gate's, 0 for none)."""
    out = ctypes.c_int64()
    check("fa_block_join_scratch",
          _lib.load().fa_block_join_scratch(rows, cols, groups, ctypes.byref(out)))
    return out.value


def join_scratch(rows: int, cols: int, groups: int, device) -> torch.Tensor:
    """Scratch for fa_block_join_gradient of these sizes."""
    return torch.empty(max(16, fa_block_join_scratch(rows, cols, groups)), dtype=torch.uint8,
                       device=device)


def fa_block_join_gradient(join: Optional[Join], out: Optional[torch.Tensor],
                           branch: Optional[torch.Tensor], dout: Optional[torch.Tensor],
                           dnormed: Optional[torch.Tensor], dresidual: Optional[torch.Tensor],
                           dbranch: Optional[torch.Tensor], scratch: Optional[torch.Tensor],
                           post_rstd: Optional[torch.Tensor] = None,
                           pre_rstd: Optional[torch.Tensor] = None,
                           post_weight: Optional[torch.Tensor] = None,
                           pre_weight: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None,
                           dpost_weight: Optional[torch.Tensor] = None,
                           dpre_weight: Optional[torch.Tensor] = None,
                           dgate: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of fa_block_join, from the stream as it stored it (``out``), the branch and the
    rstd vectors.  dout or dnormed may be None (no gradient; no second norm); a result that is
    None is not taken."""
    typed = branch if branch is not None else dnormed
    streamed = dout if dout is not None else out
    if typed is None and streamed is None:
        raise ValueError("neither a branch nor a gradient is given")
    if typed is None:
        typed = streamed
    elif streamed is None:
        streamed = dresidual if dresidual is not None else typed
    rows, cols = shape = _matrix("branch", typed)
    dtype, stream_dtype = typed.dtype, streamed.dtype
    record, wdtype = _join_record(join or _JOIN, shape, dtype, stream_dtype, branch, post_weight,
                                  pre_weight, gate)
    g = FaJoinGradient(
        *_mat_or_none("out", out, shape, stream_dtype),
        _vec_or_none("post_rstd", post_rstd, rows, _F32),
        _vec_or_none("pre_rstd", pre_rstd, rows, _F32),
        *_mat_or_none("dout", dout, shape, stream_dtype),
        *_mat_or_none("dnormed", dnormed, shape, dtype),
        *_mat_or_none("dresidual", dresidual, shape, stream_dtype),
        *_mat_or_none("dbranch", dbranch, shape, dtype),
        _vec_or_none("dpost_weight", dpost_weight, cols, wdtype),
        _vec_or_none("dpre_weight", dpre_weight, cols, wdtype),
        *_mat_or_none("dgate", dgate, (record.groups, cols), wdtype))
    if scratch is not None:
        size = scratch.numel()
        g.scratch, g.scratch_bytes = _vec_or_none("scratch", scratch, size, _U8), size
    check("fa_block_join_gradient", _lib.load().fa_block_join_gradient(
        ctypes.byref(record), ctypes.byref(g), _stream(stream)))


# ---- the router --------------------------------------------------------------------------

class RouteBuffers(NamedTuple):
    """Outputs of fa_route."""
    chosen: torch.Tensor                  # int32 [tokens, k] experts, the largest logit first
    weights: torch.Tensor                 # FP32 [tokens, k]
    lse: Optional[torch.Tensor]           # FP32 [tokens, 2]
    counts: Optional[torch.Tensor]        # int32 [experts]
    mean_prob: Optional[torch.Tensor]     # FP32 [experts]
    summary: Optional[torch.Tensor]       # FP32 [4]: the next three and the counted tokens
    loss: Optional[torch.Tensor]          # [1]
    balance: Optional[torch.Tensor]       # [1]
    z: Optional[torch.Tensor]             # [1]
    scratch: Optional[torch.Tensor]


def fa_route_scratch(tokens: int, experts: int) -> int:
    """Bytes of scratch fa_route needs."""
    out = ctypes.c_int64()
    check("fa_route_scratch",
          _lib.load().fa_route_scratch(tokens, experts, ctypes.byref(out)))
    return out.value


def route_buffers(tokens: int, experts: int, k: int, device, loss: bool = True) -> RouteBuffers:
    """``loss`` False: for a pass that takes no loss and keeps nothing for a gradient."""
    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=device)

    chosen, weights = new(tokens, k, dtype=torch.int32), new(tokens, k)
    if not loss:
        return RouteBuffers(chosen, weights, *[None] * 8)
    summary = new(4)
    scratch = new(max(16, fa_route_scratch(tokens, experts)), dtype=torch.uint8)
    return RouteBuffers(chosen, weights, new(tokens, 2), new(experts, dtype=torch.int32),
                        new(experts), summary, *summary.split(1)[:3], scratch)


def _router(logits: torch.Tensor, k: int, counted: Optional[torch.Tensor], renormalise: bool,
            weight_scale: float, balance_coef: float, z_coef: float) -> FaRouter:
    tokens, experts = shape = logits.shape
    ptr, ld = _mat("logits", logits, shape, logits.dtype)
    mask = None
    if counted is not None:  # a bool is a byte
        mask = _vec_or_none("counted", counted, tokens,
                            torch.bool if counted.dtype is torch.bool else _U8)
    return FaRouter(tokens, experts, ptr, _code("logits", logits, _FLOATS), ld, mask, k,
                    bool(renormalise), weight_scale, balance_coef, z_coef)


def _routing(out: RouteBuffers, tokens: int, experts: int) -> tuple[FaRouting, int]:
    chosen, weights, lse, counts, mean_prob, summary, _, _, _, scratch = out
    k = _matrix("chosen", chosen)[1]
    pairs = (_vec_or_none("chosen", chosen, tokens * k, _I32),
             _vec_or_none("weights", weights, tokens * k, _F32))
    if lse is None:
        return FaRouting(*pairs), k
    kept = (_vec_or_none("lse", lse, 2 * tokens, _F32),
            _vec_or_none("counts", counts, experts, _I32))
    if summary is None:  # what a gradient reads
        return FaRouting(*pairs, *kept), k
    size = scratch.numel()
    return FaRouting(*pairs, *kept, _vec_or_none("mean_prob", mean_prob, experts, _F32),
                     _vec_or_none("summary", summary, 4, _F32),
                     _vec_or_none("scratch", scratch, size, _U8), size), k


def fa_route(logits: torch.Tensor, out: RouteBuffers, counted: Optional[torch.Tensor] = None,
             renormalise: bool = True, weight_scale: float = 1.0, balance_coef: float = 0.0,
             z_coef: float = 0.0, stream=None) -> None:
    """The experts of each token (as many as ``out`` has columns for) and their weights; with
    buffers for a loss the counts and the balance and z losses.  counted (bool or uint8
    [tokens]): 0 for padding."""
    tokens, experts = _matrix("logits", logits)
    r, k = _routing(out, tokens, experts)
    x = _router(logits, k, counted, renormalise, weight_scale, balance_coef, z_coef)
    check("fa_route", _lib.load().fa_route(ctypes.byref(x), ctypes.byref(r), _stream(stream)))


def fa_route_gradient(logits: torch.Tensor, out: RouteBuffers, dlogits: torch.Tensor,
                      dweights: Optional[torch.Tensor] = None,
                      grad_loss: Optional[torch.Tensor] = None,
                      counted: Optional[torch.Tensor] = None, renormalise: bool = True,
                      weight_scale: float = 1.0, balance_coef: float = 0.0, z_coef: float = 0.0,
                      stream=None) -> None:
    """dlogits of grad_loss (a device scalar) * loss + sum of dweights * weights, from what
    fa_route wrote with the same arguments."""
    tokens, experts = _matrix("logits", logits)
    if out.lse is None:
        raise ValueError("the buffers are those of a pass without a loss: nothing was kept")
    r, k = _routing(out, tokens, experts)
    x = _router(logits, k, counted, renormalise, weight_scale, balance_coef, z_coef)
    to, to_ld = _mat("dlogits", dlogits, logits.shape, logits.dtype)
    check("fa_route_gradient", _lib.load().fa_route_gradient(
        ctypes.byref(x), ctypes.byref(r), _vec_or_none("dweights", dweights, tokens * k, _F32),
        _vec_or_none("grad_loss", grad_loss, 1, _F32), to, to_ld, _stream(stream)))
