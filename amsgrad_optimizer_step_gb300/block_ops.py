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
from .model_ops import _FLOATS, _code, _matrix, _rows, _same, _stream, _vector

__all__ = [
    "fa_dropout", "fa_block_join", "fa_block_join_scratch", "fa_block_join_gradient", "fa_route",
    "fa_route_scratch", "fa_route_gradient", "Dropout", "Join", "join_scratch", "RouteBuffers",
    "route_buffers",
]

_U64 = (1 << 64) - 1


# ---- dropout -----------------------------------------------------------------------

class Dropout(NamedTuple):
    """Which elements a dropout keeps: the same record drops the same places of a matrix of as
    many columns, in every call and on every layout (see fa_dropout_key)."""
    p: float
    seed: int = 0
    offset: int = 0  # the call's own
    counter: Optional[torch.Tensor] = None  # int64 [1] on the device, added to offset


def _key(drop: Dropout) -> FaDropoutKey:
    counter = drop.counter
    return FaDropoutKey(drop.p, drop.seed & _U64, drop.offset & _U64,
                        None if counter is None else _vector("counter", counter, 1, torch.int64))


def fa_dropout(x: torch.Tensor, out: torch.Tensor, drop: Dropout, stream=None) -> None:
    """out = x with elements dropped and the others multiplied by 1 / (1 - p); its gradient is
    the same call on the output's.  out may be x itself."""
    rows, cols = shape = _matrix("x", x)
    key = _key(drop)
    check("fa_dropout", _lib.load().fa_dropout(
        rows, cols, x.data_ptr(), _rows("x", x, shape), _code("x", x, _FLOATS),
        ctypes.byref(key), _same(x.dtype, "out", out), _rows("out", out, shape), _stream(stream)))


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


def _weight(name: str, t: Optional[torch.Tensor], shape, dtype) -> tuple[Optional[int], int]:
    """Pointer and row distance of a weight ([cols]) or gate ([groups, cols])."""
    if t is None:
        return None, shape[-1]
    ptr = _same(dtype, name, t)
    if len(shape) == 1:
        return _vector(name, t, shape[0], dtype), shape[0]
    return ptr, _rows(name, t, shape)


def _join_record(j: Join, like: torch.Tensor, stream_dtype, branch, post_weight, pre_weight, gate):
    """The C record, the weights' type and the key that it points to."""
    rows, cols = shape = like.shape
    dtype = branch.dtype if branch is not None else like.dtype
    weights = [w for w in (post_weight, pre_weight, gate) if w is not None]
    wdtype = weights[0].dtype if weights else dtype
    groups = 1
    if gate is not None:
        groups = _matrix("gate", gate)[0]
    key = None if j.dropout is None else _key(j.dropout)
    gate_ptr, gate_ld = _weight("gate", gate, (groups, cols), wdtype)
    record = FaJoin(
        rows, cols, _FLOATS.get(dtype, -1), _FLOATS.get(stream_dtype, -1),
        _FLOATS.get(wdtype, -1), int(bool(j.post_norm)),
        None if branch is None else branch.data_ptr(),
        cols if branch is None else _rows("branch", branch, shape),
        _weight("post_weight", post_weight, (cols,), wdtype)[0],
        _weight("pre_weight", pre_weight, (cols,), wdtype)[0], gate_ptr, gate_ld, groups,
        j.residual_scale, j.branch_scale, j.eps, j.weight_offset,
        None if key is None else ctypes.addressof(key))
    return record, dtype, wdtype, key


def _optional(name: str, t: Optional[torch.Tensor], shape, dtype) -> tuple[Optional[int], int]:
    return (None, shape[1]) if t is None else (_same(dtype, name, t), _rows(name, t, shape))


def _per_row(name: str, t: Optional[torch.Tensor], rows: int) -> Optional[int]:
    return None if t is None else _vector(name, t, rows, torch.float32)


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
    rows, cols = shape = _matrix("residual", residual)
    j = join or _JOIN
    like = branch if branch is not None else normed if normed is not None else residual
    if like.shape != shape:
        raise ValueError(f"shape {tuple(like.shape)}, expected {tuple(shape)}")
    record, dtype, _, key = _join_record(
        j, residual if branch is None and normed is None else like, residual.dtype, branch,
        post_weight, pre_weight, gate)
    out_ptr, out_ld = _optional("out", out, shape, residual.dtype)
    normed_ptr, normed_ld = _optional("normed", normed, shape, dtype)
    check("fa_block_join", _lib.load().fa_block_join(
        ctypes.byref(record), residual.data_ptr(), _rows("residual", residual, shape), out_ptr,
        out_ld, normed_ptr, normed_ld, _per_row("post_rstd", post_rstd, rows),
        _per_row("pre_rstd", pre_rstd, rows), _stream(stream)))


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
    j = join or _JOIN
    like = next((t for t in (branch, dnormed, dout, out) if t is not None), None)
    if like is None:
        raise ValueError("neither a branch nor a gradient is given")
    rows, cols = shape = _matrix("branch", like)
    streams = [t for t in (dout, out, dresidual) if t is not None]
    stream_dtype = streams[0].dtype if streams else like.dtype
    typed = branch if branch is not None else dnormed if dnormed is not None else like
    record, dtype, wdtype, key = _join_record(j, typed, stream_dtype, branch, post_weight,
                                              pre_weight, gate)
    g = FaJoinGradient(
        *_optional("out", out, shape, stream_dtype), _per_row("post_rstd", post_rstd, rows),
        _per_row("pre_rstd", pre_rstd, rows), *_optional("dout", dout, shape, stream_dtype),
        *_optional("dnormed", dnormed, shape, dtype),
        *_optional("dresidual", dresidual, shape, stream_dtype),
        *_optional("dbranch", dbranch, shape, dtype),
        _weight("dpost_weight", dpost_weight, (cols,), wdtype)[0],
        _weight("dpre_weight", dpre_weight, (cols,), wdtype)[0],
        *_weight("dgate", dgate, (record.groups, cols), wdtype),
        None if scratch is None else _vector("scratch", scratch, scratch.numel(), torch.uint8),
        0 if scratch is None else scratch.numel())
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
    tokens, experts = _matrix("logits", logits)
    if counted is not None and counted.dtype is torch.bool:
        counted = counted.view(torch.uint8)
    return FaRouter(tokens, experts, logits.data_ptr(), _code("logits", logits, _FLOATS),
                    _rows("logits", logits, logits.shape),
                    None if counted is None else _vector("counted", counted, tokens, torch.uint8),
                    k, int(bool(renormalise)), weight_scale, balance_coef, z_coef)


def _routing(out: RouteBuffers, tokens: int, experts: int) -> tuple[FaRouting, int]:
    k = _matrix("chosen", out.chosen)[1]
    f32, i32 = torch.float32, torch.int32
    pairs = _vector("chosen", out.chosen, tokens * k, i32), _vector("weights", out.weights,
                                                                    tokens * k, f32)
    if out.lse is None:
        return FaRouting(*pairs), k
    kept = _vector("lse", out.lse, 2 * tokens, f32), _vector("counts", out.counts, experts, i32)
    if out.summary is None:  # what a gradient reads
        return FaRouting(*pairs, *kept), k
    return FaRouting(*pairs, *kept, _vector("mean_prob", out.mean_prob, experts, f32),
                     _vector("summary", out.summary, 4, f32),
                     _vector("scratch", out.scratch, out.scratch.numel(), torch.uint8),
                     out.scratch.numel()), k


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
    f32 = torch.float32
    check("fa_route_gradient", _lib.load().fa_route_gradient(
        ctypes.byref(x), ctypes.byref(r),
        None if dweights is None else _vector("dweights", dweights, tokens * k, f32),
        None if grad_loss is None else _vector("grad_loss", grad_loss, 1, f32),
        _same(logits.dtype, "dlogits", dlogits), _rows("dlogits", dlogits, logits.shape),
        _stream(stream)))
