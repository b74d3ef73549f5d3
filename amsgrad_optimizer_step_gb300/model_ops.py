"""Binding of the model-side operators (``include/fa_model_ops.h``).

The embedding lookup and its gradient, the token log-probabilities with the preference
and the clipped policy loss, and the gated activation with its 8-bit checkpoint: each
function marshals torch tensors into the C call of the same name, as the package's other
bindings do.  Outputs and scratch are the caller's; the ``*_buffers`` helpers make them.
``layers`` has the same operators with autograd.  The RUDA documentation pages cover the
optimizer only and have no counterpart to these.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import FaLogits, FaPolicy, FaPreference, check

_FLOATS = {torch.float32: _lib.FA_F32, torch.float16: _lib.FA_F16, torch.bfloat16: _lib.FA_BF16}
_INTS = {torch.int32: 0, torch.int64: 1}
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
CHECKPOINT_BLOCK = 128

__all__ = [
    "fa_embedding_lookup", "fa_embedding_scratch", "fa_embedding_gradient", "fa_token_logprobs",
    "fa_token_logprobs_gradient", "fa_preference_loss", "fa_policy_loss", "fa_checkpoint_size",
    "fa_gated_forward", "fa_gated_backward", "embedding_scratch", "preference_buffers",
    "policy_buffers", "checkpoint_buffer", "PreferenceBuffers", "PolicyBuffers", "Checkpoint",
]


# The raw handle of the current stream, without the Stream object torch.cuda.current_stream
# builds (2.9 us of a 12.6 us call on the GB300's host; 0.1 us this way).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# The library refuses memory that is not the current device's (FA_ERR_POINTER); what raw
# pointers cannot show - shapes, strides, types - is checked here, with the message built
# only on a refusal.

def _code(name: str, t: torch.Tensor, codes: dict) -> int:
    code = codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(codes)}")
    return code


def _rows(name: str, t: torch.Tensor, shape) -> int:
    """Checks a matrix with unit stride along its rows; returns the rows' distance."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    row, col = t.stride()
    if col == 1 and row >= shape[1]:
        return row
    if col != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if shape[0] > 1 and row < shape[1]:
        raise ValueError(f"{name}: overlapping or broadcast rows")
    return max(row, shape[1])


def _vector(name: str, t: torch.Tensor, n: int, dtype) -> int:
    """Checks a dense tensor of n elements; returns its pointer."""
    if t.dtype is dtype and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name}: must be dense with {n} elements")


def _ids(name: str, t: torch.Tensor, n: int) -> tuple[int, int]:
    return _vector(name, t, n, t.dtype), _code(name, t, _INTS)


def _matrix(name: str, t: torch.Tensor):
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected a matrix")
    return t.shape


# ---- embedding -------------------------------------------------------------------

def fa_embedding_lookup(ids: torch.Tensor, table: torch.Tensor, out: torch.Tensor,
                        scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; zeros for an id outside the table."""
    n = ids.numel()
    vocab, dim = _matrix("table", table)
    ptr, idt = _ids("ids", ids, n)
    check("fa_embedding_lookup", _lib.load().fa_embedding_lookup(
        n, ptr, idt, table.data_ptr(), _code("table", table, _FLOATS), vocab, dim,
        _rows("table", table, table.shape), scale, out.data_ptr(),
        _code("out", out, _FLOATS), _rows("out", out, (n, dim)), _stream(stream)))


def fa_embedding_scratch(tokens: int, vocab: int, dim: int) -> int:
    """Bytes of scratch fa_embedding_gradient needs."""
    out = ctypes.c_int64()
    check("fa_embedding_scratch",
          _lib.load().fa_embedding_scratch(tokens, vocab, dim, ctypes.byref(out)))
    return out.value


def embedding_scratch(tokens: int, vocab: int, dim: int, device) -> torch.Tensor:
    """Scratch for fa_embedding_gradient of at most these sizes."""
    return torch.empty(max(16, fa_embedding_scratch(tokens, vocab, dim)), dtype=torch.uint8,
                       device=device)


def fa_embedding_gradient(ids: torch.Tensor, dout: torch.Tensor, dtable: torch.Tensor,
                          scratch: torch.Tensor, scale: float = 1.0, padding_idx: int = -1,
                          accumulate: bool = False, stream=None) -> None:
    """dtable[v] (+)= scale * sum of dout[t] over the tokens t with id v."""
    n = ids.numel()
    vocab, dim = _matrix("dtable", dtable)
    ptr, idt = _ids("ids", ids, n)
    size = scratch.numel()
    check("fa_embedding_gradient", _lib.load().fa_embedding_gradient(
        n, ptr, idt, dout.data_ptr(), _code("dout", dout, _FLOATS),
        _rows("dout", dout, (n, dim)), scale, padding_idx, int(bool(accumulate)),
        dtable.data_ptr(), _code("dtable", dtable, _FLOATS), vocab, dim,
        _rows("dtable", dtable, dtable.shape),
        _vector("scratch", scratch, size, torch.uint8), size, _stream(stream)))


# ---- losses from the logits ----------------------------------------------------------

def _logits(logits: torch.Tensor, labels: torch.Tensor, logit_scale: float) -> FaLogits:
    tokens, vocab = _matrix("logits", logits)
    ptr, ltype = _ids("labels", labels, tokens)
    return FaLogits(tokens, vocab, logits.data_ptr(), _code("logits", logits, _FLOATS),
                    _rows("logits", logits, logits.shape), ptr, ltype, logit_scale)


def fa_token_logprobs(logits: torch.Tensor, labels: torch.Tensor, logp: torch.Tensor,
                      lse: Optional[torch.Tensor] = None, logit_scale: float = 1.0,
                      stream=None) -> None:
    """logp[t] = log softmax(logit_scale * logits[t])[labels[t]] (0 where the label is not an
    id); lse [tokens, 2] keeps the row statistics for the gradient."""
    n = logits.shape[0]
    x = _logits(logits, labels, logit_scale)
    check("fa_token_logprobs", _lib.load().fa_token_logprobs(
        ctypes.byref(x), _vector("logp", logp, n, torch.float32),
        None if lse is None else _vector("lse", lse, 2 * n, torch.float32),
        _stream(stream)))


def _dlogits(logits: torch.Tensor, dlogits: torch.Tensor) -> int:
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits: dtype {dlogits.dtype}, expected {logits.dtype}")
    return _rows("dlogits", dlogits, logits.shape)


def fa_token_logprobs_gradient(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                               dlogp: torch.Tensor, dlogits: torch.Tensor,
                               logit_scale: float = 1.0, grad_scale: float = 1.0,
                               grad_loss: Optional[torch.Tensor] = None, stream=None) -> None:
    """dlogits from dlogp (dloss/dlogp of each token), times grad_scale and the device scalar
    grad_loss.  dlogits may be the logits themselves."""
    n = logits.shape[0]
    x = _logits(logits, labels, logit_scale)
    check("fa_token_logprobs_gradient", _lib.load().fa_token_logprobs_gradient(
        ctypes.byref(x), _vector("lse", lse, 2 * n, torch.float32),
        _vector("dlogp", dlogp, n, torch.float32), grad_scale,
        None if grad_loss is None else _vector("grad_loss", grad_loss, 1, torch.float32),
        dlogits.data_ptr(), _dlogits(logits, dlogits), _stream(stream)))


class PreferenceBuffers(NamedTuple):
    """Outputs of fa_preference_loss (FP32)."""
    loss: torch.Tensor       # [1] mean over the pairs
    pair_loss: torch.Tensor  # [pairs]
    rewards: torch.Tensor    # [pairs, 2] beta * log ratio: the preferred, the other
    logp: torch.Tensor       # [tokens]
    lse: torch.Tensor        # [tokens, 2]
    dlogp: torch.Tensor      # [tokens] dloss/dlogp


def preference_buffers(tokens: int, pairs: int, device) -> PreferenceBuffers:
    def new(*shape):
        return torch.empty(shape, dtype=torch.float32, device=device)
    return PreferenceBuffers(new(1), new(pairs), new(pairs, 2), new(tokens), new(tokens, 2),
                             new(tokens))


def fa_preference_loss(logits: torch.Tensor, labels: torch.Tensor, seq_offsets: torch.Tensor,
                       ref_logp: torch.Tensor, out: PreferenceBuffers, beta: float = 0.1,
                       label_smoothing: float = 0.0, average: bool = False,
                       logit_scale: float = 1.0, stream=None) -> None:
    """Preference loss of packed pairs: seq_offsets (int64, on the device) cuts the tokens
    into 2 * pairs sequences, of which 2k was preferred to 2k + 1."""
    n = logits.shape[0]
    pairs = out.pair_loss.numel()
    f32 = torch.float32
    x = _logits(logits, labels, logit_scale)
    a = FaPreference(
        pairs, _vector("seq_offsets", seq_offsets, 2 * pairs + 1, torch.int64),
        _vector("ref_logp", ref_logp, n, f32), beta, label_smoothing, int(bool(average)),
        _vector("loss", out.loss, 1, f32), _vector("pair_loss", out.pair_loss, pairs, f32),
        _vector("rewards", out.rewards, 2 * pairs, f32),
        _vector("logp", out.logp, n, f32), _vector("lse", out.lse, 2 * n, f32),
        _vector("dlogp", out.dlogp, n, f32))
    check("fa_preference_loss",
          _lib.load().fa_preference_loss(ctypes.byref(x), ctypes.byref(a), _stream(stream)))


class PolicyBuffers(NamedTuple):
    """Outputs of fa_policy_loss (FP32)."""
    summary: torch.Tensor        # [4]: the next four in one
    loss: torch.Tensor           # [1]
    kl: torch.Tensor             # [1] mean KL term of the counted tokens
    clip_fraction: torch.Tensor  # [1] share of them that were clipped
    count: torch.Tensor          # [1] their number
    logp: torch.Tensor           # [tokens]
    token_loss: torch.Tensor     # [tokens]
    token_kl: torch.Tensor       # [tokens]


def policy_buffers(tokens: int, device) -> PolicyBuffers:
    summary = torch.empty(4, dtype=torch.float32, device=device)
    per_token = [torch.empty(tokens, dtype=torch.float32, device=device) for _ in range(3)]
    return PolicyBuffers(summary, *summary.split(1), *per_token)


def fa_policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor,
                   advantages: torch.Tensor, out: PolicyBuffers,
                   ref_logp: Optional[torch.Tensor] = None,
                   weights: Optional[torch.Tensor] = None,
                   dlogits: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                   clip_high: float = 0.2, kl_coef: float = 0.0, denominator: float = 0.0,
                   logit_scale: float = 1.0, grad_scale: float = 1.0,
                   lse: Optional[torch.Tensor] = None, dlogp: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Clipped policy loss with a KL term; with dlogits (which may be the logits) the
    gradient too, in the same pass.  denominator 0 divides by the counted tokens.  lse and
    dlogp keep what fa_token_logprobs_gradient takes, for a gradient later."""
    n = logits.shape[0]
    f32 = torch.float32
    x = _logits(logits, labels, logit_scale)
    a = FaPolicy(
        _vector("old_logp", old_logp, n, f32), _vector("advantages", advantages, n, f32),
        None if ref_logp is None else _vector("ref_logp", ref_logp, n, f32),
        None if weights is None else _vector("weights", weights, n, f32),
        clip_low, clip_high, kl_coef, denominator, grad_scale,
        _vector("summary", out.summary, 4, f32), _vector("logp", out.logp, n, f32),
        _vector("token_loss", out.token_loss, n, f32),
        _vector("token_kl", out.token_kl, n, f32),
        None if lse is None else _vector("lse", lse, 2 * n, f32),
        None if dlogp is None else _vector("dlogp", dlogp, n, f32),
        None if dlogits is None else dlogits.data_ptr(),
        0 if dlogits is None else _dlogits(logits, dlogits))
    check("fa_policy_loss",
          _lib.load().fa_policy_loss(ctypes.byref(x), ctypes.byref(a), _stream(stream)))


# ---- gated activation -----------------------------------------------------------------

class Checkpoint(NamedTuple):
    """An 8-bit checkpoint of a gated activation's two inputs."""
    codes: torch.Tensor   # int8 [2, rows, pitch]: gate, up; pitch is cols rounded up to 128
    scales: torch.Tensor  # float32 [2, rows, pitch / 128]
    cols: int

    def values(self) -> tuple[torch.Tensor, torch.Tensor]:
        """What the codes stand for, in FP32 (for inspection; the kernels decode their own)."""
        x = self.codes.unflatten(2, (-1, CHECKPOINT_BLOCK)).float() * self.scales[..., None]
        gate, up = x.flatten(2)[:, :, :self.cols]
        return gate, up


def fa_checkpoint_size(rows: int, cols: int) -> tuple[int, int]:
    """(bytes of codes, FP32 elements of scales) of a [rows, cols] checkpoint."""
    codes, scales = ctypes.c_int64(), ctypes.c_int64()
    check("fa_checkpoint_size", _lib.load().fa_checkpoint_size(
        rows, cols, ctypes.byref(codes), ctypes.byref(scales)))
    return codes.value, scales.value


def checkpoint_buffer(rows: int, cols: int, device) -> Checkpoint:
    fa_checkpoint_size(rows, cols)  # refuses sizes out of range
    blocks = -(-cols // CHECKPOINT_BLOCK)
    return Checkpoint(
        torch.empty((2, rows, blocks * CHECKPOINT_BLOCK), dtype=torch.int8, device=device),
        torch.empty((2, rows, blocks), dtype=torch.float32, device=device), cols)


def _checkpoint(ck: Checkpoint, rows: int, cols: int) -> tuple[int, int]:
    blocks = -(-cols // CHECKPOINT_BLOCK)
    if ck.cols != cols:
        raise ValueError(f"checkpoint: of {ck.cols} columns, expected {cols}")
    return (_vector("codes", ck.codes, 2 * rows * blocks * CHECKPOINT_BLOCK, torch.int8),
            _vector("scales", ck.scales, 2 * rows * blocks, torch.float32))


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation {name!r} not in {tuple(ACTIVATIONS)}")
    return code


def _same(dtype, name: str, t: torch.Tensor) -> int:
    """The pointer of a tensor that must have the type of another."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    return t.data_ptr()


def fa_gated_forward(gate: torch.Tensor, up: torch.Tensor, h: torch.Tensor,
                     checkpoint: Optional[Checkpoint] = None, activation: str = "silu",
                     stream=None) -> None:
    """h = act(gate) * up, keeping gate and up in 8 bits in ``checkpoint`` (None: not kept)."""
    rows, cols = shape = _matrix("gate", gate)
    codes, scales = (None, None) if checkpoint is None else _checkpoint(checkpoint, rows, cols)
    check("fa_gated_forward", _lib.load().fa_gated_forward(
        rows, cols, gate.data_ptr(), _rows("gate", gate, shape), _same(gate.dtype, "up", up),
        _rows("up", up, shape), _code("gate", gate, _FLOATS), _activation(activation),
        _same(gate.dtype, "h", h), _rows("h", h, shape), codes, scales, _stream(stream)))


def fa_gated_backward(checkpoint: Checkpoint, dh: torch.Tensor, dgate: torch.Tensor,
                      dup: torch.Tensor, h: Optional[torch.Tensor] = None,
                      activation: str = "silu", stream=None) -> None:
    """Gradients of the gate and up from the checkpoint, and (with ``h``) act(gate) * up again."""
    rows, cols = shape = _matrix("dh", dh)
    codes, scales = _checkpoint(checkpoint, rows, cols)
    check("fa_gated_backward", _lib.load().fa_gated_backward(
        rows, cols, codes, scales, _activation(activation), dh.data_ptr(),
        _rows("dh", dh, shape), _code("dh", dh, _FLOATS), _same(dh.dtype, "dgate", dgate),
        _rows("dgate", dgate, shape), _same(dh.dtype, "dup", dup), _rows("dup", dup, shape),
        None if h is None else _same(dh.dtype, "h", h), 0 if h is None else _rows("h", h, shape),
        _stream(stream)))
