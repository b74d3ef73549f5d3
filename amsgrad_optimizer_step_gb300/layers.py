"""The model-side operators with autograd: what a training step calls around ``optim``.

``embedding`` is the scaled lookup whose gradient is taken by sorted tokens; ``gated_down``
the tail of a gated MLP that keeps its two inputs in 8 bits until the backward pass, and
nothing else; ``token_logprobs``, ``preference_loss`` and ``policy_loss`` go from the logits
to a loss, and ``policy_step`` takes the policy loss and the logits' gradient in one pass.
Gradients come in the operands' types, so that they go into an optimizer bucket as they are;
a non-finite one is found by the optimizer's statistics and skips its step.  All arithmetic
but the plain matrix products runs in the library's kernels.
"""

from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import model_ops as ops

__all__ = ["embedding", "gated_activation", "gated_down", "token_logprobs", "preference_loss",
           "policy_loss", "policy_step"]


def _flat(x: torch.Tensor) -> torch.Tensor:
    """A matrix of the last dimension's rows: a view where rows are adjacent elements and do not
    overlap, else a copy (the gradient of a sum over rows is one row expanded)."""
    rows, cols = x.shape[:-1].numel(), x.shape[-1]
    y = x.reshape(rows, cols)
    dense = (cols <= 1 or y.stride(1) == 1) and (rows <= 1 or y.stride(0) >= cols)
    return y if dense else y.contiguous()


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx):
        flat = ids.reshape(-1).contiguous()
        out = torch.empty((flat.numel(), weight.shape[1]), dtype=weight.dtype, device=weight.device)
        ops.fa_embedding_lookup(flat, weight, out, scale)
        ctx.save_for_backward(flat)
        ctx.table = weight.shape, weight.dtype
        ctx.scale, ctx.padding_idx = scale, padding_idx
        return out.view(*ids.shape, weight.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        (vocab, dim), dtype = ctx.table
        dtable = torch.empty((vocab, dim), dtype=dtype, device=dout.device)
        scratch = ops.embedding_scratch(ids.numel(), vocab, dim, dout.device)
        ops.fa_embedding_gradient(ids, _flat(dout), dtable, scratch, ctx.scale, ctx.padding_idx)
        return None, dtable, None, None


def embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              padding_idx: Optional[int] = None) -> torch.Tensor:
    """scale * weight[ids]; ids outside the table give zeros, and they and ``padding_idx`` no
    gradient.  ``padding_idx`` is an id as it stands in ``ids``: a negative one is outside the
    table like every negative id (it does not count from the table's end)."""
    return _Embedding.apply(ids, weight, scale, -1 if padding_idx is None else padding_idx)


# needs_input_grad of the two functions below says only which inputs require a gradient; whether
# any will be taken (no_grad, inference_mode) is asked outside: a forward method runs with
# gradients off in every mode.

def _halves(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    cols = x.shape[1] // 2
    if x.shape[1] != 2 * cols:
        raise ValueError(f"gate_up: {x.shape[1]} columns are not two halves")
    return x[:, :cols], x[:, cols:]


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate_up, activation, grad_enabled):
        gate, up = _halves(_flat(gate_up))
        h = torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
        keep = grad_enabled and ctx.needs_input_grad[0]
        checkpoint = ops.checkpoint_buffer(*gate.shape, gate.device) if keep else None
        ops.fa_gated_forward(gate, up, h, checkpoint, activation)
        if keep:  # given back with the graph's other tensors once the backward pass has run
            ctx.save_for_backward(checkpoint.codes, checkpoint.scales)
        ctx.activation, ctx.shape = activation, gate_up.shape
        return h.view(*gate_up.shape[:-1], gate.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        dh = _flat(dh)
        checkpoint = ops.Checkpoint(*ctx.saved_tensors, dh.shape[1])
        grad = torch.empty((dh.shape[0], 2 * dh.shape[1]), dtype=dh.dtype, device=dh.device)
        ops.fa_gated_backward(checkpoint, dh, *_halves(grad), None, ctx.activation)
        return grad.view(ctx.shape), None, None


def gated_activation(gate_up: torch.Tensor, activation: str = "silu") -> torch.Tensor:
    """act(gate) * up of a projection whose last dimension holds gate and up side by side, which
    are kept in 8 bits for the backward pass (nothing is kept where there will be none)."""
    return _Gated.apply(gate_up, activation, torch.is_grad_enabled())


class _GatedDown(torch.autograd.Function):
    # its matrix products, in both passes, in the type that autocast has for the forward pass
    @staticmethod
    @torch.amp.custom_fwd(device_type="cuda")
    def forward(ctx, gate_up, weight, activation, grad_enabled):
        gate, up = _halves(_flat(gate_up))
        h = torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
        keep = grad_enabled and any(ctx.needs_input_grad[:2])
        checkpoint = ops.checkpoint_buffer(*gate.shape, gate.device) if keep else None
        ops.fa_gated_forward(gate, up, h, checkpoint, activation)
        if keep:
            ctx.save_for_backward(weight, checkpoint.codes, checkpoint.scales)
        ctx.activation, ctx.shape = activation, gate_up.shape
        return (h @ weight.t()).view(*gate_up.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    @torch.amp.custom_bwd(device_type="cuda")
    def backward(ctx, dy):
        weight, *kept = ctx.saved_tensors
        dy = _flat(dy)
        dh = dy @ weight
        checkpoint = ops.Checkpoint(*kept, dh.shape[1])
        grad = torch.empty((dh.shape[0], 2 * dh.shape[1]), dtype=dh.dtype, device=dh.device)
        h = torch.empty_like(dh) if ctx.needs_input_grad[1] else None
        ops.fa_gated_backward(checkpoint, dh, *_halves(grad), h, ctx.activation)
        return grad.view(ctx.shape), None if h is None else dy.t() @ h, None, None


def gated_down(gate_up: torch.Tensor, weight: torch.Tensor,
               activation: str = "silu") -> torch.Tensor:
    """(act(gate) * up) @ weight.T.  Between the passes it holds an 8-bit checkpoint of gate and
    up alone: the activation itself, which the weight's gradient needs, is made again from it
    in the same pass as their gradients.  Under autocast the product is one of autocast's."""
    return _GatedDown.apply(gate_up, weight, activation, torch.is_grad_enabled())


def _gradient(ctx, logits, labels, lse, dlogp, grad_loss):
    dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    ops.fa_token_logprobs_gradient(logits, labels, lse, dlogp, dlogits, ctx.logit_scale,
                                   grad_loss=grad_loss)
    return dlogits


def _labels(labels: torch.Tensor) -> torch.Tensor:
    return labels.reshape(-1).contiguous()


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, logit_scale):
        flat, y = _flat(logits), _labels(labels)
        n = flat.shape[0]
        logp = torch.empty(n, dtype=torch.float32, device=flat.device)
        lse = torch.empty((n, 2), dtype=torch.float32, device=flat.device)
        ops.fa_token_logprobs(flat, y, logp, lse, logit_scale)
        ctx.save_for_backward(flat, y, lse)
        ctx.logit_scale, ctx.shape = logit_scale, logits.shape
        return logp.view(labels.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp):
        logits, labels, lse = ctx.saved_tensors
        return _gradient(ctx, logits, labels, lse, dlogp.reshape(-1).float().contiguous(),
                         None).view(ctx.shape), None, None


def token_logprobs(logits: torch.Tensor, labels: torch.Tensor,
                   logit_scale: float = 1.0) -> torch.Tensor:
    """log softmax(logit_scale * logits) at the labels, FP32; 0 where a label is no id."""
    return _TokenLogprobs.apply(logits, labels, logit_scale)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, seq_offsets, ref_logp, beta, smoothing, average, logit_scale):
        flat, y = _flat(logits), _labels(labels)
        pairs = (seq_offsets.numel() - 1) // 2
        out = ops.preference_buffers(flat.shape[0], pairs, flat.device)
        ops.fa_preference_loss(flat, y, seq_offsets, ref_logp.reshape(-1).contiguous(), out, beta,
                               smoothing, average, logit_scale)
        ctx.save_for_backward(flat, y, out.lse, out.dlogp)
        ctx.logit_scale, ctx.shape = logit_scale, logits.shape
        ctx.mark_non_differentiable(out.rewards)
        return out.loss.view(()), out.rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        grad = _gradient(ctx, *ctx.saved_tensors, dloss.reshape(1).float())
        return (grad.view(ctx.shape),) + (None,) * 7


def preference_loss(logits: torch.Tensor, labels: torch.Tensor, seq_offsets: torch.Tensor,
                    ref_logp: torch.Tensor, beta: float = 0.1, label_smoothing: float = 0.0,
                    average: bool = False,
                    logit_scale: float = 1.0) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, rewards [pairs, 2]) of packed pairs of sequences (see fa_preference_loss)."""
    if seq_offsets.numel() % 2 == 0:
        raise ValueError("seq_offsets: 2 * pairs + 1 offsets are needed")
    return _PreferenceLoss.apply(logits, labels, seq_offsets, ref_logp, beta, label_smoothing,
                                 average, logit_scale)


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, old_logp, advantages, ref_logp, weights, clip_low, clip_high,
                kl_coef, denominator, logit_scale):
        flat, y = _flat(logits), _labels(labels)
        n = flat.shape[0]
        out = ops.policy_buffers(n, flat.device)
        lse = torch.empty((n, 2), dtype=torch.float32, device=flat.device)
        dlogp = torch.empty(n, dtype=torch.float32, device=flat.device)
        ops.fa_policy_loss(flat, y, old_logp, advantages, out, ref_logp, weights, None, clip_low,
                           clip_high, kl_coef, denominator, logit_scale, lse=lse, dlogp=dlogp)
        ctx.save_for_backward(flat, y, lse, dlogp)
        ctx.logit_scale, ctx.shape = logit_scale, logits.shape
        loss, stats = out.summary[0].clone(), out.summary
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        grad = _gradient(ctx, *ctx.saved_tensors, dloss.reshape(1).float())
        return (grad.view(ctx.shape),) + (None,) * 10


def _tokens(x: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if x is None else x.reshape(-1).contiguous()


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, ref_logp: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, denominator: float = 0.0,
                logit_scale: float = 1.0) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, [loss, mean KL, clipped share, counted tokens]) of the clipped policy loss (see
    fa_policy_loss).  The gradient is taken in the backward pass, from the logits again."""
    return _PolicyLoss.apply(logits, labels, _tokens(old_logp), _tokens(advantages),
                             _tokens(ref_logp), _tokens(weights), clip_low, clip_high, kl_coef,
                             denominator, logit_scale)


def policy_step(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, ref_logp: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, denominator: float = 0.0,
                logit_scale: float = 1.0,
                loss_scale: float = 1.0) -> tuple[torch.Tensor, torch.Tensor]:
    """policy_loss and its gradient in one pass over the logits: ([loss, mean KL, clipped share,
    counted tokens], dlogits), the latter times ``loss_scale``.  The model's backward pass
    starts with ``logits.backward(dlogits)``."""
    flat = _flat(logits.detach())
    out = ops.policy_buffers(flat.shape[0], flat.device)
    dlogits = torch.empty(flat.shape, dtype=flat.dtype, device=flat.device)
    ops.fa_policy_loss(flat, _labels(labels), _tokens(old_logp), _tokens(advantages), out,
                       _tokens(ref_logp), _tokens(weights), dlogits, clip_low, clip_high, kl_coef,
                       denominator, logit_scale, loss_scale)
    return out.summary, dlogits.view(logits.shape)
