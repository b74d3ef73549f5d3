"""Preference training, then policy training, of a small language model on one GPU.

The whole step runs on the library: the scaled embedding with its gradient by sorted tokens,
gated MLPs that keep 8-bit checkpoints between the passes, the preference or the policy loss
from the logits, and FusedAdamW (FP32 masters, gradient statistics, loss scaling) on the
gradients.  The task is synthetic: a preferred continuation repeats its prompt's last token,
the other one is random; the policy is then rewarded for repeating.

    python examples/preference_training.py [--steps 60] [--dtype bf16]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from amsgrad_optimizer_step_gb300 import layers  # noqa: E402
from amsgrad_optimizer_step_gb300.optim import FusedAdamW, GradScaler  # noqa: E402


class SmallModel(torch.nn.Module):
    """Embedding, gated MLP blocks over each token and the token before it, and a head."""

    def __init__(self, vocab: int, width: int, hidden: int, blocks: int, dtype: torch.dtype,
                 device, seed: int = 0):
        super().__init__()
        gen = torch.Generator(device=device).manual_seed(seed)

        def matrix(rows, cols, sigma):
            x = torch.randn(rows, cols, device=device, generator=gen) * sigma
            return torch.nn.Parameter(x.to(dtype))

        self.embed = matrix(vocab, width, 1 / math.sqrt(width))
        self.mix = matrix(width, width, 1 / math.sqrt(width))
        self.gate_up = torch.nn.ParameterList(
            [matrix(2 * hidden, width, 1 / math.sqrt(width)) for _ in range(blocks)])
        self.down = torch.nn.ParameterList(
            [matrix(width, hidden, 0.5 / math.sqrt(hidden)) for _ in range(blocks)])
        self.head = matrix(vocab, width, 1 / math.sqrt(width))

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        """Logits of the token after each of the packed ``ids``."""
        x = layers.embedding(ids, self.embed, scale=math.sqrt(self.embed.shape[1]))
        x = x + torch.roll(x, 1, 0) @ self.mix.t()
        for gate_up, down in zip(self.gate_up, self.down):
            normed = torch.nn.functional.layer_norm(x, x.shape[-1:])
            x = x + layers.gated_down(normed @ gate_up.t(), down)
        return torch.nn.functional.layer_norm(x, x.shape[-1:]) @ self.head.t()


def pairs_batch(pairs: int, vocab: int, gen) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(ids, labels, offsets) of packed pairs; labels are the next tokens, -100 in prompts."""
    ids, labels, offsets = [], [], [0]
    for _ in range(pairs):
        prompt = torch.randint(0, vocab, (int(torch.randint(2, 9, (1,), generator=gen)),),
                               generator=gen)
        for preferred in (True, False):
            n = int(torch.randint(3, 12, (1,), generator=gen))
            answer = (prompt[-1:].repeat(n) if preferred
                      else torch.randint(0, vocab, (n,), generator=gen))
            seq = torch.cat([prompt, answer])
            ids.append(seq[:-1])
            labels.append(torch.where(torch.arange(len(seq) - 1) < len(prompt) - 1,
                                      torch.tensor(-100), seq[1:]))
            offsets.append(offsets[-1] + len(seq) - 1)
    return torch.cat(ids), torch.cat(labels), torch.tensor(offsets)


def train(steps: int = 60, dtype: str = "bf16", vocab: int = 515, width: int = 136,
          hidden: int = 360, blocks: int = 2, pairs: int = 24, log=print) -> dict:
    """Returns the losses of the preference phase, the rewards of the policy phase and the
    number of steps that the optimizer skipped."""
    device = torch.device("cuda", 0)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator().manual_seed(1)
    model = SmallModel(vocab, width, hidden, blocks, dt, device)
    reference = SmallModel(vocab, width, hidden, blocks, dt, device)
    reference.requires_grad_(False)
    opt = FusedAdamW(model.parameters(), lr=2e-3, weight_decay=0.01, max_grad_norm=1.0)
    scaler = GradScaler(init_scale=2.0 ** 10)
    losses, rewards, skipped = [], [], 0

    for step in range(steps):
        ids, labels, offsets = (x.to(device) for x in pairs_batch(pairs, vocab, gen))
        opt.zero_grad()
        with torch.no_grad():
            ref_logp = layers.token_logprobs(reference(ids), labels)
        loss, reward = layers.preference_loss(model(ids), labels, offsets, ref_logp, beta=0.5)
        scaler.scale(loss).backward()
        scaler.step(opt)
        scaler.update()
        skipped += opt.last_report["skipped"]
        losses.append(loss.item())
        if step % 20 == 0:
            log(f"preference step {step}: loss {losses[-1]:.4f}, margin "
                f"{(reward[:, 0] - reward[:, 1]).mean().item():.3f}")

    for step in range(steps):
        ids = torch.randint(0, vocab, (pairs * 16,), generator=gen).to(device)
        logits = model(ids)
        with torch.no_grad():  # one sampled token after each; 1 for repeating
            drawn = torch.distributions.Categorical(logits=logits.float()).sample()
            gain = (drawn == ids).float()
            old_logp = layers.token_logprobs(logits, drawn)
            ref_logp = layers.token_logprobs(reference(ids), drawn)
        for epoch in range(2):  # the second on tokens of an older policy
            logits = model(ids) if epoch else logits
            opt.zero_grad()
            summary, dlogits = layers.policy_step(
                logits, drawn, old_logp, (gain - gain.mean()) / (gain.std() + 1e-3), ref_logp,
                clip_low=0.2, clip_high=0.28, kl_coef=0.01, loss_scale=scaler.get_scale())
            logits.backward(dlogits)
            scaler.step(opt)
            scaler.update()
            skipped += opt.last_report["skipped"]
        rewards.append(gain.mean().item())
        if step % 20 == 0:
            loss, kl, clipped, count = summary.tolist()
            log(f"policy step {step}: reward {rewards[-1]:.3f}, loss {loss:.4f}, KL {kl:.4f}, "
                f"clipped {clipped:.3f} of {count:.0f}")
    return {"losses": losses, "rewards": rewards, "skipped": skipped}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=("f32", "f16", "bf16"), default="bf16")
    args = ap.parse_args()
    out = train(args.steps, args.dtype)
    print(f"loss {out['losses'][0]:.4f} -> {out['losses'][-1]:.4f}, reward "
          f"{out['rewards'][0]:.3f} -> {out['rewards'][-1]:.3f}, {out['skipped']} steps skipped")
