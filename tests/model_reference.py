"""The model-side operators from their definitions, in 64 bits, for the tests.

Plain torch in float64 on the inputs' device; nothing here uses the library.  Rounding
units of the output types and the FP32 error terms of the comparisons are here too.
"""

from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: U32, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SUBNORMAL = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def assert_close(got: torch.Tensor, want: torch.Tensor, fp32_error, what: str) -> None:
    """|got - want| <= one rounding to got's type + fp32_error (a bound on the FP32
    arithmetic's error, per element or one for all); non-finite values must agree."""
    dt = got.dtype
    g, w = got.double(), want.double().to(got.device)
    big = torch.finfo(dt).max
    fine = torch.isfinite(w) & (w.abs() <= big)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN in other places"
    over = ~fine & ~torch.isnan(w)
    assert bool((torch.isinf(g[over]) & (torch.sign(g[over]) == torch.sign(w[over]))).all()), \
        f"{what}: infinities differ"
    err = (g - w).abs()[fine]
    if not err.numel():
        return
    f = torch.as_tensor(fp32_error, dtype=torch.float64, device=got.device).expand(w.shape)[fine]
    bound = UNIT[dt] * (w.abs()[fine] + f) + SUBNORMAL[dt] + f
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err / bound, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} beyond the bound; worst: "
                             f"got {g[fine][i].item()!r} want {w[fine][i].item()!r} bound "
                             f"{bound[i].item():.3e}")


# ---- embedding -------------------------------------------------------------------

def lookup(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table.double()[torch.where(ok, ids, torch.zeros_like(ids)).long()] * scale
    return torch.where(ok[:, None], rows, torch.zeros_like(rows))


def embedding_gradient(ids, dout, vocab, scale, padding_idx=-1, before=None):
    """(gradient, sum of magnitudes, tokens of each id)."""
    ok = (ids >= 0) & (ids < vocab) & (ids != padding_idx)
    at = ids[ok].long()
    grad = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device)
    mag = torch.zeros_like(grad)
    d = dout[ok].double()
    grad.index_add_(0, at, d)
    mag.index_add_(0, at, d.abs())
    count = torch.bincount(at, minlength=vocab)
    grad, mag = grad * scale, mag * abs(scale)
    if before is not None:
        grad = grad + before.double()
        mag = mag + before.double().abs()
    return grad, mag, count


# ---- losses from the logits ----------------------------------------------------------

def counted(labels, vocab):
    return (labels >= 0) & (labels < vocab)


def logprobs(logits, labels, scale):
    """(logp, p): 0 where the label is not an id; p the softmax rows."""
    ok = counted(labels, logits.shape[1])
    x = logits.double() * scale
    x = torch.where(ok[:, None], x, torch.zeros_like(x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    y = torch.where(ok, labels, torch.zeros_like(labels)).long()[:, None]
    logp = (x.gather(1, y) - top - torch.log(total))[:, 0]
    return torch.where(ok, logp, torch.zeros_like(logp)), e / total


def logprobs_gradient(logits, labels, p, dlogp, scale):
    ok = counted(labels, logits.shape[1])
    c = dlogp.double() * scale
    g = -p * c[:, None]
    y = torch.where(ok, labels, torch.zeros_like(labels)).long()[:, None]
    g.scatter_add_(1, y, c[:, None])
    return torch.where(ok[:, None], g, torch.zeros_like(g))


def softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def preference(logp, ref, ok, offsets, beta, smoothing, average):
    """(loss, pair_loss, rewards, dlogp)."""
    t = logp.shape[0]
    off = [min(max(int(o), 0), t) for o in offsets]
    n = (len(off) - 1) // 2
    ratio = torch.where(ok, logp.double() - ref.double(), torch.zeros_like(logp.double()))
    dlogp = torch.zeros(t, dtype=torch.float64, device=logp.device)
    pair_loss, rewards = [], []
    for k in range(n):
        s, per = [], []
        for j in (2 * k, 2 * k + 1):
            a, b = off[j], off[j + 1]
            c = max(1, int(ok[a:b].sum())) if average else 1
            s.append(ratio[a:b].sum() / c)
            per.append(1.0 / c)
        z = beta * (s[0] - s[1])
        pair_loss.append((1 - smoothing) * softplus(-z) +
                         (smoothing * softplus(z) if smoothing else 0.0))
        dz = smoothing / (1 + torch.exp(-z)) - (1 - smoothing) / (1 + torch.exp(z))
        for q, j in enumerate((2 * k, 2 * k + 1)):
            a, b = off[j], off[j + 1]
            dlogp[a:b] += torch.where(ok[a:b], (-1) ** q * dz * beta / n * per[q], 0.0)
        rewards.append(torch.stack([beta * s[0], beta * s[1]]))
    if not n:
        z = torch.zeros(0, dtype=torch.float64, device=logp.device)
        return z.sum(), z, z.reshape(0, 2), dlogp
    pair_loss = torch.stack(pair_loss)
    return pair_loss.mean(), pair_loss, torch.stack(rewards), dlogp


def policy(logp, ok, old, adv, ref, weights, lo, hi, kl_coef, denominator):
    """dict of loss, kl, clip_fraction, count, token_loss, token_kl, dlogp."""
    zero = torch.zeros_like(logp.double())
    r = torch.exp(logp.double() - old.double())
    free, held = r * adv.double(), r.clamp(1 - lo, 1 + hi) * adv.double()
    loss = -torch.minimum(free, held)
    dlogp = torch.where(free <= held, -free, torch.where(torch.isnan(free), free, zero))
    kl = zero
    if ref is not None:
        d = ref.double() - logp.double()
        kl = torch.expm1(d) - d
        if kl_coef:
            loss = loss + kl_coef * kl
            dlogp = dlogp - kl_coef * torch.expm1(d)
    n = int(ok.sum())
    denom = denominator if denominator else max(1, n)
    w = weights.double() if weights is not None else torch.ones_like(zero)
    clipped = (free > held) & ok
    loss, kl = torch.where(ok, loss, zero), torch.where(ok, kl, zero)
    return dict(loss=(w * loss).masked_fill(~ok, 0.0).sum() / denom, kl=kl.sum() / max(1, n),
                clip_fraction=clipped.sum().double() / max(1, n), count=n, token_loss=loss,
                token_kl=kl, dlogp=torch.where(ok, dlogp * w / denom, zero))


# ---- gated activation -----------------------------------------------------------------

BLOCK = 128


def act(g, kind):
    """(value, derivative) in 64 bits."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    # the tanh form as g * sigmoid(2 u), which does not cancel for negative g
    k = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * k * (1 + 3 * 0.044715 * g * g)


def quantise(x):
    """(codes int8 [rows, pitch], scales float32 [rows, blocks]) by the stated FP32 rule."""
    x = x.float()
    pad = -x.shape[1] % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, BLOCK))
    top = b.abs().amax(2, keepdim=True)
    finite = torch.isfinite(b).all(2, keepdim=True)
    kept = finite & (top >= 2.0 ** -100)
    f127 = torch.tensor(127.0, device=x.device)
    safe = torch.where(kept, top, f127)
    codes = torch.where(kept, torch.round(b * (f127 / safe)), torch.zeros_like(b))
    scales = torch.where(kept, top / f127, torch.zeros_like(top))
    scales = torch.where(finite, scales, torch.full_like(scales, math.nan))
    return codes.to(torch.int8).flatten(1), scales[:, :, 0]


def stored(codes, scales, cols):
    """What the codes stand for, in FP32 as the kernels multiply."""
    return (codes.unflatten(1, (-1, BLOCK)).float() * scales[:, :, None]).flatten(1)[:, :cols]
