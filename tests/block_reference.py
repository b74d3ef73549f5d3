"""The residual blocks' operators from their definitions, in 64 bits, for the tests.

Plain numpy and torch in float64; nothing here uses the library.  Each result comes with the
FP32 error that the arithmetic may make, as far as the comparisons need it.
"""

from __future__ import annotations

import numpy as np
import torch

from model_reference import U32

MASK = 0xFFFFFFFF
LEVELS = 65536


# ---- dropout -----------------------------------------------------------------------

def philox(counter, key):
    """Philox 4x32-10 of uint64 arrays of 32-bit words: counter [4], key (two ints)."""
    u = np.uint64
    c = [np.asarray(x, dtype=u) for x in counter]
    k0, k1 = key
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & u(MASK), (a >> u(32)) ^ c[3] ^ u(k1), a & u(MASK)]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return c


def dropped_share(p):
    return int(np.rint(LEVELS * p))


def kept(rows, cols, p, seed, call, device):
    """Bool [rows, cols]: which elements a dropout keeps."""
    blocks = -(-cols // 8)
    at = np.arange(rows * blocks, dtype=np.uint64)
    call &= (1 << 64) - 1
    seed &= (1 << 64) - 1
    words = philox([at & np.uint64(MASK), at >> np.uint64(32), np.full_like(at, call & MASK),
                    np.full_like(at, call >> 32)], (seed & MASK, seed >> 32))
    parts = [(words[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF) for j in range(8)]
    bits = np.stack(parts, 1).reshape(rows, 8 * blocks)[:, :cols].astype(np.int64)
    return torch.from_numpy(bits >= dropped_share(p)).to(device)


def keep_scale(p):
    q = dropped_share(p)
    return LEVELS / (LEVELS - q) if q < LEVELS else 0.0


# ---- the join ----------------------------------------------------------------------

def _weight(w, offset, like):
    return torch.ones_like(like[0]) if w is None else w.double() + offset


def _gate(gate, rows):
    return 1.0 if gate is None else gate.double().repeat_interleave(rows // gate.shape[0], 0)


# The longest chain of additions that a row's sum goes through (eight pairs of a lane, five steps of a
# warp, eight groups of warps) and the roundings of its terms, in halves: what its root is off by.
ROOT = 16 * U32


def join(residual, branch, post_weight, gate, post_norm, alpha, beta, eps, offset, mask, scale):
    """(out, its FP32 error, 1 / root of the branch or None)."""
    r = residual.double()
    out, err = alpha * r, 2 * U32 * (alpha * r).abs()
    if branch is None:
        return out, err, None
    b, rstd = branch.double(), None
    if post_norm:
        rstd = 1 / torch.sqrt(b.square().mean(1, keepdim=True) + eps)
        b = b * rstd * _weight(post_weight, offset, b)
    share = beta * scale * _gate(gate, b.shape[0]) * b
    if mask is not None:
        share = torch.where(mask, share, torch.zeros_like(share))
    out = out + share
    return out, err + (ROOT + 8 * U32) * share.abs() + U32 * out.abs(), rstd


def norm(x, weight, eps, offset):
    """(normed, its FP32 error, 1 / root) of the rows as they are given."""
    x = x.double()
    rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)
    y = x * rstd * _weight(weight, offset, x)
    return y, (ROOT + 5 * U32) * y.abs(), rstd


def join_gradient(out, branch, dout, dnormed, post_rstd, pre_rstd, post_weight, pre_weight, gate,
                  post_norm, alpha, beta, offset, mask, scale):
    """{name: (gradient, FP32 error)} from the stored stream and the FP32 inverse roots."""
    rows = next(t for t in (branch, dnormed, dout) if t is not None).shape[0]
    some = next(t for t in (branch, dnormed, dout) if t is not None).double()
    zero = torch.zeros_like(some)
    total, err = (zero, zero) if dout is None else (dout.double(), zero)
    result = {}
    xh, back = zero, 0.0
    # a row's sum over its columns: as ROOT, but not halved, and the terms' own roundings
    s_err = 2 * ROOT + 8 * U32
    if dnormed is not None:
        rp = pre_rstd.double()[:, None]
        xh = out.double() * rp
        d = dnormed.double() * _weight(pre_weight, offset, some)
        mean, mean_abs = (d * xh).mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
        back = rp * mean
        err = 6 * U32 * (total.abs() + (rp * d).abs()) + (rp * xh).abs() * (
            s_err * mean_abs + 4 * U32 * mean.abs())
        total = total + rp * (d - xh * mean)
        err = err + 2 * U32 * total.abs()
        p = dnormed.double() * xh
        result["dpre_weight"] = p.sum(0), (rows + 8) * U32 * p.abs().sum(0)
    result["dresidual"] = alpha * total, abs(alpha) * err + 2 * U32 * (alpha * total).abs()
    if branch is None:
        return result
    y = branch.double()
    yh = y * post_rstd.double()[:, None] if post_norm else y
    g = _gate(gate, rows)
    w = _weight(post_weight, offset, some) if post_norm else torch.ones_like(some[0])

    def on(x):
        return x if mask is None else torch.where(mask, x, torch.zeros_like(x))

    v = on(yh)
    k, k_err = beta * scale * v * total, (beta * scale * v).abs() * (err + 6 * U32 * total.abs())
    if gate is not None:
        groups = gate.shape[0]
        x = (w * k).reshape(groups, -1, some.shape[1])
        e = (w.abs() * k_err).reshape(x.shape)
        result["dgate"] = x.sum(1), e.sum(1) + (x.shape[1] + 8) * U32 * x.abs().sum(1)
    if post_weight is not None and post_norm:
        x = g * k
        result["dpost_weight"] = x.sum(0), (abs(g) * k_err).sum(0) + (rows + 8) * U32 * x.abs().sum(0)
    a = on(beta * scale * g * w * torch.ones_like(some))
    db, db_err = a * total, a.abs() * (err + 6 * U32 * total.abs())
    if post_norm:
        rq = post_rstd.double()[:, None]
        q = a * yh
        mean = (q * total).mean(1, keepdim=True)
        size = (q * total).abs().mean(1, keepdim=True)
        if dnormed is not None:  # the kernel takes it as two sums
            size = size + (q * back * xh).abs().mean(1, keepdim=True) * 2
        mean_err = s_err * size + (q.abs() * err).mean(1, keepdim=True)
        db_err = rq * (db_err + yh.abs() * (mean_err + 4 * U32 * mean.abs()) +
                       4 * U32 * (db.abs() + (yh * mean).abs()))
        db = rq * (db - yh * mean)
    result["dbranch"] = db, db_err + 2 * U32 * db.abs()
    return result


# ---- the router ----------------------------------------------------------------------

def chosen(logits, k, counted):
    """The k largest logits' experts of each token: ties to the lower number, NaN the largest."""
    x = logits.double()
    left = torch.where(torch.isnan(x), torch.full_like(x, torch.inf), x)
    rank = torch.isnan(x).double()  # NaN before +Inf
    taken = torch.zeros_like(x, dtype=torch.bool)
    out = []
    numbers = torch.arange(x.shape[1], device=x.device)
    for _ in range(k):
        free = ~taken
        top_rank = torch.where(free, rank, -1.0).amax(1, keepdim=True)
        free = free & (rank == top_rank)
        top = torch.where(free, left, -torch.inf).amax(1, keepdim=True)
        free = free & (left == top)
        e = torch.where(free, numbers, x.shape[1]).amin(1, keepdim=True)
        taken.scatter_(1, e, True)
        out.append(e)
    e = torch.cat(out, 1)
    return e if counted is None else torch.where(counted[:, None], e, torch.full_like(e, -1))


def route(logits, k, counted, renormalise, weight_scale, balance_coef, z_coef):
    """dict of the outputs, differentiable in ``logits`` (float64)."""
    t, e = logits.shape
    on = torch.ones(t, dtype=torch.bool, device=logits.device) if counted is None else counted
    which = chosen(logits.detach(), k, None)
    x = torch.where(on[:, None], logits, torch.zeros_like(logits))
    p = torch.softmax(x, 1)
    w = p.gather(1, which)
    if renormalise:
        w = w / w.sum(1, keepdim=True)
    w = torch.where(on[:, None], w * weight_scale, torch.zeros_like(w))
    n = int(on.sum())
    counts = torch.bincount(which[on].reshape(-1), minlength=e)
    mean_prob = p[on].sum(0) / max(1, n)
    balance = e * (counts.double() / max(1, n * k) * mean_prob).sum()
    z = torch.logsumexp(x, 1)[on].square().sum() / max(1, n)
    return dict(chosen=torch.where(on[:, None], which, torch.full_like(which, -1)), weights=w,
                counts=counts, mean_prob=mean_prob, balance=balance, z=z,
                loss=balance_coef * balance + z_coef * z, n=n, p=p)
