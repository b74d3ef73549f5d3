"""The model-side operators of a training step, as measurable cases.

Embedding lookup and its gradient, the preference loss and the clipped policy loss from
the logits, and the gated activation with its 8-bit checkpoint.  ``run`` computes a case in
its plain form (elementary torch operations in FP32, rounded once at the end) or, with
``own`` set, through the library's entry points.  ``exact`` gives the same outputs from the
definitions in FP64.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BETA, CLIP_LOW, CLIP_HIGH = 0.1, 0.2, 0.28
BLOCK = 128  # columns that share one scale of an 8-bit checkpoint
TINY = 2.0 ** -100  # blocks below this magnitude are stored as zeros


def listed():
    return [
        # one generation step of 32 sequences: the decoder's table, latency only
        dict(name="lookup_decode_bf16", op="lookup", tokens=32, vocab=32000, dim=2048,
             dtype="bf16", ids="i64", scale=1.0),
        # the token batch of a training step, scaled by sqrt(dim)
        dict(name="lookup_batch_bf16", op="lookup", tokens=65536, vocab=32000, dim=2048,
             dtype="bf16", ids="i64", scale=45.254834),
        # a small odd table (a test-sized model) with FP32 gradients
        dict(name="embgrad_small_f32", op="embgrad", tokens=333, vocab=1009, dim=515,
             dtype="f32", ids="i32", scale=1.0, skew=1.0),
        # the decoder's table after a training batch whose tokens follow a Zipf law
        dict(name="embgrad_batch_bf16", op="embgrad", tokens=65536, vocab=32000, dim=2048,
             dtype="bf16", ids="i64", scale=45.254834, skew=1.0),
        # one short pair in FP32, odd vocabulary: the smallest step
        dict(name="preference_step_small_f32", op="preference", pairs=1, max_len=57, vocab=8191,
             dtype="f32", smoothing=0.1, average=False, backward=True),
        # validation: loss and rewards only, ragged pairs with prompts, FP16 logits
        dict(name="preference_eval_f16", op="preference", pairs=6, max_len=513, vocab=32000,
             dtype="f16", smoothing=0.0, average=True, backward=False),
        # a training batch of packed pairs over the decoder's vocabulary
        dict(name="preference_step_bf16", op="preference", pairs=12, max_len=1024, vocab=32000,
             dtype="bf16", smoothing=0.0, average=False, backward=True),
        # a few tokens of one rollout, FP32
        dict(name="policy_step_small_f32", op="policy", tokens=61, vocab=32000, dtype="f32",
             weighted=False, kl=0.05),
        # a large vocabulary (its row passes one SM's shared memory), weighted by sequence
        dict(name="policy_step_wide_bf16", op="policy", tokens=1111, vocab=131072, dtype="bf16",
             weighted=True, kl=0.02),
        # a policy batch over the decoder's vocabulary
        dict(name="policy_step_bf16", op="policy", tokens=16384, vocab=32000, dtype="bf16",
             weighted=False, kl=0.05),
        # a few rows of an odd width, FP16, forward then backward from the checkpoint
        dict(name="gated_step_small_f16", op="gated", rows=37, cols=1403, dtype="f16",
             act="gelu_tanh"),
        # the decoder's MLP over a training batch: gate and up are halves of one projection
        dict(name="gated_step_bf16", op="gated", rows=16384, cols=5632, dtype="bf16", act="silu"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["lookup", "embgrad", "preference", "policy", "gated"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    half = 2 if dtype == "f32" else 1
    if op in ("lookup", "embgrad"):
        dim = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            dim = (dim + 7) // 8 * 8
            dim += 8 if dim == 3072 else 0
        vocab = _log_int(rng, 100, min(131072, 65_000_000 // (dim * half)))
        tokens = _log_int(rng, 1, min(262144, 130_000_000 // (dim * half)))
        case = dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=dtype,
                    ids=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 0.5, 45.254834]))
        if op == "embgrad":
            case["skew"] = rng.choice([0.0, 1.0, 1.5])
        return case
    if op == "gated":
        cols = _log_int(rng, 65, 16384)
        if rng.random() < 0.7:
            cols = (cols + 127) // 128 * 128
            cols += 128 if cols == 3072 else 0
        rows = _log_int(rng, 1, min(65536, 90_000_000 // (cols * half)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, act=rng.choice(["silu", "gelu_tanh"]))
    vocab = _log_int(rng, 500, 131072)
    if rng.random() < 0.7:
        vocab = (vocab + 63) // 64 * 64
        vocab += 64 if vocab == 3072 else 0
    most = 400_000_000 // (vocab * half)
    if op == "policy":
        return dict(op=op, tokens=_log_int(rng, 1, min(16384, most)), vocab=vocab, dtype=dtype,
                    weighted=rng.random() < 0.5, kl=rng.choice([0.0, 0.05]))
    max_len = _log_int(rng, 3, max(4, min(2048, most // 4)))
    pairs = _log_int(rng, 1, max(1, min(64, most // (2 * max_len))))
    return dict(op=op, pairs=pairs, max_len=max_len, vocab=vocab, dtype=dtype,
                smoothing=rng.choice([0.0, 0.1]), average=rng.random() < 0.5,
                backward=rng.random() < 0.7)


# ---- inputs ------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))


def _token_ids(gen, tokens, vocab, skew):
    """Token ids whose frequencies fall as rank^-skew (0: uniform), ranks scattered."""
    rank = torch.arange(1, vocab + 1, device=DEV, dtype=torch.float64)
    cdf = torch.cumsum(rank ** -skew, 0)
    u = torch.rand(tokens, device=DEV, dtype=torch.float64, generator=gen) * cdf[-1]
    drawn = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    return torch.randperm(vocab, device=DEV, generator=gen)[drawn]


def _lengths(pairs, max_len):
    """Ragged lengths of 2 * pairs sequences: the longest first, the others between half and all."""
    low = max(1, max_len // 2)
    return [max_len - int((max_len - low + 1) * (0.618034 * j % 1.0)) for j in range(2 * pairs)]


def _logits(gen, tokens, vocab, dtype):
    """Logits of a language model: a spread of a few units with the label standing out."""
    logits = torch.empty(tokens, vocab, device=DEV, dtype=TYPES[dtype])
    labels = torch.randint(0, vocab, (tokens,), device=DEV, generator=gen)
    rows = max(1, (1 << 27) // vocab)
    logp = torch.empty(tokens, device=DEV)
    for a in range(0, tokens, rows):
        b = min(tokens, a + rows)
        x = torch.randn(b - a, vocab, device=DEV, generator=gen).mul_(2.0)
        lift = torch.rand(b - a, 1, device=DEV, generator=gen) * 14.0
        x.scatter_add_(1, labels[a:b, None], lift)
        logits[a:b] = x.to(TYPES[dtype])
        x = logits[a:b].float()
        logp[a:b] = x.gather(1, labels[a:b, None])[:, 0] - torch.logsumexp(x, 1)
    return logits, labels, logp


def _noise(gen, like, sigma):
    return like + sigma * torch.randn(like.shape, device=DEV, generator=gen)


def _off_edges(log_ratio):
    """Log ratios moved off the clip's two edges, where one rounding would choose the branch."""
    for edge in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
        log_ratio = torch.where((log_ratio - edge).abs() < 1e-4, log_ratio + 3e-4, log_ratio)
    return log_ratio


def prepare(case, seed):
    gen = _generator(seed)
    dt = TYPES[case["dtype"]]
    op = case["op"]
    s = dict(case)
    if op in ("lookup", "embgrad"):
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        ids = _token_ids(gen, t, v, case.get("skew", 1.0))
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        if op == "lookup":
            s["table"] = (torch.randn(v, d, device=DEV, generator=gen) * 0.02).to(dt)
            s["out"] = torch.empty(t, d, device=DEV, dtype=dt)
        else:
            s["dout"] = (torch.randn(t, d, device=DEV, generator=gen) * 1e-3).to(dt)
            s["dtable"] = torch.empty(v, d, device=DEV, dtype=dt)
        return s
    if op == "gated":
        r, c = case["rows"], case["cols"]
        # gate and up are the two halves of one projection's output, and so are their gradients
        x = (torch.randn(r, 2 * c, device=DEV, generator=gen) * 1.5).to(dt)
        s["gate"], s["up"] = x[:, :c], x[:, c:]
        s["dh"] = (torch.randn(r, c, device=DEV, generator=gen) * 1e-2).to(dt)
        s["h"] = torch.empty(r, c, device=DEV, dtype=dt)
        s["h_again"] = torch.empty(r, c, device=DEV, dtype=dt)
        s["dx"] = torch.empty(r, 2 * c, device=DEV, dtype=dt)
        return s
    if op == "preference":
        lens = torch.tensor(_lengths(case["pairs"], case["max_len"]))
        off = torch.zeros(2 * case["pairs"] + 1, dtype=torch.int64)
        off[1:] = torch.cumsum(lens, 0)
        tokens = int(off[-1])
        s["offsets"] = off.to(DEV)
    else:
        tokens = case["tokens"]
    logits, labels, logp = _logits(gen, tokens, case["vocab"], case["dtype"])
    if op == "preference":
        # a prompt opens each sequence: its tokens are not counted, and neither are a few others
        pos = torch.arange(tokens, device=DEV)
        seq = torch.bucketize(pos, s["offsets"][1:], right=True)
        prompt = (s["offsets"][1:] - s["offsets"][:-1]) // 4
        hidden = (pos - s["offsets"][:-1][seq]) < prompt[seq]
        s["ref_logp"] = _noise(gen, logp, 0.3)
    else:
        hidden = torch.rand(tokens, device=DEV, generator=gen) < 0.1
        s["old_logp"] = logp - _off_edges(0.2 * torch.randn(tokens, device=DEV, generator=gen))
        s["ref_logp"] = _noise(gen, logp, 0.4)
        s["advantages"] = 0.5 + torch.randn(tokens, device=DEV, generator=gen)
        s["weights"] = None
        if case["weighted"]:
            s["weights"] = torch.rand(tokens, device=DEV, generator=gen) / max(1, tokens)
    s["labels"] = torch.where(hidden, torch.full_like(labels, -100), labels)
    s["logits"] = logits
    s["dlogits"] = torch.empty_like(logits)
    # the loss scale of mixed precision keeps FP16 gradients in range
    s["grad_scale"] = 65536.0 if case["dtype"] == "f16" else 1.0
    return s


# ---- one pass ------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import amsgrad_optimizer_step_gb300 as fa
    op = s["op"]
    if op == "lookup":
        fa.fa_embedding_lookup(s["ids"], s["table"], s["out"], s["scale"])
        return s["out"]
    if op == "embgrad":
        if "scratch" not in s:
            s["scratch"] = fa.embedding_scratch(s["tokens"], s["vocab"], s["dim"], DEV)
        fa.fa_embedding_gradient(s["ids"], s["dout"], s["dtable"], s["scratch"], s["scale"])
        return s["dtable"]
    if op == "gated":
        if "checkpoint" not in s:
            s["checkpoint"] = fa.checkpoint_buffer(s["rows"], s["cols"], DEV)
        c = s["cols"]
        fa.fa_gated_forward(s["gate"], s["up"], s["h"], s["checkpoint"], s["act"])
        fa.fa_gated_backward(s["checkpoint"], s["dh"], s["dx"][:, :c], s["dx"][:, c:],
                             s["h_again"], s["act"])
        return {"h": s["h"], "dx": s["dx"], "h_again": s["h_again"]}
    if op == "preference":
        if "buffers" not in s:
            s["buffers"] = fa.preference_buffers(s["logits"].shape[0], s["pairs"], DEV)
        b = s["buffers"]
        fa.fa_preference_loss(s["logits"], s["labels"], s["offsets"], s["ref_logp"], b,
                              beta=BETA, label_smoothing=s["smoothing"], average=s["average"])
        out = {"loss": b.loss, "pair_loss": b.pair_loss, "rewards": b.rewards, "logp": b.logp}
        if s["backward"]:
            fa.fa_token_logprobs_gradient(s["logits"], s["labels"], b.lse, b.dlogp, s["dlogits"],
                                          grad_scale=s["grad_scale"])
            out["dlogits"] = s["dlogits"]
        return out
    if "buffers" not in s:
        s["buffers"] = fa.policy_buffers(s["tokens"], DEV)
    b = s["buffers"]
    fa.fa_policy_loss(s["logits"], s["labels"], s["old_logp"], s["advantages"], b,
                      ref_logp=s["ref_logp"], weights=s["weights"], dlogits=s["dlogits"],
                      clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=s["kl"],
                      denominator=1.0 if s["weighted"] else 0.0, grad_scale=s["grad_scale"])
    return {"loss": b.loss, "kl": b.kl, "clip_fraction": b.clip_fraction, "logp": b.logp,
            "token_loss": b.token_loss, "token_kl": b.token_kl, "dlogits": s["dlogits"]}


def _run_plain(s):
    op = s["op"]
    dt = TYPES[s["dtype"]]
    if op == "lookup":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(dt)
    if op == "embgrad":
        acc = torch.zeros(s["vocab"], s["dim"], device=DEV)
        acc.index_add_(0, s["ids"].long(), s["dout"].float())
        return (acc * s["scale"]).to(dt)
    if op == "gated":
        return _gated_plain(s, dt)
    x = s["logits"].float()
    counted = s["labels"] >= 0
    y = s["labels"].clamp(min=0)[:, None]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    logp = (x.gather(1, y) - top - torch.log(total))[:, 0]
    logp = torch.where(counted, logp, torch.zeros_like(logp))
    if op == "preference":
        out, dlogp = _preference_plain(s, logp, counted)
        out["logp"] = logp
    else:
        out, dlogp = _policy_plain(s, logp, counted)
        out["logp"] = logp
    if s.get("backward", True):
        c = (dlogp * s["grad_scale"])[:, None]
        g = e * (-c / total)
        g.scatter_add_(1, y, c)
        out["dlogits"] = torch.where(counted[:, None], g, torch.zeros_like(g)).to(dt)
    return out


def _preference_plain(s, logp, counted):
    seqs, tokens = 2 * s["pairs"], logp.shape[0]
    pos = torch.arange(tokens, device=DEV)
    member = (pos >= s["offsets"][:-1, None]) & (pos < s["offsets"][1:, None]) & counted
    ratio = torch.where(counted, logp - s["ref_logp"], torch.zeros_like(logp))
    sums = torch.where(member, ratio, torch.zeros_like(ratio)).sum(1)
    count = member.sum(1).float() if s["average"] else torch.ones(seqs, device=DEV)
    mean = sums / count.clamp(min=1.0)
    m = BETA * (mean[0::2] - mean[1::2])
    eps = s["smoothing"]

    def softplus(z):
        return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))

    pair_loss = (1 - eps) * softplus(-m) + eps * softplus(m)
    dm = (-(1 - eps) / (1 + torch.exp(m)) + eps / (1 + torch.exp(-m))) * BETA / s["pairs"]
    dsum = torch.stack([dm, -dm], 1).reshape(-1) / count.clamp(min=1.0)
    dlogp = torch.where(member, dsum[:, None], torch.zeros_like(dsum)[:, None]).sum(0)
    return {"loss": pair_loss.mean().reshape(1), "pair_loss": pair_loss,
            "rewards": (BETA * mean).reshape(-1, 2)}, dlogp


def _policy_plain(s, logp, counted):
    zero = torch.zeros_like(logp)
    r = torch.exp(logp - s["old_logp"])
    a = s["advantages"]
    free, held = r * a, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
    d = s["ref_logp"] - logp
    kl = torch.where(counted, torch.expm1(d) - d, zero)
    token_loss = torch.where(counted, -torch.minimum(free, held) + s["kl"] * kl, zero)
    n = counted.sum().float()
    w = s["weights"] if s["weighted"] else 1.0 / n.clamp(min=1.0)
    dlogp = torch.where(free <= held, -free, zero) - s["kl"] * torch.expm1(d)
    clipped = (counted & (free > held)).sum().float()
    n = n.clamp(min=1.0)
    return {"loss": (w * token_loss).sum().reshape(1), "kl": (kl.sum() / n).reshape(1),
            "clip_fraction": (clipped / n).reshape(1), "token_loss": token_loss,
            "token_kl": kl}, dlogp * w


def _in_blocks(x):
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    if blocks * BLOCK != cols:
        x = torch.cat([x, x.new_zeros(rows, blocks * BLOCK - cols)], 1)
    return x.reshape(rows, blocks, BLOCK)


def _stored_plain(x):
    """What an 8-bit checkpoint of x stands for."""
    b = _in_blocks(x)
    top = b.abs().amax(2, keepdim=True)
    kept = top >= TINY
    most = torch.full_like(top, 127.0)  # a tensor: division by a number may use its reciprocal
    inv = torch.where(kept, most / top, torch.zeros_like(top))
    scale = torch.where(kept, top / most, torch.zeros_like(top))
    return (torch.round(b * inv) * scale).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _act_plain(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    k = math.sqrt(2 / math.pi)
    u = k * (g + 0.044715 * g * g * g)
    sig = 1 / (1 + torch.exp(-2 * u))
    return g * sig, sig + g * sig * (1 - sig) * 2 * k * (1 + 3 * 0.044715 * g * g)


def _gated_plain(s, dt):
    g, u, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
    h = _act_plain(g, s["act"])[0] * u
    g, u = _stored_plain(g), _stored_plain(u)
    a, da = _act_plain(g, s["act"])
    return {"h": h.to(dt), "dx": torch.cat([dh * u * da, dh * a], 1).to(dt),
            "h_again": (a * u).to(dt)}


# ---- the definitions in FP64 -----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "lookup":
        return torch.nn.functional.embedding(s["ids"].long(), s["table"].to(f64)) * case["scale"]
    if op == "embgrad":
        w = torch.zeros(case["vocab"], case["dim"], device=DEV, dtype=f64, requires_grad=True)
        y = torch.nn.functional.embedding(s["ids"].long(), w) * case["scale"]
        return torch.autograd.grad(y, w, s["dout"].to(f64))[0]
    if op == "gated":
        act = (torch.nn.functional.silu if case["act"] == "silu"
               else lambda z: torch.nn.functional.gelu(z, approximate="tanh"))

        def stored(x):
            pad = -x.shape[1] % BLOCK
            b = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, BLOCK))
            step = b.abs().amax(2, keepdim=True).clamp(min=TINY) / 127
            return (torch.round(b / step) * step).flatten(1)[:, :x.shape[1]]

        g, u = s["gate"].to(f64), s["up"].to(f64)
        h = act(g) * u
        g, u = stored(g).requires_grad_(), stored(u).requires_grad_()
        again = act(g) * u
        dg, du = torch.autograd.grad(again, (g, u), s["dh"].to(f64))
        return {"h": h, "dx": torch.cat([dg, du], 1), "h_again": again.detach()}
    x = s["logits"].to(f64).requires_grad_(case.get("backward", True))
    counted = s["labels"] >= 0
    logp = torch.log_softmax(x, 1).gather(1, s["labels"].clamp(min=0)[:, None])[:, 0]
    logp = logp.masked_fill(~counted, 0.0)
    ref = s["ref_logp"].to(f64)
    if op == "preference":
        off = s["offsets"].tolist()
        sums = []
        for a, b in zip(off[:-1], off[1:]):
            total = (logp[a:b] - ref[a:b])[counted[a:b]].sum()
            sums.append(total / max(1, int(counted[a:b].sum())) if case["average"] else total)
        rewards = BETA * torch.stack(sums).reshape(-1, 2)
        m = rewards[:, 0] - rewards[:, 1]
        eps = case["smoothing"]
        soft = torch.nn.functional.softplus
        pair_loss = (1 - eps) * soft(-m) + eps * soft(m)
        loss = pair_loss.mean().reshape(1)
        out = {"loss": loss.detach(), "pair_loss": pair_loss.detach(),
               "rewards": rewards.detach(), "logp": logp.detach()}
        if case["backward"]:
            out["dlogits"] = torch.autograd.grad(loss.sum() * s["grad_scale"], x)[0]
        return out
    ratio = torch.exp(logp - s["old_logp"].to(f64))
    adv = s["advantages"].to(f64)
    free, held = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    d = ref - logp
    kl = (torch.exp(d) - d - 1).masked_fill(~counted, 0.0)
    token_loss = (-torch.minimum(free, held)).masked_fill(~counted, 0.0) + case["kl"] * kl
    n = counted.sum().to(f64)
    w = s["weights"].to(f64) if case["weighted"] else 1 / n.clamp(min=1)
    loss = (w * token_loss).sum()
    g = torch.autograd.grad(loss * s["grad_scale"], x)[0]
    share = ((free > held) & counted).sum().to(f64) / n.clamp(min=1)
    return {"loss": loss.detach().reshape(1),
            "kl": (kl.detach().sum() / n.clamp(min=1)).reshape(1),
            "clip_fraction": share.reshape(1), "logp": logp.detach(), "token_loss": token_loss.detach(),
            "token_kl": kl.detach(), "dlogits": g}


# ---- what a pass cannot do without -------------------------------------------------------

def _distinct(tokens, vocab):
    """Expected distinct ids among Zipf-distributed tokens: rows of the table that are read."""
    p = torch.arange(1, vocab + 1, dtype=torch.float64) ** -1.0
    return float((1 - (1 - p / p.sum()) ** tokens).sum())


def work(case):
    b = SIZE[case["dtype"]]
    op = case["op"]
    if op in ("lookup", "embgrad"):
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        ids = t * (4 if case["ids"] == "i32" else 8)
        if op == "lookup":
            return {"bytes": ids + (_distinct(t, v) + t) * d * b, "flops": t * d}
        return {"bytes": ids + (t + v) * d * b, "flops": t * d}
    if op == "gated":
        n = case["rows"] * case["cols"]
        scales = case["rows"] * -(-case["cols"] // BLOCK) * 2 * 4
        return {"bytes": n * (2 * b + b + 2) + n * (2 + b + 3 * b) + 2 * scales, "flops": 40 * n}
    if op == "policy":
        # one token in ten is not counted: its row need not be read
        n = case["tokens"] * case["vocab"]
        return {"bytes": int(1.9 * n) * b + 36 * case["tokens"], "flops": 6 * n}
    lens = _lengths(case["pairs"], case["max_len"])
    tokens = sum(lens)
    n = tokens * case["vocab"]
    # prompts are a quarter of each sequence: their rows of logits need not be read
    read = sum(length - length // 4 for length in lens) * case["vocab"]
    if not case["backward"]:
        return {"bytes": read * b + 20 * tokens, "flops": 3 * n}
    return {"bytes": (read + n) * b + 28 * tokens, "flops": 6 * n}
