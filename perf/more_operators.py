"""The operators of a training step's residual blocks, as measurable cases.

The join of a block's output to the residual stream (the norm behind the block, its gate,
dropout and the scaled addition, and the norm before the next block) with its gradient,
dropout from a counter-based generator, and the router of gated experts with its balance
loss.  ``run`` computes a case in its plain form (elementary torch operations in FP32,
rounded once at the end) or, with ``own`` set, through the library's entry points.
``exact`` gives the same outputs from the definitions in FP64.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
LEVELS = 65536  # a dropout probability is a multiple of 1 / LEVELS
BALANCE, ZLOSS = 0.01, 0.001


def listed():
    return [
        # one generation step of 32 sequences: both norms around the addition, latency only
        dict(name="join_decode_bf16", op="join", rows=32, cols=2048, dtype="bf16", stream="bf16",
             groups=0, post=True, pre=True, drop=0.0, offset=0.0, backward=False),
        # a test-sized model of odd width in FP32: three sequences with a gate each
        dict(name="join_step_small_f32", op="join", rows=39, cols=515, dtype="f32", stream="f32",
             groups=3, post=True, pre=True, drop=0.1, offset=0.0, backward=True),
        # a validation batch (an odd number of tokens), a gate for each channel
        dict(name="join_eval_f16", op="join", rows=4093, cols=4096, dtype="f16", stream="f16",
             groups=1, post=False, pre=True, drop=0.0, offset=0.0, backward=False),
        # the decoder's width over a training batch, everything on
        dict(name="join_step_bf16", op="join", rows=16384, cols=2048, dtype="bf16", stream="bf16",
             groups=1, post=True, pre=True, drop=0.1, offset=1.0, backward=True),
        # a wider model that holds its residual stream in FP32, a gate for each sequence
        dict(name="join_step_mixed", op="join", rows=4096, cols=5120, dtype="bf16", stream="f32",
             groups=8, post=True, pre=True, drop=0.0, offset=0.0, backward=True),
        # a few rows of an odd width, forward then backward
        dict(name="dropout_small_f32", op="dropout", rows=61, cols=1403, dtype="f32", drop=0.5,
             strided=False),
        # rows of odd width inside a wider matrix
        dict(name="dropout_odd_f16", op="dropout", rows=4099, cols=5633, dtype="f16", drop=0.2,
             strided=True),
        # the decoder's MLP activations of a training batch, forward then backward
        dict(name="dropout_step_bf16", op="dropout", rows=16384, cols=5632, dtype="bf16", drop=0.1,
             strided=False),
        # one generation step of 32 sequences: the choice of experts and their weights alone
        dict(name="route_decode_bf16", op="route", tokens=32, experts=64, k=8, dtype="bf16",
             renormalise=True, hidden=0.0, backward=False),
        # a small step with padding and an expert count that is no power of two
        dict(name="route_step_small_f32", op="route", tokens=333, experts=60, k=4, dtype="f32",
             renormalise=False, hidden=0.2, backward=True),
        # a training batch of tokens
        dict(name="route_step_bf16", op="route", tokens=65536, experts=128, k=8, dtype="bf16",
             renormalise=True, hidden=0.0, backward=True),
        # the router kept in FP32, many experts, a padded batch
        dict(name="route_step_wide_f32", op="route", tokens=65536, experts=256, k=8, dtype="f32",
             renormalise=False, hidden=0.1, backward=True),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["join", "dropout", "route"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    half = 2 if dtype == "f32" else 1
    if op == "join":
        stream = dtype if rng.random() < 0.7 else "f32"
        half = 2 if stream == "f32" else 1
        cols = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        rows = _log_int(rng, 1, min(65536, 33_000_000 // (cols * half)))
        groups = rng.choice([0, 1, _log_int(rng, 1, min(64, rows))])
        rows = rows // groups * groups if groups else rows
        post = rng.random() < 0.6
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, stream=stream, groups=groups,
                    post=post, pre=rng.random() < 0.8, drop=rng.choice([0.0, 0.0, 0.1, 0.3]),
                    offset=rng.choice([0.0, 1.0]), backward=rng.random() < 0.7)
    if op == "dropout":
        cols = _log_int(rng, 33, 16384)
        if rng.random() < 0.7:
            cols = (cols + 7) // 8 * 8
        return dict(op=op, rows=_log_int(rng, 1, min(65536, 92_000_000 // (cols * half))),
                    cols=cols, dtype=dtype, drop=rng.choice([0.05, 0.1, 0.2, 0.5]),
                    strided=rng.random() < 0.3)
    experts = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 384])
    k = rng.choice([1, 2, 4, 6, 8])
    return dict(op=op, tokens=_log_int(rng, 1, min(65536, 16_000_000 // (experts * half))),
                experts=experts, k=k, dtype=dtype, renormalise=rng.random() < 0.5,
                hidden=rng.choice([0.0, 0.0, 0.1]), backward=rng.random() < 0.7)


# ---- inputs ------------------------------------------------------------------------

def _randn(gen, *shape, dtype=torch.float32, sigma=1.0):
    return (torch.randn(*shape, device=DEV, generator=gen) * sigma).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))
    dt = TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] != "route":
        # the generator's key, the position of this call and the step, which lives on the device
        s["seed"] = int(seed) * 0x9E3779B1 % (1 << 63)
        s["call"] = 11
        s["counter"] = torch.full((1,), int(seed) % 1000 * 64, dtype=torch.int64, device=DEV)
    if case["op"] == "join":
        return _prepare_join(case, s, gen, dt)
    if case["op"] == "dropout":
        r, c = case["rows"], case["cols"]
        pad = 24 if case["strided"] else 0

        def matrix(sigma):
            return _randn(gen, r, c + pad, dtype=dt, sigma=sigma)[:, :c]

        s["x"], s["dout"] = matrix(1.5), matrix(1e-2)
        s["out"], s["dx"] = matrix(0.0), matrix(0.0)
        return s
    t, e = case["tokens"], case["experts"]
    # some experts are liked more than others, as before a balance loss has done its work
    s["logits"] = (_randn(gen, t, e, sigma=1.5) + _randn(gen, 1, e, sigma=0.7)).to(dt)
    s["counted"] = None
    if case["hidden"]:
        s["counted"] = torch.rand(t, device=DEV, generator=gen) >= case["hidden"]
    s["dweights"] = _randn(gen, t, case["k"], sigma=1e-2)
    # the loss scale of mixed precision
    s["grad_loss"] = torch.full((1,), 65536.0 if case["dtype"] == "f16" else 1.0, device=DEV)
    s["dlogits"] = torch.empty_like(s["logits"])
    return s


def _prepare_join(case, s, gen, dt):
    r, c, st = case["rows"], case["cols"], TYPES[case["stream"]]
    # a few channels of the stream are far larger than the others, in every row
    wide = 1 + 15 * (torch.rand(c, device=DEV, generator=gen) < 0.01)
    s["residual"] = (_randn(gen, r, c, sigma=2.0) * wide).to(st)
    s["branch"] = (_randn(gen, r, c) * torch.exp(0.5 * _randn(gen, r, 1))).to(dt)
    for name, on in (("post_weight", case["post"]), ("pre_weight", case["pre"])):
        s[name] = (1 - case["offset"] + _randn(gen, c, sigma=0.2)).to(dt) if on else None
    s["gate"] = None
    if case["groups"]:
        s["gate"] = (0.5 + _randn(gen, case["groups"], c, sigma=0.3)).to(dt)
    s["residual_scale"], s["branch_scale"] = 0.9, 0.7
    s["out"] = torch.empty(r, c, device=DEV, dtype=st)
    s["normed"] = torch.empty(r, c, device=DEV, dtype=dt) if case["pre"] else None
    if case["backward"]:
        s["dout"] = _randn(gen, r, c, dtype=st, sigma=1e-2)
        s["dnormed"] = _randn(gen, r, c, dtype=dt, sigma=1e-2) if case["pre"] else None
        s["dresidual"] = torch.empty(r, c, device=DEV, dtype=st)
        s["dbranch"] = torch.empty(r, c, device=DEV, dtype=dt)
        for name in ("post_weight", "pre_weight", "gate"):
            s["d" + name] = None if s[name] is None else torch.empty_like(s[name])
    return s


# ---- one pass ------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


JOIN_GRADIENTS = ("dresidual", "dbranch", "dpost_weight", "dpre_weight", "dgate")


def _join_outputs(s):
    names = ("out", "normed") + (JOIN_GRADIENTS if s["backward"] else ())
    return {name: s[name] for name in names if s[name] is not None}


def _run_own(s):
    import amsgrad_optimizer_step_gb300 as fa
    if s["op"] == "route":
        if "route" not in s:
            s["route"] = fa.route_buffers(s["tokens"], s["experts"], s["k"], DEV,
                                          loss=s["backward"])
        b = s["route"]
        fa.fa_route(s["logits"], b, counted=s["counted"], renormalise=s["renormalise"],
                    balance_coef=BALANCE, z_coef=ZLOSS)
        out = {"chosen": b.chosen, "weights": b.weights}
        if s["backward"]:
            fa.fa_route_gradient(s["logits"], b, s["dlogits"], dweights=s["dweights"],
                                 grad_loss=s["grad_loss"], counted=s["counted"],
                                 renormalise=s["renormalise"], balance_coef=BALANCE, z_coef=ZLOSS)
            out.update(counts=b.counts, loss=b.loss, balance=b.balance, z=b.z,
                       mean_prob=b.mean_prob, dlogits=s["dlogits"])
        return out
    drop = fa.Dropout(s["drop"], s["seed"], s["call"], s["counter"])
    if s["op"] == "dropout":
        fa.fa_dropout(s["x"], s["out"], drop)
        fa.fa_dropout(s["dout"], s["dx"], drop)
        return {"out": s["out"], "dx": s["dx"]}
    if "join" not in s:
        s["join"] = fa.Join(s["post"], s["residual_scale"], s["branch_scale"], EPS, s["offset"],
                            drop if s["drop"] else None)
        s["rstd"] = torch.empty(2, s["rows"], device=DEV)
        if s["backward"]:
            s["scratch"] = fa.join_scratch(s["rows"], s["cols"], s["groups"], DEV)
    # a validation or generation pass keeps nothing for a gradient
    post_rstd = s["rstd"][0] if s["post"] and s["backward"] else None
    pre_rstd = s["rstd"][1] if s["pre"] and s["backward"] else None
    fa.fa_block_join(s["join"], s["residual"], s["branch"], s["out"], s["normed"], post_rstd,
                     pre_rstd, s["post_weight"], s["pre_weight"], s["gate"])
    if s["backward"]:
        fa.fa_block_join_gradient(s["join"], s["out"], s["branch"], s["dout"], s["dnormed"],
                                  s["dresidual"], s["dbranch"], s["scratch"], post_rstd, pre_rstd,
                                  s["post_weight"], s["pre_weight"], s["gate"],
                                  s["dpost_weight"], s["dpre_weight"], s["dgate"])
    return _join_outputs(s)


def _run_plain(s):
    if s["op"] == "route":
        return _route_plain(s)
    if s["op"] == "dropout":
        m = _factors(s)
        zero = torch.zeros((), device=DEV)
        return {name: torch.where(m > 0, s[x].float() * m, zero).to(s[x].dtype)
                for name, x in (("out", "x"), ("dx", "dout"))}
    return _join_plain(s)


def _factors(s):
    """What dropout multiplies each element by: 0, or the inverse of the share that is kept.
    Each eight columns of a row take the eight 16-bit parts of one Philox 4x32-10 block."""
    blocks = -(-s["cols"] // 8)
    low = 0xFFFFFFFF
    at = torch.arange(s["rows"] * blocks, device=DEV)
    call = (s["counter"] + s["call"]).expand_as(at)
    c0, c1, c2, c3 = at & low, (at >> 32) & low, call & low, (call >> 32) & low
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64 bits, the top one in the sign
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(s["rows"], 8 * blocks)
    dropped = round(s["drop"] * LEVELS)
    kept = bits[:, :s["cols"]] >= dropped
    return kept.float() * (LEVELS / (LEVELS - dropped))


def _mean(x):
    return x.sum(1, keepdim=True) / x.shape[1]


def _join_plain(s):
    dt, st = TYPES[s["dtype"]], TYPES[s["stream"]]
    y, alpha, beta = s["branch"].float(), s["residual_scale"], s["branch_scale"]
    one = torch.ones(1, s["cols"], device=DEV)
    m = _factors(s) if s["drop"] else one
    g = one
    if s["groups"]:
        g = s["gate"].float().repeat_interleave(s["rows"] // s["groups"], 0)
    yh, b = y, y
    if s["post"]:
        y_rstd = 1 / torch.sqrt(_mean(y * y) + EPS)
        w_post = s["post_weight"].float() + s["offset"]
        yh = y * y_rstd
        b = yh * w_post
    # the next norm is of the stream as it is stored
    out = (alpha * s["residual"].float() + beta * g * m * b).to(st)
    result = {"out": out}
    x = out.float()
    if s["pre"]:
        x_rstd = 1 / torch.sqrt(_mean(x * x) + EPS)
        w_pre = s["pre_weight"].float() + s["offset"]
        xh = x * x_rstd
        result["normed"] = (xh * w_pre).to(dt)
    if not s["backward"]:
        return result
    total = s["dout"].float()
    if s["pre"]:
        dn = s["dnormed"].float()
        d = dn * w_pre
        total = total + x_rstd * (d - xh * _mean(d * xh))
        result["dpre_weight"] = (dn * xh).sum(0).to(dt)
    result["dresidual"] = (alpha * total).to(st)
    if s["groups"]:
        d = beta * m * b * total
        result["dgate"] = d.reshape(s["groups"], -1, s["cols"]).sum(1).to(dt)
    db = beta * g * m * total
    if s["post"]:
        result["dpost_weight"] = (db * yh).sum(0).to(dt)
        db = db * w_post
        db = y_rstd * (db - yh * _mean(db * yh))
    result["dbranch"] = db.to(dt)
    return result


def _route_plain(s):
    e, k = s["experts"], s["k"]
    x = s["logits"].float()
    on = torch.ones(s["tokens"], 1, device=DEV) if s["counted"] is None else \
        s["counted"].float()[:, None]
    chosen = torch.sort(x, stable=True, dim=1, descending=True)[1][:, :k]  # equal: the lower index
    top = x.amax(1, keepdim=True)
    ex = torch.exp(x - top)
    total = ex.sum(1, keepdim=True)
    p = ex / total
    picked = ex.gather(1, chosen)
    w = picked / (picked.sum(1, keepdim=True) if s["renormalise"] else total) * on
    out = {"chosen": torch.where(on > 0, chosen, torch.full_like(chosen, -1)).int(), "weights": w}
    if not s["backward"]:
        return out
    lse = top + torch.log(total)
    counts = torch.zeros(e, device=DEV, dtype=torch.int64)
    counts.index_add_(0, chosen.reshape(-1), on.long().expand(-1, k).reshape(-1))
    n = on.sum().clamp(min=1.0)
    f = counts.float() / (n * k)
    mean_prob = (p * on).sum(0) / n
    balance = e * (f * mean_prob).sum().reshape(1)
    z = ((lse * lse) * on).sum().reshape(1) / n
    dw = s["dweights"] * w
    back = dw.sum(1, keepdim=True)
    d = p * (f - (p * f).sum(1, keepdim=True)) * (BALANCE * e / n) + p * lse * (2 * ZLOSS / n)
    d = d * s["grad_loss"]
    if s["renormalise"]:
        d.scatter_add_(1, chosen, dw - w * back)
    else:
        d = (d - p * back).scatter_add_(1, chosen, dw)
    out.update(counts=counts.int(), loss=BALANCE * balance + ZLOSS * z, balance=balance, z=z,
               mean_prob=mean_prob, dlogits=(d * on).to(TYPES[s["dtype"]]))
    return out


# ---- the definitions in FP64 -----------------------------------------------------------

def _exact_factors(s):
    """The dropout factors in FP64, on the host's 64-bit integers."""
    blocks = -(-s["cols"] // 8)
    u64, low, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    call = (int(s["counter"].item()) + s["call"]) % (1 << 64)
    dropped = round(s["drop"] * LEVELS)
    kept = np.empty((s["rows"] * blocks, 8), dtype=bool)
    step = 1 << 20
    for a in range(0, len(kept), step):
        part = kept[a:a + step]
        at = np.arange(a, a + len(part), dtype=u64)
        x = [at & low, at >> half, np.full_like(at, call & 0xFFFFFFFF), np.full_like(at, call >> 32)]
        key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
        for _ in range(10):
            a0, a2 = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
            x = [(a2 >> half) ^ x[1] ^ u64(key[0]), a2 & low,
                 (a0 >> half) ^ x[3] ^ u64(key[1]), a0 & low]
            key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
        for j in range(8):
            part[:, j] = ((x[j // 2] >> u64(16 * (j % 2))) & u64(0xFFFF)) >= u64(dropped)
    kept = torch.from_numpy(kept.reshape(s["rows"], 8 * blocks)[:, :s["cols"]].copy()).to(DEV)
    return kept.double() * (LEVELS / (LEVELS - dropped))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "dropout":
        m = _exact_factors(s)
        return {"out": s["x"].to(f64) * m, "dx": s["dout"].to(f64) * m}
    if case["op"] == "route":
        return _route_exact(case, s)
    leaves = {name: s[name].to(f64).requires_grad_(case["backward"])
              for name in ("residual", "branch", "post_weight", "pre_weight", "gate")
              if s[name] is not None}

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (w + case["offset"])

    b = leaves["branch"]
    if case["post"]:
        b = norm(b, leaves["post_weight"])
    if case["drop"]:
        b = b * _exact_factors(s)
    if case["groups"]:
        b = (b.unflatten(0, (case["groups"], -1)) * leaves["gate"][:, None]).flatten(0, 1)
    out = s["residual_scale"] * leaves["residual"] + s["branch_scale"] * b
    result = {"out": out.detach()}
    ends, grads = [out], [s["dout"].to(f64) if case["backward"] else None]
    if case["pre"]:
        # of the stored stream; its rounding has the gradient of no rounding
        stored = out + (out.detach().to(TYPES[case["stream"]]).to(f64) - out.detach())
        normed = norm(stored, leaves["pre_weight"])
        result["normed"] = normed.detach()
        ends.append(normed)
        grads.append(s["dnormed"].to(f64) if case["backward"] else None)
    if case["backward"]:
        found = torch.autograd.grad(ends, list(leaves.values()), grads)
        result.update({"d" + name: g for name, g in zip(leaves, found)})
    return result


def _route_exact(case, s):
    x = s["logits"].to(torch.float64).requires_grad_(case["backward"])
    t, e, k = case["tokens"], case["experts"], case["k"]
    on = torch.ones(t, dtype=torch.bool, device=DEV) if s["counted"] is None else s["counted"]
    left, chosen = x.detach().clone(), []
    for _ in range(k):  # the largest, and of equal ones the first
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, torch.arange(e, device=DEV), e).amin(1, keepdim=True)
        left.scatter_(1, at, -math.inf)
        chosen.append(at)
    chosen = torch.cat(chosen, 1)
    p = torch.softmax(x, 1)
    w = p.gather(1, chosen)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    w = w * on[:, None]
    out = {"chosen": torch.where(on[:, None], chosen, -1).int(), "weights": w.detach()}
    if not case["backward"]:
        return out
    counts = torch.bincount(chosen[on].reshape(-1), minlength=e)
    n = max(1, int(on.sum()))
    mean_prob = p[on].sum(0) / n
    balance = e * (counts.double() / (n * k) * mean_prob).sum().reshape(1)
    z = torch.logsumexp(x, 1)[on].square().sum().reshape(1) / n
    loss = BALANCE * balance + ZLOSS * z
    (dx,) = torch.autograd.grad([loss, w], x, [s["grad_loss"].double(), s["dweights"].double()])
    out.update(counts=counts.int(), loss=loss.detach(), balance=balance.detach(), z=z.detach(),
               mean_prob=mean_prob.detach(), dlogits=dx)
    return out


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n * b, "flops": 2 * n}
    if case["op"] == "route":
        t, n = case["tokens"], case["tokens"] * case["experts"]
        read = int(round((1 - case["hidden"]) * n)) * b  # a token that is not counted is not read
        pairs = 8 * t * case["k"]
        if not case["backward"]:
            return {"bytes": read + pairs, "flops": 4 * n}
        return {"bytes": 2 * read + n * b + pairs + pairs // 2, "flops": 14 * n}
    n, sb = case["rows"] * case["cols"], SIZE[case["stream"]]
    rows = (case["post"] + case["pre"] + case["groups"]) * case["cols"] * b  # weights and gate
    total = n * (2 * sb + b + b * case["pre"]) + rows
    if not case["backward"]:
        return {"bytes": total, "flops": 12 * n}
    # the stored stream is read for the second norm's gradient alone
    total += n * (2 * sb + 2 * b + (sb + b) * case["pre"]) + 2 * rows
    return {"bytes": total, "flops": 36 * n}
