"""The autograd forms of the residual blocks' operators, against torch's autograd in 64 bits, and a
routed block that uses them together."""

import math
import os
import sys

import pytest
import torch

import block_reference as B
from conftest import ROOT
from model_reference import DTYPES, U32, UNIT, assert_close
from test_gpu_model_ops import gen, randn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def layers():
    from amsgrad_optimizer_step_gb300 import build
    build.build()
    from amsgrad_optimizer_step_gb300 import layers
    return layers


def close(got, want, terms, what, unit=None):
    """Within two roundings to the type (a result, and the stored stream it follows from) and 200
    FP32 ones of the terms that it is made of."""
    unit = UNIT[got.dtype] if unit is None else unit
    bound = (2 * unit + 200 * U32) * want.abs() + (2 * unit + 200 * U32) * terms
    assert bool(((got.double() - want).abs() <= bound).all()), what


@pytest.mark.parametrize("dt", list(DTYPES))
def test_dropout(layers, dt):
    for shape in ((4, 5, 72), (33,), (3, 0), (0, 8)):
        x = randn(gen(1), *shape, dtype=DTYPES[dt]).requires_grad_()
        y = layers.dropout(x, 0.3, seed=5, offset=9)
        rows, cols = math.prod(shape[:-1]), shape[-1]
        keep = B.kept(rows, cols, 0.3, 5, 9, DEV).view(shape)
        scale = B.keep_scale(0.3)
        want = torch.where(keep, x.detach().double() * scale, 0.0)
        assert_close(y.detach(), want, 2 * U32 * want.abs(), "dropout")
        dy = randn(gen(2), *shape, dtype=DTYPES[dt])
        (dx,) = torch.autograd.grad(y, x, dy)
        want = torch.where(keep, dy.double() * scale, 0.0)
        assert_close(dx, want, 2 * U32 * want.abs(), "gradient")


def test_dropout_of_what_does_not_lie_densely(layers):
    x = randn(gen(3), 6, 40, 7).transpose(1, 2).requires_grad_()
    y = layers.dropout(x, 0.5, 1)
    assert torch.equal(y, layers.dropout(x.detach().contiguous(), 0.5, 1))
    (a,) = torch.autograd.grad(y, x, torch.ones(40, device=DEV).expand(6, 7, 40))
    assert torch.equal(a, B.kept(42, 40, 0.5, 1, 0, DEV).view(6, 7, 40).float() * 2.0)


def test_a_counter_that_moved_on_before_the_backward_pass_is_refused(layers):
    counter = torch.tensor([3], device=DEV)
    x, r, w = randn(gen(4), 6, 40), randn(gen(5), 6, 40), torch.ones(40, device=DEV)
    x.requires_grad_()
    for run in (lambda: layers.dropout(x, 0.5, 1, 2, counter),
                lambda: layers.block_join(r, x, w, pre_norm=False, p=0.5, seed=1, counter=counter)):
        y = run()
        step = int(counter)
        counter.add_(1)
        with pytest.raises(RuntimeError):
            y.sum().backward()
        y = run()
        y.sum().backward()
        counter.add_(1)  # after the backward pass it may
        assert int(counter) == step + 2


@pytest.mark.parametrize("kind", [("f32", "f32", "f32"), ("f16", "f16", "f16"),
                                  ("bf16", "f32", "bf16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("post,gates,pre,p", [
    (True, 3, True, 0.0), (True, 1, True, 0.25), (False, 0, True, 0.25), (True, 0, False, 0.0)])
def test_block_join(layers, kind, post, gates, pre, p):
    dt, st, wt = (DTYPES[k] for k in kind)
    g = gen(6)
    shape = (3, 10, 136)
    r, y = randn(g, *shape, dtype=st), randn(g, *shape, dtype=dt)
    w1 = (1 + randn(g, 136, sigma=0.3)).to(wt) if post else None
    w2 = (1 + randn(g, 136, sigma=0.3)).to(wt) if pre else None
    gate = (0.5 + randn(g, *((136,) if gates == 1 else (gates, 136)), sigma=0.3)).to(wt) \
        if gates else None
    leaves = [t.requires_grad_() for t in (r, y, w1, gate, w2) if t is not None]
    args = dict(post_norm=post, pre_norm=pre, residual_scale=0.9, branch_scale=1.2, eps=1e-5, p=p,
                seed=11, offset=3)
    got = layers.block_join(r, y, w1, gate, w2, **args)
    got = got if pre else (got,)
    assert got[0].dtype == st and got[0].shape == shape

    mask = B.kept(30, 136, p, 11, 3, DEV) if p else None
    d = [t.detach().double().requires_grad_() for t in leaves]
    it = iter(d)
    r64, y64 = next(it), next(it)
    w164 = next(it) if post else None
    gate64 = next(it).reshape(-1, 136) if gates else None
    w264 = next(it) if pre else None
    out, _, _ = B.join(r64.reshape(30, 136), y64.reshape(30, 136), w164, gate64, post, 0.9, 1.2,
                       1e-5, 0.0, mask, B.keep_scale(p) if p else 1.0)
    wants = [out]
    if pre:  # of the stored stream; its rounding has the gradient of no rounding
        stored = out + (got[0].detach().double().view(30, 136) - out.detach())
        wants.append(B.norm(stored, w264, 1e-5, 0.0)[0])
    for x, want in zip(got, wants):
        assert bool(((x.detach().double().view(30, 136) - want).abs() <=
                     (2 * UNIT[x.dtype] + 100 * U32) * (1 + want.abs()) * 4).all())
    dys = [randn(g, *shape, dtype=x.dtype) for x in got]
    grads = torch.autograd.grad(got, leaves, dys)
    exact = torch.autograd.grad(wants, d, [dy.double().view(30, 136) for dy in dys])
    for a, b, leaf in zip(grads, exact, leaves):
        assert a.dtype == leaf.dtype and a.shape == leaf.shape
        # the terms that a gradient is a sum of are of the order of its largest ones
        close(a, b, b.abs().max(), "gradient")


def test_norm(layers):
    for dt, to in (("f32", None), ("bf16", None), ("f32", torch.bfloat16)):
        x = randn(gen(7), 5, 7, 200, dtype=DTYPES[dt]).requires_grad_()
        w = randn(gen(8), 200, sigma=0.2, dtype=to or DTYPES[dt]).requires_grad_()
        y = layers.norm(x, w, 1e-5, 1.0, to)
        assert y.dtype == (to or x.dtype)
        x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
        want = torch.nn.functional.rms_norm(x64, (200,), w64 + 1, 1e-5)
        assert_close(y.detach(), want.detach(), 30 * U32 * want.detach().abs(), "norm")
        dy = randn(gen(9), 5, 7, 200, dtype=y.dtype)
        for a, b in zip(torch.autograd.grad(y, (x, w), dy),
                        torch.autograd.grad(want, (x64, w64), dy.double())):
            close(a, b, b.abs().max(), "norm gradient")
    x = randn(gen(7), 5, 200)
    want = torch.nn.functional.rms_norm(x.double(), (200,), None, 1e-6)
    assert_close(layers.norm(x), want, 30 * U32 * want.abs(), "norm without weights")


def test_a_join_with_some_gradients_only(layers):
    """One result unused, some operands without a gradient, and none at all."""
    g = gen(10)
    r, y, w1, w2 = randn(g, 40, 72), randn(g, 40, 72), torch.ones(72, device=DEV), randn(g, 72)
    y.requires_grad_()
    w2.requires_grad_()
    dy = randn(g, 40, 72)
    for take in (0, 1):
        outs = layers.block_join(r, y, w1, None, w2)
        got = torch.autograd.grad(outs[take], (y, w2), dy, allow_unused=True)
        y64, w64 = y.detach().double().requires_grad_(), w2.detach().double().requires_grad_()
        out = B.join(r, y64, w1, None, True, 1.0, 1.0, 1e-6, 0.0, None, 1.0)[0]
        want = (out, B.norm(out, w64, 1e-6, 0.0)[0])[take]
        exact = torch.autograd.grad(want, (y64, w64), dy.double(), allow_unused=True)
        for a, b in zip(got, exact):
            if b is None:
                assert a is None
            else:
                close(a, b, b.abs().max(), "gradient")
    with torch.no_grad():
        again = layers.block_join(r, y, w1, None, w2)
    assert all(torch.equal(a, b) for a, b in zip(outs, again)) and not again[0].requires_grad


def test_gradients_of_gradients_are_refused(layers):
    x = randn(gen(11), 5, 16).requires_grad_()
    for y in (layers.dropout(x, 0.5, 1), layers.norm(x), layers.block_join(x, x.detach())[1],
              layers.route(x, 2)[1]):
        (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), x)


def test_gradients_that_are_expanded(layers):
    g = gen(12)
    x, w = randn(g, 30, 72).requires_grad_(), torch.ones(72, device=DEV).requires_grad_()
    row = randn(g, 72).expand(30, 72)
    for run in (lambda: layers.dropout(x, 0.5, 1), lambda: layers.norm(x, w),
                lambda: layers.block_join(x, x.detach(), w)[1]):
        inputs = (x,)
        a = torch.autograd.grad(run(), inputs, row)
        b = torch.autograd.grad(run(), inputs, row.contiguous())
        assert torch.equal(a[0], b[0])
    logits = randn(g, 30, 16).requires_grad_()
    one = torch.ones(1, device=DEV)
    a = torch.autograd.grad(layers.route(logits, 4)[1], logits, one.expand(30, 4))
    b = torch.autograd.grad(layers.route(logits, 4)[1], logits, torch.ones(30, 4, device=DEV))
    assert torch.equal(a[0], b[0])


def test_layers_with_nothing(layers):
    w = torch.ones(16, device=DEV, requires_grad=True)
    gate = torch.ones(1, 16, device=DEV, requires_grad=True)
    for shape in ((0, 16), (3, 0, 16)):
        x = torch.empty(shape, device=DEV, requires_grad=True)
        out, normed = layers.block_join(x, x * 1.0, w, gate, w)
        grads = torch.autograd.grad(out.sum() + normed.sum(), (x, w, gate))
        assert grads[0].shape == x.shape and not grads[1].any() and not grads[2].any()
        (g,) = torch.autograd.grad(layers.norm(x, w).sum(), w)
        assert not g.any()
    logits = torch.empty((0, 8), device=DEV, requires_grad=True)
    chosen, weights, loss, counts = layers.route(logits, 2, balance_coef=0.1)
    (g,) = torch.autograd.grad(loss + weights.sum(), logits)
    assert g.shape == (0, 8) and loss.item() == 0 and not counts.any()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_route(layers, dt):
    g = gen(13)
    logits = randn(g, 50, 24, dtype=DTYPES[dt], sigma=1.5).requires_grad_()
    counted = torch.rand(50, device=DEV, generator=g) < 0.8
    chosen, weights, loss, counts = layers.route(logits, 3, counted, False, 2.0, 0.5, 0.1)
    x = logits.detach().double().requires_grad_()
    want = B.route(x, 3, counted, False, 2.0, 0.5, 0.1)
    assert torch.equal(chosen.long(), want["chosen"]) and torch.equal(counts.long(), want["counts"])
    assert not chosen.requires_grad and not counts.requires_grad
    dw = randn(g, 50, 3)
    for got, ref in (((weights * dw).sum() + 7.0 * loss,
                      (want["weights"] * dw.double()).sum() + 7.0 * want["loss"]),
                     (loss * 7.0, want["loss"] * 7.0),
                     ((weights * dw).sum(), (want["weights"] * dw.double()).sum())):
        (a,) = torch.autograd.grad(got, logits, retain_graph=True)
        (b,) = torch.autograd.grad(ref, x, retain_graph=True)
        close(a, b, b.abs().max(), "route gradient")


def test_a_routed_block(layers):
    """Norm, router, gated experts, join with a norm behind and the next one before, dropout and the
    losses, forward and backward, as a model calls them, in FP32 against the same in 64 bits."""
    g = gen(14)
    tokens, dim, hidden, experts, k = 60, 48, 64, 6, 2
    x = randn(g, tokens, dim)
    names = dict(w0=(dim,), wr=(experts, dim), up=(experts, 2 * hidden, dim),
                 down=(experts, dim, hidden), w1=(dim,), gate=(dim,), w2=(dim,))
    params = {}
    for name, shape in names.items():
        sigma = 0.3 if len(shape) == 1 else shape[-1] ** -0.5
        params[name] = randn(g, *shape, sigma=sigma) + (1.0 if len(shape) == 1 else 0.0)
    counted = torch.arange(tokens, device=DEV) < 55
    mask = B.kept(tokens, dim, 0.1, 77, 2, DEV)
    dout, dnormed = randn(g, tokens, dim), randn(g, tokens, dim)

    def experts_of(h, chosen, weights, up, down):
        y = torch.zeros_like(h)
        for e in range(experts):
            t, j = torch.nonzero(chosen == e, as_tuple=True)
            gate, value = (h[t] @ up[e].t()).chunk(2, 1)
            y = y.index_add(0, t, weights[t, j, None] *
                            ((torch.nn.functional.silu(gate) * value) @ down[e].t()))
        return y

    p = {n: t.clone().requires_grad_() for n, t in params.items()}
    h = layers.norm(x, p["w0"])
    chosen, weights, aux, counts = layers.route(h @ p["wr"].t(), k, counted, balance_coef=0.1,
                                                z_coef=0.01)
    out, normed = layers.block_join(x, experts_of(h, chosen.long(), weights, p["up"], p["down"]),
                                    p["w1"], p["gate"], p["w2"], p=0.1, seed=77, offset=2)
    total = (out * dout).sum() + (normed * dnormed).sum() + 50.0 * aux
    grads = torch.autograd.grad(total, list(p.values()))

    q = {n: t.double().requires_grad_() for n, t in params.items()}
    h = B.norm(x, q["w0"], 1e-6, 0.0)[0]
    r = B.route(h @ q["wr"].t(), k, counted, True, 1.0, 0.1, 0.01)
    assert torch.equal(r["chosen"], chosen.long()) and torch.equal(r["counts"], counts.long())
    y = experts_of(h, r["chosen"], r["weights"], q["up"], q["down"])
    out64 = B.join(x, y, q["w1"], q["gate"][None], True, 1.0, 1.0, 1e-6, 0.0, mask,
                   B.keep_scale(0.1))[0]
    normed64 = B.norm(out64, q["w2"], 1e-6, 0.0)[0]
    want = (out64 * dout.double()).sum() + (normed64 * dnormed.double()).sum() + 50.0 * r["loss"]
    for name, a, b in zip(p, grads, torch.autograd.grad(want, list(q.values()))):
        # products of up to 64 terms on both sides of every operator, of the order of the largest
        assert bool(((a.double() - b).abs() <= 2000 * U32 * b.abs().max()).all()), name


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import preference_training
    finally:
        sys.path.pop(0)
    return preference_training


@pytest.mark.parametrize("dt", list(DTYPES))
def test_the_example_trains_with_joined_blocks(example, dt):
    out = example.train(steps=6, dtype=dt, joins=True, log=lambda *_: None)
    assert all(math.isfinite(x) for x in out["losses"]) and out["skipped"] <= 2


def test_the_examples_gradients(layers, example):
    """Along its own gradient a loss changes by the gradient's square: central differences in FP32,
    dropout on.  The MLPs' gradients come from inputs kept in 8 bits, each off by 1/254 of its
    block's largest at most; a hundredth of the whole is a generous bound on their sum."""
    model = example.SmallModel(97, 48, 64, 2, torch.float32, DEV, joins=True, dropout=0.2)
    ids = torch.randint(0, 97, (200,), device=DEV, generator=gen(15))

    def loss():
        model.calls = 0  # the same elements are dropped
        return layers.token_logprobs(model(ids), ids).double().mean()

    params = list(model.parameters())
    grads = torch.autograd.grad(loss(), params)
    assert all(bool(g.any()) for g in grads)
    square = sum(g.double().square().sum() for g in grads).item()
    step = 1e-2 / math.sqrt(square)
    ends = []
    for sign in (1, -1):
        with torch.no_grad():
            for w, g in zip(params, grads):
                w.add_(g, alpha=sign * step)
        ends.append(loss().item())
        with torch.no_grad():
            for w, g in zip(params, grads):
                w.sub_(g, alpha=sign * step)
    change = (ends[0] - ends[1]) / (2 * step)
    assert abs(change - square) < 0.01 * square
