"""The autograd layer over the model-side operators, against torch's autograd in 64 bits, and
the example that trains with all of them."""

import math
import os
import sys

import pytest
import torch

import model_reference as R
from conftest import ROOT
from model_reference import DTYPES, U32, assert_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from amsgrad_optimizer_step_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def layers():
    from amsgrad_optimizer_step_gb300 import layers
    return layers


def randn(seed, *shape, dtype=torch.float32, sigma=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * sigma).to(dtype)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_embedding(layers, dt):
    """Batched ids, a scale, a padding id and ids outside the table; a strided gradient."""
    w = randn(1, 40, 24, dtype=DTYPES[dt]).requires_grad_()
    g = torch.Generator(device=DEV).manual_seed(2)
    ids = torch.randint(-2, 42, (5, 7), device=DEV, generator=g)
    y = layers.embedding(ids, w, scale=3.0, padding_idx=4)
    want = R.lookup(ids.reshape(-1), w.detach(), 3.0).view(5, 7, 24)
    assert_close(y, want, 2 * U32 * want.abs(), "embedding")
    dy = randn(3, 5, 24, 7, dtype=DTYPES[dt]).transpose(1, 2)
    y.backward(dy)
    grad, mag, count = R.embedding_gradient(ids.reshape(-1), dy.reshape(-1, 24), 40, 3.0, 4)
    assert_close(w.grad, grad, (count[:, None] + 2) * U32 * mag, "embedding gradient")


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_layers(layers, kind):
    """gated_activation and gated_down: the gradients are those at the 8-bit values of gate and
    up, which is what the definition says; FP32, so that matrix products round alike."""
    gu = randn(4, 3, 5, 2 * 200).requires_grad_()
    w = randn(5, 24, 200, sigma=0.1).requires_grad_()
    flat = gu.detach().reshape(15, 400)
    stored = [R.stored(*R.quantise(flat[:, k * 200:(k + 1) * 200]), 200).double() for k in (0, 1)]
    g64, u64 = (s.requires_grad_() for s in stored)
    dh = randn(6, 3, 5, 200)
    h = layers.gated_activation(gu, kind)
    (da,) = torch.autograd.grad(h, gu, dh)
    h64 = R.act(g64, kind)[0] * u64
    dg, du = torch.autograd.grad(h64, (g64, u64), dh.reshape(15, 200).double(), retain_graph=True)
    want = torch.cat([dg, du], 1).view(3, 5, 400)
    assert bool(((da.double() - want).abs() <= 60 * U32 * (1 + want.abs())).all())
    y = layers.gated_down(gu, w, kind)
    dy = randn(7, 3, 5, 24)
    y.backward(dy)
    w64 = w.detach().double().requires_grad_()
    exact = R.act(flat[:, :200].double(), kind)[0] * flat[:, 200:].double() @ w64.detach().t()
    # products of 200 (forward) or 24 terms; TF32 is off by default
    assert bool(((y.reshape(15, 24).double() - exact).abs() <= 400 * U32 * (1 + exact.abs())).all())
    y64 = (R.act(g64, kind)[0] * u64) @ w64.t()
    dg, du, dw = torch.autograd.grad(y64, (g64, u64, w64), dy.reshape(15, 24).double())
    want = torch.cat([dg, du], 1).view(3, 5, 400)
    assert bool(((gu.grad.double() - want).abs() <= 100 * U32 * (1 + want.abs())).all())
    assert bool(((w.grad.double() - dw).abs() <= 100 * U32 * (1 + dw.abs())).all())


def test_gradients_that_are_expanded(layers):
    """Gradients of sums and means come as one row, or one element, expanded."""
    w = randn(20, 40, 24).requires_grad_()
    ids = torch.arange(30, device=DEV) % 7
    c = randn(21, 24)
    (dw,) = torch.autograd.grad(layers.embedding(ids, w).sum(0), w, c)
    count = torch.bincount(ids, minlength=40)[:, None]
    assert_close(dw, count.double() * c.double(), 31 * U32 * count * c.abs(), "embedding")
    gu = randn(22, 15, 2 * 130).requires_grad_()
    down = randn(23, 24, 130).requires_grad_()
    rows = randn(24, 130).expand(15, 130)
    ones = randn(25, 24).expand(15, 24)
    for run, d, inputs in ((lambda: layers.gated_activation(gu), rows, (gu,)),
                           (lambda: layers.gated_down(gu, down), ones, (gu, down))):
        for x, y in zip(torch.autograd.grad(run(), inputs, d),
                        torch.autograd.grad(run(), inputs, d.contiguous())):
            assert torch.equal(x, y)
    logits = randn(26, 9, 50).requires_grad_()
    labels = torch.arange(9, device=DEV)
    one = torch.tensor([0.25], device=DEV)
    x, y = (torch.autograd.grad(layers.token_logprobs(logits, labels), logits, d)[0]
            for d in (one.expand(9), one.expand(9).contiguous()))
    assert torch.equal(x, y)


def test_gradients_of_gradients_are_refused(layers):
    """The backward passes are not differentiable: asked for twice, they say so."""
    w = randn(30, 11, 8).requires_grad_()
    gu = randn(31, 5, 16).requires_grad_()
    logits = randn(32, 5, 11).requires_grad_()
    ids = torch.arange(5, device=DEV)
    flat = torch.zeros(5, device=DEV)
    for y, x in ((layers.embedding(ids, w).square().sum(), w),
                 (layers.gated_activation(gu).square().sum(), gu),
                 (layers.gated_down(gu, w).square().sum(), gu),
                 (layers.token_logprobs(logits, ids).square().sum(), logits),
                 (layers.policy_loss(logits, ids, flat, flat + 1.0)[0].square(), logits),
                 (layers.preference_loss(logits, ids, torch.tensor([0, 3, 5], device=DEV), flat,
                                         )[0].square(), logits)):
        (g,) = torch.autograd.grad(y, x, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), x)


def test_a_checkpoint_is_given_back_after_the_backward_pass(layers):
    gu = randn(33, 512, 2 * 2048).requires_grad_()
    h = layers.gated_activation(gu)
    dh, gu.grad = torch.ones_like(h), torch.zeros_like(gu)
    before = torch.cuda.memory_allocated()
    h.backward(dh)
    freed = before - torch.cuda.memory_allocated()
    assert freed >= 2 * 512 * 2048  # the codes, though h and its graph live on
    with pytest.raises(RuntimeError):
        h.backward(dh)


def test_layers_with_nothing(layers):
    w = randn(34, 6, 8).requires_grad_()
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    (g,) = torch.autograd.grad(layers.embedding(none, w).sum(), w)
    assert torch.equal(g, torch.zeros_like(g))
    for shape in ((0, 16), (3, 0, 16), (3, 0)):
        gu = torch.empty(shape, device=DEV, requires_grad=True)
        h = layers.gated_activation(gu)
        assert h.shape == (*shape[:-1], shape[-1] // 2)
        (g,) = torch.autograd.grad(h.sum(), gu)
        assert g.shape == gu.shape
    logits = torch.empty((0, 7), device=DEV, requires_grad=True)
    (g,) = torch.autograd.grad(layers.token_logprobs(logits, none).sum(), logits)
    assert g.shape == (0, 7)


def test_gated_down_keeps_eight_bits(layers):
    """What lives from the forward to the backward pass of gated_down: two bytes a column and a
    scale for 128 of them, for gate and up together, not their six bytes and the activation."""
    rows, cols = 4096, 2048
    w = randn(8, 64, cols, dtype=torch.bfloat16, sigma=0.02).requires_grad_()
    x = randn(9, rows, 64, dtype=torch.bfloat16)
    up = randn(10, 2 * cols, 64, dtype=torch.bfloat16, sigma=0.1).requires_grad_()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = layers.gated_down(x @ up.t(), w)
    kept = torch.cuda.memory_allocated() - before - y.numel() * 2
    assert kept <= 1.05 * rows * cols * (2 + 8 / 128)
    y.sum().backward()
    assert bool(torch.isfinite(up.grad).all())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_loss_layers(layers, dt):
    """Losses and gradients against autograd in 64 bits, through an upstream factor."""
    logits = randn(11, 30, 130, dtype=DTYPES[dt], sigma=2.0).requires_grad_()
    g = torch.Generator(device=DEV).manual_seed(12)
    labels = torch.randint(0, 130, (30,), device=DEV, generator=g)
    labels[::5] = -100
    ok = labels >= 0
    x = logits.detach().double().requires_grad_()
    logp = torch.log_softmax(0.8 * x, 1).gather(1, labels.clamp(min=0)[:, None])[:, 0]
    logp = logp.masked_fill(~ok, 0.0)
    unit = R.UNIT[DTYPES[dt]]

    def close(got, want, what):
        scale = want.abs().max()
        assert bool(((got.double() - want).abs() <= (unit + 200 * U32) * want.abs() +
                     200 * U32 * scale).all()), what

    w = randn(13, 30)
    got = layers.token_logprobs(logits, labels, 0.8)
    close(got, logp.detach(), "logp")
    (grad,) = torch.autograd.grad(got, logits, w)
    close(grad, torch.autograd.grad(logp, x, w.double(), retain_graph=True)[0], "logp gradient")

    off = torch.tensor([0, 7, 15, 20, 30], device=DEV)
    ref = (logp.detach() + randn(14, 30) * 0.5).float()
    loss, rewards = layers.preference_loss(logits, labels, off, ref, 0.3, 0.1, True, 0.8)
    ratio = (logp - ref.double()).masked_fill(~ok, 0.0)
    means = torch.stack([ratio[a:b].sum() / ok[a:b].sum() for a, b in
                         zip(off[:-1].tolist(), off[1:].tolist())])
    z = 0.3 * (means[0::2] - means[1::2])
    want = (0.9 * R.softplus(-z) + 0.1 * R.softplus(z)).mean()
    assert abs(loss.item() - want.item()) <= 100 * U32 * (1 + want.item())
    (grad,) = torch.autograd.grad(loss * 7.0, logits)
    close(grad, torch.autograd.grad(want * 7.0, x, retain_graph=True)[0], "preference gradient")
    assert not rewards.requires_grad

    old = (logp.detach() + randn(15, 30) * 0.05).float()
    adv = randn(16, 30)
    args = (labels, old, adv, ref, None, 0.2, 0.28, 0.1, 0.0, 0.8)
    loss, stats = layers.policy_loss(logits, *args)
    r = torch.exp(logp - old.double())
    d = ref.double() - logp
    per = -torch.minimum(r * adv, r.clamp(0.8, 1.28) * adv) + 0.1 * (torch.exp(d) - d - 1)
    want = per.masked_fill(~ok, 0.0).sum() / ok.sum()
    assert abs(loss.item() - want.item()) <= 200 * U32 * (1 + abs(want.item()))
    assert stats[3].item() == int(ok.sum())
    (grad,) = torch.autograd.grad(loss * 3.0, logits)
    exact = torch.autograd.grad(want * 3.0, x)[0]
    close(grad, exact, "policy gradient")
    summary, dlogits = layers.policy_step(logits, *args, loss_scale=3.0)
    close(dlogits, exact, "policy step gradient")
    assert torch.equal(summary, stats)


def test_a_nonfinite_activation_skips_the_step(layers):
    """An infinity in a gate makes the MLP's gradients NaN through the checkpoint, and the
    optimizer's statistics skip the step."""
    from amsgrad_optimizer_step_gb300.optim import FusedAdamW, GradScaler
    w = torch.nn.Parameter(randn(17, 8, 256, sigma=0.1))
    up = torch.nn.Parameter(randn(18, 512, 16, sigma=0.1))
    opt, scaler = FusedAdamW([w, up], lr=1e-2), GradScaler(init_scale=1.0)
    x = randn(19, 10, 16)
    for bad in (False, True):
        opt.zero_grad()
        gu = x @ up.t()
        if bad:
            gu = gu + torch.where(torch.arange(512, device=DEV) == 3, math.inf, 0.0)
        before = w.detach().clone()
        layers.gated_down(gu, w).sum().backward()
        scaler.step(opt)
        assert opt.last_report["skipped"] == bad
        assert torch.equal(before, w.detach()) == bad


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_example_learns(dt):
    """The example: the preference loss falls from ln 2, and the policy comes to repeat."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import preference_training
    finally:
        sys.path.pop(0)
    out = preference_training.train(steps=30, dtype=dt, log=lambda *_: None)
    assert abs(out["losses"][0] - math.log(2)) < 0.05
    assert sum(out["losses"][-5:]) / 5 < 0.5 * out["losses"][0]
    assert sum(out["rewards"][-5:]) / 5 > 3 * max(out["rewards"][0], 0.01)
    assert out["skipped"] <= 2
