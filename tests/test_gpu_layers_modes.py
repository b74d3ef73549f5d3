"""The autograd layer in other modes than a plain training pass."""

import pytest
import torch

import model_reference as R
from model_reference import DTYPES, UNIT

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def layers():
    from amsgrad_optimizer_step_gb300 import build
    build.build()
    from amsgrad_optimizer_step_gb300 import layers
    return layers


def randn(seed, *shape, dtype=torch.float32, sigma=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * sigma).to(dtype)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("gate_up_dt", ["same", "f32"])
def test_gated_down_under_autocast(layers, dt, gate_up_dt):
    """FP32 weights, 16-bit products, the backward pass outside the autocast region.  A product
    rounds both factors and itself to 16 bits, and may join parts of its sum in 16 bits: four
    units of the terms' magnitudes and two of the result."""
    d = DTYPES[dt]
    u = UNIT[d]
    gu = randn(1, 3, 5, 400, dtype=d if gate_up_dt == "same" else torch.float32).requires_grad_()
    w = randn(2, 24, 200, sigma=0.1).requires_grad_()
    with torch.autocast("cuda", dtype=d):
        y = layers.gated_down(gu, w)
    assert y.dtype == d and y.shape == (3, 5, 24)
    dy = randn(3, 3, 5, 24, dtype=d)
    y.backward(dy)
    assert gu.grad.dtype == gu.dtype and w.grad.dtype == torch.float32

    flat, w64, d64 = gu.detach().reshape(15, 400), w.detach().double(), dy.reshape(15, 24).double()
    h = R.act(flat[:, :200].double(), "silu")[0] * flat[:, 200:].double()
    want = h @ w64.t()
    bound = 4 * u * (h.abs() @ w64.abs().t()) + 2 * u * want.abs()
    assert bool(((y.detach().reshape(15, 24).double() - want).abs() <= bound).all())
    gq, uq = (R.stored(*R.quantise(flat[:, k:k + 200]), 200).double() for k in (0, 200))
    a, da = R.act(gq, "silu")
    dh, dh_mag = d64 @ w64, d64.abs() @ w64.abs()
    for k, factor in ((0, uq * da), (200, a)):
        got = gu.grad.reshape(15, 400)[:, k:k + 200].double()
        want = dh * factor
        bound = (4 * u * dh_mag + 2 * u * dh.abs()) * factor.abs() * (1 + u) + 2 * u * want.abs()
        bound = bound + R.SUBNORMAL[d]
        assert bool(((got - want).abs() <= bound).all())
    hq = a * uq
    want = d64.t() @ hq
    bound = 4 * u * (d64.abs().t() @ hq.abs()) + 2 * u * want.abs()
    assert bool(((w.grad.double() - want).abs() <= bound).all())


def test_gated_down_with_one_gradient_under_autocast(layers):
    gu, w = randn(4, 7, 64), randn(5, 8, 32)
    for x in (gu, w):
        x.requires_grad_()
        with torch.autocast("cuda", dtype=torch.bfloat16):
            y = layers.gated_down(gu, w)
        y.float().sum().backward()
        assert bool(torch.isfinite(x.grad).all())
        x.requires_grad_(False)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_checkpoint_without_gradients(layers, monkeypatch, mode):
    """Parameters that would have a gradient, in a pass that has none: nothing is kept, and the
    results are the training pass's bit for bit."""
    gu = randn(6, 9, 2 * 130).requires_grad_()
    w = randn(7, 24, 130).requires_grad_()
    want = layers.gated_activation(gu).detach(), layers.gated_down(gu, w).detach()

    def refuse(*args):
        raise AssertionError("a checkpoint is made")
    monkeypatch.setattr(layers.ops, "checkpoint_buffer", refuse)
    with mode():
        got = layers.gated_activation(gu), layers.gated_down(gu, w)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_a_padding_id_is_an_id_as_it_stands(layers):
    """padding_idx is compared with the ids: a negative one is outside the table like any other
    negative id, and no row loses its gradient for it."""
    w = randn(8, 5, 8).requires_grad_()
    ids = torch.tensor([4, -1, 0, 4], device=DEV)
    (got,) = torch.autograd.grad(layers.embedding(ids, w, padding_idx=-1).sum(), w)
    assert got.sum(1).tolist() == [8.0, 0.0, 0.0, 0.0, 16.0]
    (got,) = torch.autograd.grad(layers.embedding(ids, w, padding_idx=4).sum(), w)
    assert got.sum(1).tolist() == [8.0, 0.0, 0.0, 0.0, 0.0]
