"""Values at the ends of the types' range through the model-side operators."""

import math

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import model_reference as R
import test_gpu_model_ops as M
from model_reference import DTYPES, U32
from test_gpu_model_ops import DEV, INF, NAN, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from amsgrad_optimizer_step_gb300 import build
    build.build()


# ---- gated activation -----------------------------------------------------------------

@pytest.mark.parametrize("dt,top", [("f32", 1e19), ("f32", 2e19), ("f32", 1e30), ("f32", 3e38),
                                    ("bf16", 1e19), ("bf16", 2e19), ("bf16", 1e30),
                                    ("bf16", 3.38e38), ("f16", 6e4)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gates_whose_square_overflows(dt, top, kind):
    """Saturated gates: act is the gate or zero and its slope one or zero, up to a few
    roundings, however large the gate."""
    d = DTYPES[dt]
    g = gen(1)
    gate = randn(g, 6, 256, dtype=d)
    gate[:, :128] = top
    gate[:, 1:128:2] = -top
    up = (0.25 + 0.5 * torch.rand(6, 256, device=DEV, generator=g)).to(d)
    dh = randn(g, 6, 256, dtype=d, sigma=0.1)
    h, dg, du, again = (torch.full_like(gate, NAN) for _ in range(4))
    ck = fa.checkpoint_buffer(6, 256, DEV)
    fa.fa_gated_forward(gate, up, h, ck, kind)
    fa.fa_gated_backward(ck, dh, dg, du, again, kind)
    gq, uq = (x.double() for x in ck.values())
    a = gq[:, :128].clamp(min=0)
    on = (gq[:, :128] > 0).double()
    u, x = uq[:, :128], dh[:, :128].double()
    for got, want in ((h, gate[:, :128].double().clamp(min=0) * up[:, :128].double()),
                      (again, a * u), (dg, x * u * on), (du, x * a)):
        R.assert_close(got[:, :128], want, 8 * U32 * want.abs(), kind)
    assert all(bool(torch.isfinite(t).all()) for t in (h, dg, du, again))


@pytest.mark.parametrize("kind,bound", [("silu", 1.1e-36), ("gelu_tanh", 1.3e-37)])
def test_the_range_where_the_activation_comes_out_as_zero(kind, bound):
    """The sigmoid's values below 2^-126 count as zero.  |act| is the gate's magnitude times
    that at most: 89 for silu (past ln 2^128 the value itself is smaller), 11 for the tanh form."""
    gate = torch.linspace(-130.0, 0.0, 128 * 64, device=DEV).view(64, 128)
    one = torch.ones_like(gate)
    h = torch.empty_like(gate)
    fa.fa_gated_forward(gate, one, h, None, kind)
    want = R.act(gate.double(), kind)[0]
    terms = M.act_terms(gate.double(), kind) * want.abs()
    assert bool(((h.double() - want).abs() <= bound + terms).all())


# ---- policy loss ------------------------------------------------------------------------

def overflowing(vocab, dtype="f32"):
    """Tokens 0 to 4: ratios past FP32 with advantage 0 and 1, then a weight of 0 beside an
    overflowing loss, an overflowing KL term and a masked label; the rest as they come."""
    logits, labels, old, adv, ref, w = M.rollout(11, 40, vocab, dtype, hidden=0.0)
    logp = R.logprobs(logits, labels, 1.0)[0]
    w = w + 0.1
    old[:3] = (logp[:3] - 100.0).float()
    ref = (logp + 0.3).float()
    adv[:3] = torch.tensor([0.0, 1.0, -1.0], device=DEV)
    w[2:5] = 0.0
    ref[3] = logp[3].float() + 200.0
    logits[4, labels[4]] = -INF
    ref[4] = 0.0
    return logits, labels, old, adv, ref, w


def test_the_kl_term_of_a_masked_label_is_infinite():
    """exp(d) - d - 1 at d = +inf (the reference model allows a label that the logits mask) and
    at d = -inf is infinite, as towards it; of two infinities NaN."""
    logits, labels, old, adv, ref, _ = M.rollout(12, 4, 67, hidden=0.0)
    for t in (0, 1):
        logits[t, labels[t]] = -INF
    ref[:3] = torch.tensor([-3.0, -INF, -INF], device=DEV)
    b, _ = M.run_policy(logits, labels, old, adv, ref_logp=ref, kl_coef=0.05)
    assert b.token_kl[0].item() == INF and math.isnan(b.token_kl[1].item())
    assert b.token_kl[2].item() == INF and math.isfinite(b.token_kl[3].item())


@pytest.mark.parametrize("vocab", [67, 1003, 32_000])
@pytest.mark.parametrize("denominator", [0.0, 13.0])
def test_nothing_times_an_overflow_is_nothing(vocab, denominator):
    """A token without an advantage or without a weight adds nothing to the loss and has no
    gradient, where its ratio or its loss is past FP32 too: as the formula in 64 bits has it."""
    logits, labels, old, adv, ref, w = overflowing(vocab)
    b, d = M.run_policy(logits, labels, old, adv, ref_logp=ref, weights=w, kl_coef=0.05,
                        clip_high=0.28, denominator=denominator)
    assert torch.isfinite(b.token_loss[:2]).all()
    assert bool((b.token_loss[2:5] == INF).all())
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[4] = False  # infinite in 64 bits as well; the others are the formula's
    logp, p = R.logprobs(logits, labels, 1.0)
    want = R.policy(torch.where(keep, logp, logp.new_tensor(-1.0)), keep | ~keep, old, adv,
                    torch.where(keep, ref, -1.0), w, 0.2, 0.28, 0.05, denominator)
    finite = w.double() * want["token_loss"].abs()
    # 60 units of a log-probability's error, through ratios that are at most e of one another
    assert abs(b.loss.item() - want["loss"].item()) <= 400 * U32 * finite.sum().item() / (
        denominator or 40)
    assert not d[2:5].any() and bool(torch.isfinite(d).all())
    grad = R.logprobs_gradient(logits, labels, p, want["dlogp"], 1.0)
    assert bool(((d.double() - grad).abs() <= 400 * U32 * (
        want["dlogp"].abs().max())).all())
    # the gradient taken later
    lse, dlogp = torch.empty(40, 2, device=DEV), torch.empty(40, device=DEV)
    M.run_policy(logits, labels, old, adv, grad=False, ref_logp=ref, weights=w, kl_coef=0.05,
                 clip_high=0.28, denominator=denominator, lse=lse, dlogp=dlogp)
    assert not dlogp[2:5].any() and bool(torch.isfinite(dlogp).all())


def test_a_nan_is_not_hidden_by_a_zero():
    logits, labels, old, adv, ref, w = overflowing(300)
    for make in ("advantage", "weight"):
        x, a, v = logits.clone(), adv.clone(), w.clone()
        x[7, 3] = NAN
        a[7] = 0.0 if make == "advantage" else 1.0
        v[7] = 0.0 if make == "weight" else 1.0
        b, d = M.run_policy(x, labels, old, a, ref_logp=ref, weights=v, kl_coef=0.05)
        assert math.isnan(b.loss.item()) and bool(torch.isnan(d[7]).all())
        assert bool(torch.isfinite(d[8:]).all())
