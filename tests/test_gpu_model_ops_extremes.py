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


# ---- policy loss ------------------------------------------------------------------------

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
