"""What the row sums of the log-probabilities owe their accuracy to, each by rows that show it:
errors of one sign add up over the tokens of a sequence, where those of either sign do not.

The row's statistics (m, s) are compared with the sum in 64 bits: relative errors of s.  A unit
is 2^-24 here."""

import math

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
from model_reference import DTYPES, U32
from test_gpu_model_ops import DEV, INF, gen, randn

pytestmark = pytest.mark.gpu

# The hardware's exponential is low by half a unit in the last place on average (4.3e-8 over all
# mantissas); what a correction by one unit or none may leave on average is half of that.
MEAN = U32 * 0.5 / math.log(2) / 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from amsgrad_optimizer_step_gb300 import build
    build.build()


def errors(logits, labels, scale=1.0):
    """(relative errors of s, errors of logp) against 64 bits."""
    n = logits.shape[0]
    logp, lse = torch.empty(n, device=DEV), torch.empty(n, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse, scale)
    of_s, of_logp = [], []
    for a in range(0, n, 2048):
        x = logits[a:a + 2048].double() * scale
        top = x.amax(1)
        s = torch.exp(x - top[:, None]).sum(1)
        assert torch.equal(lse[a:a + 2048, 0], logits[a:a + 2048].amax(1).float())
        of_s.append(lse[a:a + 2048, 1].double() / s - 1)
        want = x.gather(1, labels[a:a + 2048, None])[:, 0] - top - torch.log(s)
        of_logp.append(logp[a:a + 2048].double() - want)
    return torch.cat(of_s), torch.cat(of_logp)


def assert_mean(e, bound):
    """|mean| within the bound, and four standard errors of the sample."""
    assert abs(e.mean().item()) <= bound + 4 * e.std().item() / math.sqrt(e.numel()), e.mean().item()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("rows,vocab", [(20_000, 1000), (8000, 32_000)])
@pytest.mark.parametrize("sigma,scale", [(0.3, 1.0), (2.0, 1.0), (2.0, 0.7), (1.0, 1.9)])
def test_errors_have_no_sign(dt, rows, vocab, sigma, scale):
    """Rows of a language model's kind, at scales whose k = scale log2(e) rounds by different
    parts: neither the exponential nor k's rounding shows in the mean of s or of logp."""
    g = gen(vocab)
    logits = randn(g, rows, vocab, dtype=DTYPES[dt], sigma=sigma)
    labels = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    of_s, of_logp = errors(logits, labels, scale)
    assert_mean(of_s, MEAN)
    assert_mean(of_logp, MEAN)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_rising_rows_have_no_sign(dt):
    """The maximum rises with every batch: what the sum so far is multiplied by is as good as
    exact."""
    g = gen(1)
    logits = randn(g, 4000, 32_000, sigma=2.0).sort(1).values.to(DTYPES[dt])
    labels = torch.randint(0, 32_000, (4000,), device=DEV, generator=g)
    assert_mean(errors(logits, labels)[0], MEAN)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_small_terms_beside_a_large_one(dt):
    """One logit at 0 and 31999 equal ones far below.  A thread adds its 125 elements in eight
    batches; each batch's sum, five steps of a warp, and as many of the parts round by half a unit in
    the last place; the one exponential in play is off by one at most, which is two units.  (Added
    one by one, 62 equal roundings a lane would come to 62 units.)"""
    t = torch.linspace(-17.0, -8.0, 256, device=DEV)
    logits = t[:, None].expand(256, 32_000).to(DTYPES[dt]).contiguous()
    logits[:, 5] = 0.0
    labels = torch.full((256,), 5, device=DEV)
    of_s, _ = errors(logits, labels)
    assert of_s.abs().max().item() <= (8 + 5 + 5 + 2) * U32


def half_unit(x):
    return 2.0 ** (torch.floor(torch.log2(x.abs())) - 24)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_equal_logits_are_counted_exactly(dt):
    """s is the number of logits of a uniform row, and logp the rounded logarithm of it (to 8e-9
    more, the error stated for the logarithm twice)."""
    sizes = list(range(1, 1500)) + [2047, 4099, 8191, 32_000, 50_021, 100_003, 131_072]
    logp, lse = torch.empty(len(sizes), device=DEV), torch.empty(len(sizes), 2, device=DEV)
    row = torch.full((1, max(sizes)), 1.375, dtype=DTYPES[dt], device=DEV)
    label = torch.zeros(1, dtype=torch.int64, device=DEV)
    for i, n in enumerate(sizes):
        fa.fa_token_logprobs(row[:, :n], label, logp[i:i + 1], lse[i:i + 1])
    count = torch.tensor(sizes, dtype=torch.float64, device=DEV)
    assert torch.equal(lse[:, 1].double(), count)
    want = -torch.log(count[1:])
    assert bool(((logp[1:].double() - want).abs() <= half_unit(want) + 8e-9).all())


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("vocab", [64, 1003, 32_000])
def test_equal_logits_among_masked_ones_are_counted_exactly(dt, vocab):
    g = gen(vocab)
    counts = torch.arange(1, 65, device=DEV)
    order = torch.rand(64, vocab, device=DEV, generator=g).argsort(1)
    logits = torch.full((64, vocab), -INF, dtype=DTYPES[dt], device=DEV)
    logits[order < counts[:, None]] = -2.5
    # runs of neighbours too: what one vector holds
    for k in range(16):
        logits[k] = -INF
        logits[k, 3:4 + k] = -2.5
    labels = logits.argmax(1)
    logp, lse = torch.empty(64, device=DEV), torch.empty(64, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse)
    assert torch.equal(lse[:, 1], counts.float())
    want = -torch.log(counts.double())
    close = (logp.double() - want).abs()[1:] <= half_unit(want[1:]) + 8e-9
    assert bool(close.all()) and logp[0].item() == 0.0
