"""The residual blocks' operators where their numbers or their callers come to an end: choices that
one list of the router holds alone, squares next to FP32's largest, losses that nobody asked
for, and calls of several threads at once."""

import threading


import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import block_reference as B
from amsgrad_optimizer_step_gb300 import _lib
from model_reference import U32, assert_close
from test_gpu_block_ops import DEV, Case, _built, check_route  # noqa: F401
from test_gpu_model_ops import gen, randn

pytestmark = pytest.mark.gpu


# ---- the router's choice ---------------------------------------------------------------

def lanes(experts):
    """Lanes that share a token's logits: each has every so many-th run of eight."""
    return next(n for most, n in ((8, 1), (16, 2), (32, 4), (64, 8), (128, 8), (256, 16),
                                  (1024, 32)) if experts <= most)


@pytest.mark.parametrize("experts", [64, 72, 128, 129, 160, 256, 300, 384, 512, 520, 1024])
@pytest.mark.parametrize("spread", ["ulp", "same", "wide"])
def test_the_largest_logits_with_one_lane(experts, spread):
    """The nine (or more) largest logits of a token lie with one lane; the eighth and the ninth are
    one step of FP32 apart, either way round, or equal, or far apart."""
    g = gen(experts)
    tokens, width = 96, lanes(experts)
    logits = -4.0 - torch.rand(tokens, experts, device=DEV, generator=g)
    for t in range(tokens):
        part = t % width
        mine = [e for e in range(experts) if e // 8 % width == part]
        order = torch.randperm(len(mine), generator=torch.Generator().manual_seed(t)).tolist()
        mine = [mine[i] for i in order][:9 + t % 3]
        if t % 4 == 0:  # the first run of the lane and the first expert of the next
            mine = sorted(e for e in range(experts) if e // 8 % width == part)[:9]
        for place, e in enumerate(mine):
            logits[t, e] = 9.0 - place if place < 7 else 1.0
        if len(mine) > 8:
            step = {"ulp": 2.0 ** -23, "same": 0.0, "wide": 0.25}[spread]
            logits[t, mine[7 + t // 4 % 2]] += step
    check_route(logits, 8)
    check_route(logits, 7)


# ---- squares next to FP32's largest -----------------------------------------------------

@pytest.mark.parametrize("kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("cols,least", [(4104, 1e38), (8192, 1e38), (8192, 2.8e38), (16383, 1e38),
                                        (16384, 1e38)])
def test_norms_of_the_largest_rows(kind, cols, least):
    """Elements of 1e38 to 3e38: their roots' inverses are FP32's subnormals, which are off by half
    of 2^-149, and the norms are of order one."""
    half = 2.0 ** -150
    for rows in (3, 40):
        c = Case(rows, cols, *kind, alpha=1.0, p=0.1 if rows == 40 else 0.0, seed=cols)
        for t, most in ((c.residual, 2.9e38), (c.branch, 3.3e38)):
            t.copy_((least + (most - least) * torch.rand(rows, cols, device=DEV, generator=c.g)) *
                    torch.sign(t.float()))
        c.forward(check=False)
        want, err, rstd = B.join(c.residual, c.branch, c.post_weight, c.gate, True, c.alpha, c.beta,
                                 c.eps, 0.0, c.mask, c.scale)
        share = (want - c.residual.double()).abs()
        assert_close(c.out, want, err + share * (half / rstd), "out")
        normed, err, pre_rstd = B.norm(c.out, c.pre_weight, c.eps, 0.0)
        assert_close(c.normed, normed, err + normed.abs() * (half / pre_rstd), "normed")
        for got, root in ((c.post_rstd, rstd), (c.pre_rstd, pre_rstd)):
            assert bool(((got.double()[:, None] - root).abs() <= B.ROOT * root + 2 * half).all())
        got = c.backward(check=False)
        want = B.join_gradient(c.out, c.branch, c.dout, c.dnormed, c.post_rstd, c.pre_rstd,
                               c.post_weight, c.pre_weight, c.gate, True, c.alpha, c.beta, 0.0,
                               c.mask, c.scale)
        yh = c.branch.double() * c.post_rstd.double()[:, None]
        for name, x in got.items():
            value, err = want[name]
            if name == "dbranch":  # a difference of two subnormal products
                err = err + 4 * half * (1 + yh.abs())
            assert_close(x, value, err, name)


# ---- losses ------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_loss_that_has_no_weight_adds_nothing(dt):
    """Logits whose squared log-sum-exp passes FP32: without a z coefficient the loss is the balance's."""
    logits = (randn(gen(3), 70, 40) + 5e19).to(dt)
    b = fa.route_buffers(70, 40, 4, DEV)
    for balance in (0.5, 0.0):
        fa.fa_route(logits, b, balance_coef=balance)
        assert b.z.item() == float("inf") and bool(torch.isfinite(b.balance).all())
        assert b.loss.item() == balance * b.balance.item()
    logits[3, 5] = float("nan")  # what is not a number stays so
    fa.fa_route(logits, b)
    assert bool(torch.isnan(b.loss).all())


def test_the_log_of_sums_next_to_one():
    """p * lse of the larger of two logits, 0 and -d, which the z loss's gradient is."""
    n = 20000
    d = torch.linspace(0, 9, n, device=DEV)
    logits = torch.stack([torch.zeros_like(d), -d], 1)
    b, dlogits = fa.route_buffers(n, 2, 1, DEV), torch.empty_like(logits)
    fa.fa_route(logits, b, z_coef=n / 2)
    fa.fa_route_gradient(logits, b, dlogits, grad_loss=torch.ones(1, device=DEV), z_coef=n / 2)
    d, x = d.double(), logits.double()
    lse, p = torch.logsumexp(x, 1), torch.softmax(x, 1)[:, 0]
    # the exponential: its argument's two roundings and two units; of the sum 1 + e its share; the
    # sum's own rounding is one of 1; the logarithm's unit; then the coefficient, p and the product
    share = torch.exp(-d) * (2 * d + 4) / (1 + torch.exp(-d))
    err = p * (share + 1 + 2 * lse) * U32 + p * lse * (share + 5) * U32
    assert bool(((dlogits[:, 0].double() - p * lse).abs() <= err).all())


def test_a_route_without_a_loss(monkeypatch):
    """layers.route of a generation step: the same choice and weights, and no sums over the tokens."""
    from amsgrad_optimizer_step_gb300 import layers
    summed = []
    plain = layers.blocks.fa_route
    monkeypatch.setattr(layers.blocks, "fa_route", lambda x, out, *args: (
        summed.append(out.summary is not None), plain(x, out, *args))[1])
    logits = randn(gen(4), 50, 72).requires_grad_()
    want = layers.route(logits, 3, None, False, 2.0)
    assert summed.pop()
    with torch.no_grad():
        got = layers.route(logits, 3, None, False, 2.0, loss=False)
        assert not summed.pop() and got[2:] == (None, None) and not got[1].requires_grad
        layers.route(logits, 3)
        assert summed.pop()  # who does not say so has the loss and the counts as ever
    for a, b in zip(got[:2], want):
        assert torch.equal(a, b)
    got = layers.route(logits.detach(), 3, loss=False)
    assert not summed.pop() and got[2:] == (None, None)
    got = layers.route(logits, 3, None, False, 2.0, loss=False)  # with a gradient, which needs them
    assert summed.pop() and got[2:] == (None, None) and not got[0].requires_grad
    assert torch.equal(got[1], want[1])
    dw = randn(gen(5), 50, 3)
    (a,), (b,) = (torch.autograd.grad(x, logits, dw) for x in (got[1], want[1]))
    assert torch.equal(a, b)


# ---- several threads ---------------------------------------------------------------------

class Recorded:
    """The library, with the arguments of the joins' calls kept."""

    def __init__(self):
        self.lib, self.calls = _lib.load(), []

    def __getattr__(self, name):
        call = getattr(self.lib, name)
        if name not in ("fa_block_join", "fa_block_join_gradient"):
            return call

        def keep(*args):
            self.calls.append((call, args))
            return call(*args)

        return keep


@pytest.mark.parametrize("shapes,which", [
    (((304, 264, "bf16"), (31, 5120, "bf16")), 0), (((1, 2048, "bf16"), (1, 5120, "bf16")), 1),
    (((1, 6160, "f32"), (1, 16384, "f32")), 1), (((1, 515, "bf16"), (1, 16383, "bf16")), 1)])
def test_joins_of_two_widths_by_several_threads(shapes, which):
    """One kernel with two amounts of shared memory, called as fast as threads can: no launch is
    refused, and the results are those of a call alone."""
    work = []
    for i in range(6):
        c, lib, stream = Case(*shapes[i // 3], p=0.1), Recorded(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream), _lib.using(lib):
            c.forward(check=False)
            made = c.backward(check=False)
        stream.synchronize()
        made = [c.out, c.normed, *made.values()]
        work.append((made, [t.clone() for t in made], lib.calls[which], c))
    torch.cuda.synchronize()
    start, refused = threading.Event(), [0] * len(work)

    def run(i):
        call, args = work[i][2]
        start.wait()
        for _ in range(3000):
            refused[i] += call(*args) != 0

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    start.set()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(refused), refused
    for made, want, _, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(made, want))
