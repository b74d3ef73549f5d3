"""The residual blocks' operators on the GPU against their definitions in 64 bits.

Tolerances are bounds derived from the arithmetic: one rounding to the output's type plus the
FP32 error of the operation (``block_reference`` states its terms).  Sizes cover zero, one, the
edges of the kernels' runs, teams, rings and groups, and rows too wide for each of them; strided,
misaligned and in-place operands; streams and graphs.
"""

import math

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import block_reference as B
from model_reference import DTYPES, SUBNORMAL, U32, UNIT, assert_close
from test_gpu_model_ops import LAYOUTS, gen, outside_is_nan, placed, randn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    from amsgrad_optimizer_step_gb300 import build
    build.build()


# ---- dropout -----------------------------------------------------------------------

def check_dropout(x, drop, call=None, layout=(0, 0)):
    rows, cols = x.shape
    src, _ = placed(x, *layout)
    out, buf = placed(torch.full_like(x, NAN), *layout)
    fa.fa_dropout(src, out, drop)
    keep = B.kept(rows, cols, drop.p, drop.seed, drop.offset if call is None else call, DEV)
    want = torch.where(keep, x.double() * B.keep_scale(drop.p), 0.0)
    # the scale in FP32 and one product
    assert_close(out, want, 2 * U32 * want.abs(), "dropout")
    assert bool((out[~keep] == 0).all()) and outside_is_nan(out, buf)
    return out


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (1, 8), (5, 64), (4, 65), (33, 515), (7, 1408),
                                   (2, 5633), (513, 8)])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout_sizes_and_types(dt, shape, p):
    x = randn(gen(1), *shape, dtype=DTYPES[dt])
    check_dropout(x, fa.Dropout(p, 1234567890123, 77))


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("cols", [5, 64, 200, 1003])
def test_dropout_layouts(dt, layout, cols):
    x = randn(gen(2), 9, cols, dtype=DTYPES[dt])
    a = check_dropout(x, fa.Dropout(0.3, 5), layout=layout)
    b = check_dropout(x, fa.Dropout(0.3, 5))
    assert torch.equal(a, b)  # the mask does not depend on the layout


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 1 - 2.0 ** -16, 1 - 2.0 ** -18, 1.0])
def test_dropout_probabilities(p):
    x = randn(gen(3), 40, 264)
    out = check_dropout(x, fa.Dropout(p, 9, 9))
    if p < 2.0 ** -16:
        assert torch.equal(out, x)
    if p > 1 - 2.0 ** -17:
        assert not out.any()


@pytest.mark.parametrize("seed,offset", [(0, 0), (-1, -1), (2 ** 63, 2 ** 64 - 1),
                                         (0x0123456789ABCDEF, 0xFEDCBA9876543210)])
def test_dropout_keys_and_a_counter_that_wraps(seed, offset):
    x = randn(gen(4), 6, 100)
    for step in (0, 1, 2 ** 62):
        counter = torch.tensor([step], device=DEV)
        check_dropout(x, fa.Dropout(0.4, seed, offset, counter), call=offset + step)


def test_dropout_drops_what_is_not_finite():
    x = randn(gen(5), 8, 520)
    keep = B.kept(8, 520, 0.5, 3, 4, DEV)
    x[~keep] = torch.where(torch.arange(int((~keep).sum()), device=DEV) % 2 == 0, NAN, INF)
    assert bool(torch.isfinite(check_dropout(x, fa.Dropout(0.5, 3, 4))).all())
    x[keep] = NAN
    check_dropout(x, fa.Dropout(0.5, 3, 4))


def test_dropout_in_place_and_of_nothing():
    for cols, layout in ((512, (0, 0)), (515, (0, 0)), (96, (3, 1))):
        x, _ = placed(randn(gen(6), 20, cols, dtype=torch.bfloat16), *layout)
        want = torch.empty(20, cols, dtype=x.dtype, device=DEV)
        fa.fa_dropout(x, want, fa.Dropout(0.2, 1))
        fa.fa_dropout(x, x, fa.Dropout(0.2, 1))
        assert torch.equal(x, want)
    for shape in ((0, 5), (5, 0)):
        x = torch.empty(shape, device=DEV)
        fa.fa_dropout(x, torch.empty_like(x), fa.Dropout(0.2))


def test_dropout_share():
    """The kept share of 2^24 elements: within five standard deviations of 1 - q / 65536."""
    x = torch.ones(4096, 4096, device=DEV)
    out = torch.empty_like(x)
    for p in (0.1, 0.75):
        fa.fa_dropout(x, out, fa.Dropout(p, 2024))
        q = B.dropped_share(p) / B.LEVELS
        share = (out == 0).double().mean().item()
        assert abs(share - q) < 5 * math.sqrt(q * (1 - q) / x.numel())


# ---- the join ----------------------------------------------------------------------

class Case:
    """Operands of a join, with what the library and the reference take."""

    def __init__(self, rows, cols, dt="bf16", st=None, wt=None, groups=1, post=True, pre=True,
                 weights=True, branch=True, p=0.0, alpha=0.9, beta=0.7, offset=0.0, eps=1e-6,
                 seed=0, layout=(0, 0), sigma=1.0):
        g = gen(seed)
        self.dt, self.st = DTYPES[dt], DTYPES[st or dt]
        self.wt = DTYPES[wt or dt]
        self.rows, self.cols, self.layout = rows, cols, layout
        self.residual = self.place(randn(g, rows, cols, dtype=self.st, sigma=2.0 * sigma))
        self.branch = self.place(randn(g, rows, cols, dtype=self.dt, sigma=sigma)) if branch else None

        def weight(on):
            return (1 - offset + randn(g, cols, sigma=0.3)).to(self.wt) if on and weights else None

        post = post and branch
        self.post_weight, self.pre_weight = weight(post), weight(pre)
        self.gate = None
        if groups and branch:
            self.gate = self.place((0.5 + randn(g, groups, cols, sigma=0.4)).to(self.wt))
        self.post, self.pre, self.groups = post, pre, groups if branch else 0
        self.drop = fa.Dropout(p, 42 + seed, 7) if p else None
        self.mask = B.kept(rows, cols, p, 42 + seed, 7, DEV) if p and branch else None
        self.scale = B.keep_scale(p) if p else 1.0
        self.alpha, self.beta, self.eps, self.offset = alpha, beta, eps, offset
        self.record = fa.Join(post, alpha, beta, eps, offset, self.drop)
        self.g = g

    def place(self, x):
        return placed(x, *self.layout)[0]

    def empty(self, dtype):
        return placed(torch.full((self.rows, self.cols), NAN, dtype=dtype, device=DEV), *self.layout)

    def forward(self, check=True):
        out, out_buf = self.empty(self.st)
        normed, normed_buf = self.empty(self.dt) if self.pre else (None, None)
        rstd = torch.full((2, self.rows), NAN, device=DEV)
        self.post_rstd = rstd[0] if self.post else None
        self.pre_rstd = rstd[1] if self.pre else None
        fa.fa_block_join(self.record, self.residual, self.branch, out, normed, self.post_rstd,
                         self.pre_rstd, self.post_weight, self.pre_weight, self.gate)
        self.out, self.normed = out, normed
        if not check:
            return
        want, err, post_rstd = B.join(self.residual, self.branch, self.post_weight, self.gate,
                                      self.post, self.alpha, self.beta, self.eps, self.offset,
                                      self.mask, self.scale)
        assert_close(out, want, err, "out")
        assert outside_is_nan(out, out_buf)
        if self.post:
            self.check_root(self.post_rstd, post_rstd)
        if self.pre:
            want, err, pre_rstd = B.norm(out, self.pre_weight, self.eps, self.offset)
            assert_close(normed, want, err, "normed")
            assert outside_is_nan(normed, normed_buf)
            self.check_root(self.pre_rstd, pre_rstd)

    @staticmethod
    def check_root(got, want):
        got = got.double()[:, None]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        close = (got - want).abs() <= (B.ROOT + 4 * U32) * want
        assert bool((close | torch.isnan(want)).all())

    def draw(self, dout=True, dnormed=True):
        self.dout = self.dnormed = None
        if dout:
            self.dout = self.place(randn(self.g, self.rows, self.cols, dtype=self.st))
        if dnormed and self.pre:
            self.dnormed = self.place(randn(self.g, self.rows, self.cols, dtype=self.dt))
        return self

    def backward(self, dout=True, dnormed=True, only=None, check=True, draw=True):
        layout = self.layout
        if draw:
            self.draw(dout, dnormed)
        pre = self.dnormed is not None

        def like(name, t):
            if t is None or (only is not None and name not in only):
                return None, None
            if t.dim() == 2:
                return placed(torch.full_like(t, NAN), *layout)
            return torch.full_like(t, NAN), None

        made = {"dresidual": like("dresidual", self.residual),
                "dbranch": like("dbranch", self.branch),
                "dpost_weight": like("dpost_weight", self.post_weight),
                "dpre_weight": like("dpre_weight", self.pre_weight if pre else None),
                "dgate": like("dgate", self.gate)}
        scratch = fa.join_scratch(self.rows, self.cols, self.groups, DEV)
        scratch.fill_(0xff)  # NaN: what is read has been written
        fa.fa_block_join_gradient(
            self.record, self.out if pre else None, self.branch, self.dout, self.dnormed,
            made["dresidual"][0], made["dbranch"][0], scratch, self.post_rstd,
            self.pre_rstd if pre else None, self.post_weight, self.pre_weight if pre else None,
            self.gate, made["dpost_weight"][0], made["dpre_weight"][0], made["dgate"][0])
        got = {k: v[0] for k, v in made.items() if v[0] is not None}
        if not check:
            return got
        want = B.join_gradient(self.out, self.branch, self.dout, self.dnormed, self.post_rstd,
                               self.pre_rstd, self.post_weight, self.pre_weight if pre else None,
                               self.gate, self.post, self.alpha, self.beta, self.offset,
                               self.mask, self.scale)
        for name, x in got.items():
            assert_close(x, *want[name], name)
            if made[name][1] is not None:
                assert outside_is_nan(x, made[name][1]), name
        return got


KINDS = [("f32", "f32", "f32"), ("f16", "f16", "f16"), ("bf16", "bf16", "bf16"),
         ("f16", "f32", "f16"), ("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"),
         ("f16", "f32", "f32")]
FLAGS = [dict(), dict(p=0.2, offset=1.0), dict(post=False), dict(pre=False, p=0.1),
         dict(post=False, pre=False, groups=0), dict(branch=False), dict(weights=False, groups=0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("shape", [(5, 96), (700, 264), (3, 515)])
def test_join_types_and_parts(kind, flags, shape):
    c = Case(*shape, *kind, **flags)
    c.forward()
    c.backward()


# a few rows and many of each width: one run, the edges of a warp's lanes and of two runs a lane, the
# gradient's edges (6144 and 8192 columns), and rows that no ring has room for
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 64, 256, 257, 264, 512, 1000, 2048, 4104, 6144, 6152,
                                  8192, 8200, 16384])
@pytest.mark.parametrize("kind", [KINDS[2], KINDS[4], KINDS[0]])
def test_join_widths(cols, kind):
    for rows in (1, 3, max(4, 200_000 // cols)):
        c = Case(rows, cols, *kind, p=0.1, seed=cols)
        c.forward()
        c.backward()


@pytest.mark.parametrize("rows", [1, 2, 31, 33, 151, 153, 455, 457, 913, 5000])
def test_join_lengths(rows):
    for cols in (40, 1032):
        c = Case(rows, cols, "bf16", seed=rows)
        c.forward()
        c.backward()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", KINDS)
def test_join_layouts(layout, kind):
    for rows, cols in ((4, 40), (300, 515), (200, 1032)):
        c = Case(rows, cols, *kind, layout=layout, p=0.1, groups=2)
        c.forward()
        c.backward()


@pytest.mark.parametrize("rows,groups,cols", [
    (6, 6, 40), (700, 700, 264), (700, 7, 264), (701, 1, 264), (2000, 1000, 96), (1368, 24, 2048),
    (5000, 2, 1032), (11001, 3667, 24), (600, 5, 6152), (40, 8, 8200), (12000, 6000, 24),
    (9000, 9000, 24), (304, 19, 515)])
def test_join_groups(rows, groups, cols):
    """Groups of one row, of many, inside a CTA's rows and over several CTAs', more than CTAs."""
    c = Case(rows, cols, "bf16", "f32", "f32", groups=groups, p=0.1)
    c.forward()
    c.backward()


@pytest.mark.parametrize("only", [("dresidual",), ("dbranch",), ("dpost_weight",), ("dgate",),
                                  ("dpre_weight", "dgate"), ()])
def test_join_gradients_asked_for_alone(only):
    for rows, cols, groups in ((50, 264, 5), (400, 515, 1), (20, 8200, 2)):
        c = Case(rows, cols, "bf16", groups=groups, p=0.2)
        c.forward(check=False)
        got = c.backward(only=only)
        assert set(got) == set(only)


@pytest.mark.parametrize("dout,dnormed", [(True, False), (False, True)])
def test_join_with_one_gradient(dout, dnormed):
    for rows, cols in ((50, 264), (400, 515), (20, 8200)):
        c = Case(rows, cols, "f16", p=0.2)
        c.forward(check=False)
        c.backward(dout=dout, dnormed=dnormed)


def test_join_in_place():
    for rows, cols in ((3, 2048), (700, 264), (300, 515)):
        c = Case(rows, cols, "bf16", p=0.1)
        c.forward(check=False)
        x = c.residual.clone()
        normed = torch.empty_like(x)
        fa.fa_block_join(c.record, x, c.branch, x, normed, None, None, c.post_weight,
                         c.pre_weight, c.gate)
        assert torch.equal(x, c.out) and torch.equal(normed, c.normed)


def test_the_norm_can_be_taken_again_from_the_stored_stream():
    """normed is the norm of out as it is stored: a join without a branch gives it bit for bit,
    whatever the number of rows (each has its own kernel)."""
    for rows, cols, dt, st in ((700, 264, "bf16", "bf16"), (5, 2048, "f16", "f16"),
                               (900, 1032, "bf16", "f32")):
        c = Case(rows, cols, dt, st)
        c.forward(check=False)
        for part in (slice(None), slice(0, 2)):
            again = torch.empty_like(c.normed[part])
            fa.fa_block_join(fa.Join(False, eps=c.eps), c.out[part], None, None, again,
                             pre_weight=c.pre_weight)
            if part == slice(None):
                assert torch.equal(again, c.normed)
            else:  # another order of the sums
                want, err, _ = B.norm(c.out[part], c.pre_weight, c.eps, 0.0)
                assert_close(again, want, err, "normed")


def test_join_of_huge_rows():
    """Rows whose squares pass FP32 are normed all the same, and their gradients are finite."""
    for rows, cols in ((4, 264), (700, 264), (300, 515), (6, 8200)):
        c = Case(rows, cols, "f32", beta=1e19)
        c.residual.mul_(1e19)
        c.branch.mul_(1e22)
        c.forward()
        c.backward()


def test_join_rows_that_are_not_finite():
    """A NaN or an infinity in a row stays in that row (and in the weights' gradients)."""
    for rows, cols in ((6, 264), (700, 264), (300, 515)):
        c = Case(rows, cols, "f32")
        c.residual[1, 3], c.branch[2, 5], c.branch[4, 7] = NAN, NAN, INF
        c.forward()
        got = c.backward(check=False)
        fine = torch.ones(rows, dtype=torch.bool, device=DEV)
        fine[[1, 2, 4]] = False
        for name in ("dresidual", "dbranch"):
            assert bool(torch.isfinite(got[name][fine]).all())


def test_join_drops_what_is_not_finite():
    """Without the first norm, a dropped element adds nothing and has no gradient, whatever it is."""
    for rows, cols in ((6, 264), (700, 264), (300, 515), (5, 8200)):
        c = Case(rows, cols, "f32", post=False, p=0.5)
        c.branch[~c.mask] = NAN
        c.forward()
        dirty = c.branch
        c.branch = torch.where(c.mask, c.branch, torch.zeros_like(c.branch))
        want = c.backward()
        c.branch = dirty
        got = c.backward(check=False, draw=False)
        assert all(torch.equal(want[name], got[name]) for name in want)
        assert not got["dbranch"][~c.mask].any()


def test_join_zero_rows_and_columns():
    for rows, cols in ((0, 264), (5, 0)):
        c = Case(rows, cols, "bf16", groups=1)
        c.forward(check=False)
        got = c.backward(check=False)
        for name in ("dpost_weight", "dpre_weight", "dgate"):
            assert not got[name].any()
    x = torch.zeros(700, 264, device=DEV)  # rows of zeros: eps keeps them
    out, normed = torch.empty_like(x), torch.empty_like(x)
    fa.fa_block_join(None, x, x.clone(), out, normed)
    assert not out.any() and not normed.any()


def test_join_is_reproducible():
    c = Case(3000, 2048, "bf16", groups=6, p=0.1)
    c.forward(check=False)
    first = c.backward(check=False)
    for _ in range(3):
        again = c.backward(check=False, draw=False)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_join_gradient_against_differences():
    """The gradient of a scalar against central differences of the forward pass, FP32."""
    rows, cols, h = 3, 24, 1e-2
    c = Case(rows, cols, "f32", p=0.2, groups=3, alpha=0.8, beta=1.3)
    c.forward()
    got = c.backward()

    def value():
        out, normed = torch.empty(rows, cols, device=DEV), torch.empty(rows, cols, device=DEV)
        fa.fa_block_join(c.record, c.residual, c.branch, out, normed, None, None, c.post_weight,
                         c.pre_weight, c.gate)
        return ((out * c.dout).double().sum() + (normed * c.dnormed).double().sum()).item()

    for name, t in (("dresidual", c.residual), ("dbranch", c.branch), ("dgate", c.gate),
                    ("dpost_weight", c.post_weight), ("dpre_weight", c.pre_weight)):
        flat = t.view(-1)
        for i in (0, 7, flat.numel() - 1):
            keep = flat[i].item()
            flat[i] = keep + h
            up = value()
            flat[i] = keep - h
            down = value()
            flat[i] = keep
            # the difference's own error: h^2 of third derivatives of order ten, and FP32 sums of
            # some hundred terms of order one over 2 h
            assert abs((up - down) / (2 * h) - got[name].view(-1)[i].item()) < 2e-2, (name, i)


# ---- the router ----------------------------------------------------------------------

def logits_for(g, tokens, experts, dt, kind="normal"):
    x = randn(g, tokens, experts, sigma=1.5)
    if kind == "ties":  # a handful of values
        x = torch.round(x)
    if kind == "equal":
        x = torch.zeros_like(x)
    if kind == "close":  # FP32 logits that agree in their upper bits
        x = 3.0 + torch.randint(0, 9, x.shape, device=DEV, generator=g) * 2.0 ** -22
    if kind == "signed zeros":
        x = torch.where(x > 0, 0.0, -0.0)
    return x.to(DTYPES[dt])


def check_route(logits, k, counted=None, renormalise=True, weight_scale=1.0, balance=0.01,
                z=0.001, layout=(0, 0), gradient=True):
    tokens, experts = logits.shape
    src, _ = placed(logits, *layout)
    b = fa.route_buffers(tokens, experts, k, DEV)
    b.scratch.fill_(0xff)
    fa.fa_route(src, b, counted, renormalise, weight_scale, balance, z)
    x = logits.double().requires_grad_()
    want = B.route(x, k, counted, renormalise, weight_scale, balance, z)
    assert torch.equal(b.chosen.long(), want["chosen"])
    assert torch.equal(b.counts.long(), want["counts"])
    # an exponential is off by its argument's rounding and two units, a sum by its additions (16 of
    # a lane, five of a warp), weights and probabilities by both and a quotient
    span = (logits.double().amax(1) - logits.double().amin(1)).nan_to_num(posinf=40.0).clamp(max=40.0)
    span = span if counted is None else torch.where(counted, span, torch.zeros_like(span))
    rel = (2 * span + 40) * U32
    w = want["weights"].detach()
    assert_close(b.weights, w, rel[:, None] * w.abs(), "weights")
    top = rel.max().item() if tokens else 0.0
    n = max(1, want["n"])
    # sums over tokens: at most as many additions as a lane has turns, and the joining ones
    many = (tokens / 456 + 60) * U32
    mp = want["mean_prob"].detach()
    assert_close(b.mean_prob, mp, (top + many) * mp, "mean_prob")
    bal, zs = want["balance"].detach(), want["z"].detach()
    assert_close(b.balance, bal.view(1), (top + many + 8 * U32) * bal, "balance")
    big = logits.double().abs().amax().nan_to_num(posinf=0.0) if tokens else bal
    lse_err = (top + 8 * U32) * (1 + big + math.log(experts))
    assert_close(b.z, zs.view(1), many * zs + 2 * lse_err * (1 + zs.sqrt()), "z")
    assert b.summary[3].item() == want["n"]
    only = fa.route_buffers(tokens, experts, k, DEV, loss=False)
    fa.fa_route(src, only, counted, renormalise, weight_scale)
    assert torch.equal(only.chosen, b.chosen)
    assert torch.equal(only.weights.nan_to_num(7.0), b.weights.nan_to_num(7.0))
    if not gradient:
        return b
    g = gen(98)
    dweights = randn(g, tokens, k)
    grad_loss = torch.tensor([3.0], device=DEV)
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        dx, buf = placed(torch.full_like(logits, NAN), *layout)
        fa.fa_route_gradient(src, b, dx, dweights if use_w else None, grad_loss if use_l else None,
                             counted, renormalise, weight_scale, balance, z)
        value = (want["weights"] * dweights.double()).sum() * use_w + 3.0 * want["loss"] * use_l
        (grad,) = torch.autograd.grad(value, x, retain_graph=True)
        grad = torch.where(torch.isnan(logits.double()).any(1, keepdim=True), NAN, grad) \
            if counted is None else grad
        # the terms of the formula, each within ``rel``
        p = want["p"].detach()
        wd = (w * dweights.double()).abs().sum(1, keepdim=True) * use_w
        terms = p * wd + torch.zeros_like(p).scatter_add_(
            1, want["chosen"].clamp(min=0), (w * (dweights.double().abs() + wd / weight_scale)) * use_w)
        f = want["counts"].double() / (n * k)
        lse = torch.logsumexp(x.detach(), 1, keepdim=True).abs()
        terms = terms + use_l * 3.0 / n * p * (balance * experts * (f + (p * f).sum(1, keepdim=True)) +
                                               2 * z * (lse + lse_err / top if top else lse))
        err = (2 * rel[:, None] + 30 * U32) * terms
        if counted is not None:
            err = torch.where(counted[:, None], err, torch.zeros_like(err))
        assert_close(dx, grad, err.nan_to_num(), "dlogits")
        assert outside_is_nan(dx, buf)
    return b


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("experts", [1, 2, 7, 8, 9, 16, 17, 33, 60, 64, 100, 128, 129, 256, 300,
                                     512, 520, 1024])
def test_route_sizes_and_types(dt, experts):
    for k in sorted({1, min(2, experts), min(8, experts), min(9, experts), min(32, experts)}):
        logits = logits_for(gen(experts + k), 37, experts, dt)
        check_route(logits, k, renormalise=k % 2 == 0, weight_scale=2.5)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", ["ties", "equal", "close", "signed zeros"])
@pytest.mark.parametrize("experts", [8, 60, 128, 512])
def test_route_ties(dt, kind, experts):
    logits = logits_for(gen(experts), 70, experts, dt, kind)
    for k in (1, 4, 8):
        check_route(logits, k)


@pytest.mark.parametrize("tokens", [0, 1, 2, 3, 31, 32, 33, 255, 257, 5000, 20011])
def test_route_lengths(tokens):
    for experts, k, dt in ((64, 8, "bf16"), (256, 4, "f32"), (10, 2, "f16")):
        check_route(logits_for(gen(tokens + 1), tokens, experts, dt), k)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_route_layouts(layout, dt):
    for experts in (5, 60, 128, 600):
        check_route(logits_for(gen(3), 29, experts, dt), 4, layout=layout)


@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_route_tokens_that_do_not_count(share):
    """Padding is never read, whatever it holds; with no token left the losses are 0."""
    g = gen(5)
    for experts, k in ((60, 4), (256, 8)):
        logits = logits_for(g, 300, experts, "f32")
        counted = torch.rand(300, device=DEV, generator=g) >= share
        want = check_route(logits, k, counted)
        logits[~counted] = NAN
        b = fa.route_buffers(300, experts, k, DEV)
        fa.fa_route(logits, b, counted.to(torch.uint8), balance_coef=0.01, z_coef=0.001)
        for name in ("chosen", "weights", "counts", "mean_prob", "summary", "lse"):
            assert torch.equal(getattr(b, name), getattr(want, name)), name
        dx = torch.full_like(logits, NAN)
        fa.fa_route_gradient(logits, b, dx, torch.ones(300, k, device=DEV),
                             torch.ones(1, device=DEV), counted, balance_coef=0.01, z_coef=0.001)
        assert bool(torch.isfinite(dx).all()) and not dx[~counted].any()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_route_logits_that_are_not_finite(dt):
    """-Inf is never chosen before another and has no weight; NaN and +Inf make their own rows NaN,
    whose choices are experts all the same."""
    experts, k = 40, 8
    logits = logits_for(gen(6), 12, experts, dt)
    logits[0, ::2] = -INF
    logits[1, 3:] = -INF  # three finite ones for eight choices
    b = check_route(logits, k)
    assert b.weights[1, 3:].eq(0).all()
    logits[2, 5], logits[3, 6], logits[4] = NAN, INF, -INF
    logits[5, 7] = -torch.tensor(NAN)
    r = fa.route_buffers(12, experts, k, DEV)
    fa.fa_route(logits, r, balance_coef=1.0, z_coef=1.0)
    assert torch.equal(r.chosen.long(), B.chosen(logits, k, None))
    bad = torch.zeros(12, dtype=torch.bool, device=DEV)
    bad[2:6] = True
    assert torch.equal(torch.isnan(r.weights).any(1), bad) and bool(torch.isnan(r.loss).all())
    assert int(r.counts.sum()) == 12 * k


def test_route_is_reproducible():
    logits = logits_for(gen(7), 30_000, 128, "bf16")
    b = check_route(logits, 8, gradient=False)
    first = [b.summary.clone(), b.mean_prob.clone()]
    for _ in range(3):
        fa.fa_route(logits, b, balance_coef=0.01, z_coef=0.001)
        assert torch.equal(first[0], b.summary) and torch.equal(first[1], b.mean_prob)


# ---- streams and graphs ------------------------------------------------------------------

def everything(c, logits, b, dlogits, x, y, counter):
    """One pass of all the operators."""
    fa.fa_dropout(x, y, fa.Dropout(0.3, 1, 2, counter))
    c.record = c.record._replace(dropout=fa.Dropout(0.2, 3, 4, counter))
    c.forward(check=False)
    got = c.backward(check=False, draw=False)
    fa.fa_route(logits, b, balance_coef=0.01)
    fa.fa_route_gradient(logits, b, dlogits, grad_loss=torch.ones(1, device=DEV),
                         balance_coef=0.01)
    return [y, c.out, c.normed, *got.values(), b.weights, b.counts, b.summary, dlogits]


def test_another_stream_and_a_graph_that_is_replayed():
    def operands():
        g = gen(11)
        return (Case(300, 264, "bf16", p=0.2).draw(), logits_for(g, 100, 64, "bf16"),
                fa.route_buffers(100, 64, 4, DEV), torch.empty(100, 64, dtype=torch.bfloat16,
                                                                device=DEV),
                randn(g, 30, 200), torch.empty(30, 200, device=DEV))

    wants = []
    for step in (5, 6):
        wants.append([t.clone() for t in everything(*operands(), torch.tensor([step], device=DEV))])
    assert not torch.equal(wants[0][0], wants[1][0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything(*operands(), torch.tensor([5], device=DEV))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, wants[0]))

    ops, counter = operands(), torch.tensor([5], device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = everything(*ops, counter)
    for step, want in zip((5, 6), wants):
        counter.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_waited_in_vain():
    torch.cuda.synchronize()
    assert fa.fa_device_error() == 0
