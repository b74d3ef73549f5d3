"""The model-side operators on the GPU against their definitions in 64 bits.

Tolerances are bounds derived from the arithmetic: one rounding to the output's type plus
the FP32 error of the operation (each test states its terms).  Sizes cover zero, one and
the edges of the kernels' vectors, chunks and units; masks that leave nothing; strided,
misaligned and in-place operands; streams, graphs and offsets past 32 bits.
"""

import math

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import model_reference as R
from model_reference import DTYPES, U32, assert_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    from amsgrad_optimizer_step_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, sigma=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * sigma).to(dtype)


def placed(x, pad=0, off=0):
    """x as a view of a larger matrix: rows pad elements apart, off elements in, the rest NaN
    (for outputs: so that a write outside shows)."""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + off + 8,), NAN, dtype=x.dtype, device=x.device)
    view = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view, buf


def outside_is_nan(view, buf):
    """No element of the buffer but the view's was written."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool(torch.isnan(buf[mask]).all())


LAYOUTS = [(0, 0), (8, 0), (3, 1), (5, 8)]  # (row padding, offset) in elements


# ---- embedding -------------------------------------------------------------------

@pytest.mark.parametrize("tdt", list(DTYPES))
@pytest.mark.parametrize("odt", list(DTYPES))
def test_lookup_types(tdt, odt):
    g = gen(1)
    table = randn(g, 301, 72, dtype=DTYPES[tdt])
    ids = torch.randint(-3, 305, (97,), device=DEV, generator=g)
    for it in (torch.int32, torch.int64):
        out = torch.full((97, 72), NAN, dtype=DTYPES[odt], device=DEV)
        fa.fa_embedding_lookup(ids.to(it), table, out, 45.254834)
        want = R.lookup(ids, table, 45.254834)
        # the scale in FP32 and one product
        assert_close(out, want, 2 * U32 * want.abs(), f"{tdt}->{odt}")


@pytest.mark.parametrize("dim", [1, 8, 12, 515, 2048])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_lookup_layouts(dim, layout):
    g = gen(2)
    table, _ = placed(randn(g, 50, dim, dtype=torch.bfloat16), *layout)
    ids = torch.randint(0, 50, (7,), device=DEV, generator=g, dtype=torch.int32)
    out, buf = placed(torch.zeros(7, dim, dtype=torch.bfloat16, device=DEV), *layout)
    fa.fa_embedding_lookup(ids, table, out)
    assert torch.equal(out, table[ids.long()]) and outside_is_nan(out, buf)


def test_lookup_of_no_token_no_table_and_one():
    table = randn(gen(3), 5, 16)
    fa.fa_embedding_lookup(torch.empty(0, dtype=torch.int64, device=DEV), table,
                           torch.empty(0, 16, device=DEV))
    out = torch.full((2, 16), NAN, device=DEV)
    ids = torch.tensor([0, 1], device=DEV)
    fa.fa_embedding_lookup(ids, torch.empty(0, 16, device=DEV), out)
    assert not out.any()
    out = torch.empty(1, 16, device=DEV)
    fa.fa_embedding_lookup(ids[:1], table, out)
    assert torch.equal(out, table[:1])
    # a row that is not asked for may hold anything
    table[3] = NAN
    fa.fa_embedding_lookup(ids[1:], table, out)
    assert torch.equal(out, table[1:2])


def embedding_grad(ids, dout, vocab, tdt, scale=1.0, padding=-1, before=None, layout=(0, 0)):
    start = before if before is not None else torch.full((vocab, dout.shape[1]), NAN,
                                                         dtype=tdt, device=DEV)
    dtable, buf = placed(start, *layout)
    scratch = fa.embedding_scratch(ids.numel(), vocab, dout.shape[1], DEV)
    scratch.fill_(0xa5)
    fa.fa_embedding_gradient(ids, dout, dtable, scratch, scale, padding, before is not None)
    assert outside_is_nan(dtable, buf) or not buf.numel()
    return dtable


def check_embedding_grad(ids, dout, vocab, tdt, **kw):
    got = embedding_grad(ids, dout, vocab, tdt, **kw)
    want, mag, count = R.embedding_gradient(ids, dout, vocab, kw.get("scale", 1.0),
                                            kw.get("padding", -1), kw.get("before"))
    # n terms added in some order: n - 1 roundings of partial sums, then scale and accumulate
    assert_close(got, want, (count[:, None] + 2) * U32 * mag, "embedding gradient")
    if kw.get("before") is not None:
        assert torch.equal(got[count == 0], kw["before"][count == 0])
    return got


def zipf(g, n, vocab):
    cdf = torch.cumsum(1.0 / torch.arange(1, vocab + 1, device=DEV, dtype=torch.float64), 0)
    u = torch.rand(n, device=DEV, dtype=torch.float64, generator=g) * cdf[-1]
    return torch.randperm(vocab, device=DEV, generator=g)[
        torch.searchsorted(cdf, u).clamp(max=vocab - 1)]


@pytest.mark.parametrize("tokens", [0, 1, 2, 31, 32, 33, 64, 65, 1000, 4095, 4097, 8191, 8192,
                                    8193, 20011])
@pytest.mark.parametrize("kind", ["zipf", "same", "distinct"])
def test_embedding_gradient_lengths(tokens, kind):
    g = gen(10 + tokens)
    vocab = 1009 if kind != "distinct" else max(1, tokens)
    ids = {"zipf": lambda: zipf(g, tokens, vocab),
           "same": lambda: torch.full((tokens,), 7, device=DEV),
           "distinct": lambda: torch.randperm(vocab, device=DEV, generator=g)[:tokens]}[kind]()
    dout = randn(g, tokens, 24, dtype=torch.bfloat16)
    check_embedding_grad(ids, dout, vocab, torch.bfloat16, scale=0.5)


@pytest.mark.parametrize("ddt", list(DTYPES))
@pytest.mark.parametrize("tdt", list(DTYPES))
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_types(ddt, tdt, accumulate):
    g = gen(20)
    ids = torch.randint(-5, 210, (700,), device=DEV, generator=g, dtype=torch.int32)
    dout = randn(g, 700, 136, dtype=DTYPES[ddt])
    before = randn(g, 200, 136, dtype=DTYPES[tdt]) if accumulate else None
    check_embedding_grad(ids, dout, 200, DTYPES[tdt], scale=3.0, padding=11, before=before)


@pytest.mark.parametrize("dim", [1, 3, 8, 100, 515, 1032, 4104])
@pytest.mark.parametrize("layout", [(0, 0), (3, 1)])
def test_embedding_gradient_widths(dim, layout):
    g = gen(30 + dim)
    ids = zipf(g, 300, 61)
    dout, _ = placed(randn(g, 300, dim, dtype=torch.float16), *layout)
    before = randn(g, 61, dim, dtype=torch.float16)
    check_embedding_grad(ids, dout, 61, torch.float16, layout=layout)
    check_embedding_grad(ids, dout, 61, torch.float16, layout=layout, before=before)


@pytest.mark.parametrize("vocab", [1, 2, 15, 16, 17, 255, 256, 65535, 65536, 65537, 131072])
def test_embedding_gradient_vocabularies(vocab):
    """Every id of the table's ends, and none of the others' rows left out or written twice."""
    g = gen(40)
    ids = torch.randint(0, vocab, (9000,), device=DEV, generator=g)
    ids[:4] = torch.tensor([0, vocab - 1, vocab - 1, 0], device=DEV)
    check_embedding_grad(ids, randn(g, 9000, 8), vocab, torch.float32)


def test_embedding_gradient_skips_what_is_masked():
    """Tokens without an id add nothing, whatever their rows hold; all masked: zeros."""
    g = gen(50)
    ids = torch.randint(0, 30, (500,), device=DEV, generator=g)
    dout = randn(g, 500, 16)
    ids[::3] = -1
    ids[1::3] = 2 ** 40
    dout[::3] = NAN
    dout[1::3] = INF
    check_embedding_grad(ids, dout, 30, torch.float32)
    got = embedding_grad(torch.full_like(ids, -100), dout, 30, torch.float32)
    assert not got.any()


def test_embedding_gradient_is_reproducible():
    g = gen(60)
    ids = zipf(g, 50_000, 5000)
    dout = randn(g, 50_000, 64)
    first = embedding_grad(ids, dout, 5000, torch.float32)
    for _ in range(3):
        assert torch.equal(first, embedding_grad(ids, dout, 5000, torch.float32))


# ---- losses from the logits ----------------------------------------------------------

def logp_error(logits, scale):
    """FP32 error of a row's log-probability: the sum's and the two roundings of terms in
    2^(k x - k top) (the scaled distance below the top is at most span, but terms beyond 2^-30
    of the sum do not matter), the logarithm and the final difference."""
    x = logits.double() * scale
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    span = (x.amax(1) - x.amin(1)).clamp(max=40.0)
    terms = min(2 + math.ceil(logits.shape[1] / 256 / 4) + 8, 80)
    return U32 * (2 * span + terms + 12)


def check_logprobs(logits, labels, scale=1.0, in_place=False, layout=(0, 0)):
    logits, _ = placed(logits, *layout)
    n, vocab = logits.shape
    logp = torch.full((n,), NAN, device=DEV)
    lse = torch.full((n, 2), NAN, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse, scale)
    want, p = R.logprobs(logits, labels, scale)
    err = logp_error(logits, scale)
    assert_close(logp, want, err + 2 * U32 * want.abs().nan_to_num(posinf=0.0), "logp")
    only = torch.full((n,), NAN, device=DEV)
    fa.fa_token_logprobs(logits, labels, only, None, scale)
    assert torch.equal(only.nan_to_num(7.0), logp.nan_to_num(7.0))
    dlogp = randn(gen(99), n, sigma=0.1)
    loss_grad = torch.tensor([0.5], device=DEV)
    # the definition in 64 bits first: in place, the kernel overwrites the logits
    grad = R.logprobs_gradient(logits, labels, p, dlogp.double() * 3.0 * 0.5, scale)
    fp = (dlogp.double().abs() * 3.0 * 0.5 * scale)[:, None] * (
        p * (2 * err[:, None] + 8 * U32) + 6 * U32 * (p > 0.25))
    if in_place:
        out, buf = logits, None
    else:
        out, buf = placed(torch.full_like(logits, NAN), *layout)
    fa.fa_token_logprobs_gradient(logits, labels, lse, dlogp, out, scale, 3.0, loss_grad)
    # the label's entry is c - c p: an FP32 rounding of c
    ok = R.counted(labels, vocab)
    fp = fp.nan_to_num()
    rows = torch.arange(n, device=DEV)[ok]
    fp[rows, labels[ok].long()] += (dlogp.double().abs() * 3.0 * 0.5 * scale)[ok] * 6 * U32
    assert_close(out, grad, fp, "dlogits")
    if buf is not None:
        assert outside_is_nan(out, buf)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 127, 1000, 2047, 2049, 8191, 32000, 65552])
def test_logprobs_sizes_and_types(dt, vocab):
    g = gen(vocab)
    logits = randn(g, 9, vocab, dtype=DTYPES[dt], sigma=3.0)
    labels = torch.randint(0, vocab, (9,), device=DEV, generator=g)
    labels[2] = -100
    labels[5] = vocab
    check_logprobs(logits, labels)
    check_logprobs(logits, labels.to(torch.int32), scale=0.7, in_place=True)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 5, 1003, 1024, 4099])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_logprobs_layouts(dt, vocab, layout):
    g = gen(vocab + 1)
    logits = randn(g, 6, vocab, dtype=DTYPES[dt], sigma=2.0)
    labels = torch.randint(0, vocab, (6,), device=DEV, generator=g)
    check_logprobs(logits, labels, layout=layout)
    check_logprobs(logits, labels, layout=layout, in_place=True)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tokens,vocab", [(4865, 1), (5003, 67), (5003, 1003), (4866, 4096),
                                          (3649, 5001)])
def test_logprobs_many_rows(dt, tokens, vocab):
    """More rows than the SMs run blocks: several to a block, the last one not full."""
    g = gen(tokens + vocab)
    logits = randn(g, tokens, vocab, dtype=DTYPES[dt], sigma=3.0)
    labels = torch.randint(0, vocab, (tokens,), device=DEV, generator=g)
    labels[torch.rand(tokens, device=DEV, generator=g) < 0.2] = -100
    check_logprobs(logits, labels)
    check_logprobs(logits, labels.to(torch.int32), scale=0.7, layout=(3, 1))


@pytest.mark.parametrize("vocab", [100_003, 131_072, 262_147])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logprobs_wide_rows(dt, vocab):
    g = gen(vocab)
    logits = randn(g, 3, vocab, dtype=DTYPES[dt], sigma=3.0)
    labels = torch.tensor([0, vocab - 1, vocab // 2], device=DEV)
    check_logprobs(logits, labels)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_logprobs_gradient_between_buffers_of_other_alignment(dt):
    """dlogits whose rows start elsewhere in a 16-byte line than the logits' rows."""
    g = gen(4)
    logits = randn(g, 5, 999, dtype=DTYPES[dt], sigma=2.0)
    labels = torch.randint(0, 999, (5,), device=DEV, generator=g)
    logp, lse = torch.empty(5, device=DEV), torch.empty(5, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse)
    dlogp = torch.ones(5, device=DEV)
    a = torch.empty_like(logits)
    fa.fa_token_logprobs_gradient(logits, labels, lse, dlogp, a)
    b, buf = placed(torch.zeros_like(logits), 2, 1)
    fa.fa_token_logprobs_gradient(logits, labels, lse, dlogp, b)
    assert torch.equal(a, b) and outside_is_nan(b, buf)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("vocab", [40, 5000])
def test_logprobs_masks(dt, vocab):
    """-inf and the type's lowest value as masks, rows with one entry left, rows all at the
    lowest value (uniform), huge spreads, rows of tokens that are not counted."""
    d = DTYPES[dt]
    low = torch.finfo(d).min
    g = gen(6)
    logits = randn(g, 10, vocab, dtype=d, sigma=2.0)
    labels = torch.full((10,), 3, device=DEV)
    logits[0, 5:] = -INF
    logits[1, :] = -INF
    logits[1, 3] = 1.5          # one entry left: logp 0, gradient 0
    logits[2, 5:] = low
    logits[3, :] = low          # every entry alike: uniform
    logits[4, 3] = -INF         # the label itself is masked: logp -inf
    logits[5, :] = NAN          # not counted
    labels[5] = -1
    logits[6, :] = INF          # not counted
    labels[6] = -100
    logits[7, 3] = low          # the label at the lowest value
    logits[8, :] = torch.finfo(d).max
    logits[9, ::2] = -INF
    n = 10
    logp, lse = torch.empty(n, device=DEV), torch.empty(n, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse)
    want, p = R.logprobs(logits, labels, 1.0)
    big = want.abs() > 1e30     # the label at FP32's or BF16's lowest value
    assert_close(logp[~big], want[~big], 80 * U32 * (1 + want[~big].abs().nan_to_num(posinf=0.0)),
                 "logp")
    assert bool((logp[big] < -1e30).all())
    out = torch.full_like(logits, NAN)
    fa.fa_token_logprobs_gradient(logits, labels, lse, torch.ones(n, device=DEV), out)
    grad = R.logprobs_gradient(logits, labels, p, torch.ones(n, device=DEV), 1.0)
    assert_close(out, grad, 100 * U32, "dlogits")
    assert not out[5].any() and not out[6].any()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("where", [0, 777, 4999])
def test_logprobs_rows_that_are_no_distribution(dt, where):
    """A NaN or +inf anywhere in a counted row, or no finite logit: NaN for that row, in the
    log-probability and in the whole gradient row; the others are untouched by it."""
    d = DTYPES[dt]
    g = gen(8)
    logits = randn(g, 4, 5000, dtype=d)
    labels = torch.tensor([1, 2, 3, 4], device=DEV)
    logits[0, where] = NAN
    logits[1, where] = INF
    logits[2] = -INF
    logp, lse = torch.empty(4, device=DEV), torch.empty(4, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse)
    assert torch.isnan(logp).tolist() == [True, True, True, False]
    out = torch.zeros_like(logits)
    fa.fa_token_logprobs_gradient(logits, labels, lse, torch.ones(4, device=DEV), out)
    assert bool(torch.isnan(out[:3]).all()) and bool(torch.isfinite(out[3]).all())


def test_logprobs_gradient_against_differences():
    """The directional derivative of sum(w * logp) by central differences of the kernel's own
    values.  With |x''' | bounded by 1 along a unit direction scaled to h, the truncation is
    h^2 / 6 * sum|w|; each value carries the FP32 error of its terms."""
    g = gen(9)
    logits = randn(g, 16, 501, sigma=2.0)
    labels = torch.randint(0, 501, (16,), device=DEV, generator=g)
    w = randn(g, 16)
    logp, lse = torch.empty(16, device=DEV), torch.empty(16, 2, device=DEV)
    fa.fa_token_logprobs(logits, labels, logp, lse)
    grad = torch.empty_like(logits)
    fa.fa_token_logprobs_gradient(logits, labels, lse, w, grad)
    h = 2.0 ** -6
    for seed in range(5):
        d = randn(gen(100 + seed), 16, 501)
        d = d / d.abs().amax()
        values = []
        for sign in (1, -1):
            fa.fa_token_logprobs((logits.double() + sign * h * d.double()).float(), labels, logp)
            values.append((w.double() * logp.double()).sum())
        slope = (values[0] - values[1]) / (2 * h)
        want = (grad.double() * d.double()).sum()
        # third derivative of logsumexp along |d| <= 1: at most 8 (a third central moment)
        bound = w.abs().sum().item() * (h * h / 6 * 8 + 60 * U32 / h)
        assert abs(slope - want) <= bound, (slope, want, bound)


def run_preference(logits, labels, offsets, ref, **kw):
    pairs = (offsets.numel() - 1) // 2
    b = fa.preference_buffers(logits.shape[0], pairs, DEV)
    for t in b:
        t.fill_(NAN)
    fa.fa_preference_loss(logits, labels, offsets, ref, b, **kw)
    return b


def check_preference(logits, labels, offsets, ref, beta=0.1, smoothing=0.0, average=False):
    b = run_preference(logits, labels, offsets, ref, beta=beta, label_smoothing=smoothing,
                       average=average)
    vocab = logits.shape[1]
    ok = R.counted(labels, vocab)
    logp, _ = R.logprobs(logits, labels, 1.0)
    loss, pair_loss, rewards, dlogp = R.preference(logp, ref, ok, offsets.tolist(), beta, smoothing,
                                                   average)
    err = logp_error(logits, 1.0) if logits.numel() else torch.zeros(logits.shape[0], device=DEV)
    each = torch.where(ok, err + 3 * U32 * (logp.abs() + ref.abs()), 0.0)
    off = [min(max(o, 0), logits.shape[0]) for o in offsets.tolist()]
    sums = torch.stack([each[a:b_].sum() / (max(1, int(ok[a:b_].sum())) if average else 1)
                        for a, b_ in zip(off[:-1], off[1:])]) if len(off) > 1 else each.new_zeros(0)
    reward_err = (beta * sums).reshape(-1, 2) + 4 * U32 * rewards.abs()
    assert_close(b.rewards, rewards, reward_err, "rewards")
    z_err = reward_err.sum(1)
    # |d loss / dz| <= 1; the transcendental functions within 4 units
    assert_close(b.pair_loss, pair_loss, z_err + 8 * U32 * (1 + pair_loss), "pair loss")
    mean_err = (z_err + 8 * U32 * (1 + pair_loss)).mean() if len(pair_loss) else 0.0
    assert_close(b.loss, loss.reshape(1), mean_err + 2 * U32 * loss, "loss")
    # |d^2 loss / dz^2| <= 1/4 and |d loss / dz| <= 1, times dz / dlogp <= beta over the pairs
    widest = z_err.max().item() if len(pair_loss) else 0.0
    assert_close(b.dlogp, dlogp, (widest / 4 + 16 * U32) * beta / max(1, len(pair_loss)), "dlogp")
    return b


def packed(seed, lens, vocab, dtype="f32", prompt=True):
    g = gen(seed)
    off = torch.tensor([0] + torch.cumsum(torch.tensor(lens), 0).tolist(), device=DEV)
    t = int(off[-1])
    logits = randn(g, t, vocab, dtype=DTYPES[dtype], sigma=2.0)
    labels = torch.randint(0, vocab, (t,), device=DEV, generator=g)
    if prompt and t:
        labels[torch.rand(t, device=DEV, generator=g) < 0.3] = -100
    ref = -3.0 + randn(g, t)
    return logits, labels, off, ref


@pytest.mark.parametrize("lens", [[1, 1], [5, 3], [0, 4], [0, 0], [3, 0, 700, 1, 2, 333],
                                  [17, 16] * 20, [257, 1025]])
@pytest.mark.parametrize("smoothing", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("average", [False, True])
def test_preference(lens, smoothing, average):
    check_preference(*packed(sum(lens), lens, 211), smoothing=smoothing, average=average)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_preference_types_and_the_decoder_vocabulary(dt):
    check_preference(*packed(3, [21, 34, 9, 13], 32000, dt), beta=0.3)


def test_preference_offsets_that_leave_tokens_out():
    """Tokens before the first offset and past the last, and offsets past the end, belong to
    no sequence: coefficient 0."""
    logits, labels, _, ref = packed(5, [40], 100)
    off = torch.tensor([3, 10, 20], device=DEV)
    b = check_preference(logits, labels, off, ref)
    assert not b.dlogp[:3].any() and not b.dlogp[20:].any()
    check_preference(logits, labels, torch.tensor([-5, 20, 400], device=DEV), ref)


def test_preference_with_nothing():
    logits, labels, off, ref = packed(6, [4, 4], 50)
    b = check_preference(logits, torch.full_like(labels, -100), off, ref)  # nothing counted
    assert abs(b.loss.item() - math.log(2)) <= 4 * U32 and not b.dlogp.any()
    b = run_preference(logits, labels, torch.tensor([0], device=DEV), ref)  # no pairs
    assert b.loss.item() == 0.0 and not b.dlogp.any()
    empty = torch.empty(0, 50, device=DEV)
    b = run_preference(empty, labels[:0], torch.tensor([0, 0, 0], device=DEV), ref[:0])
    assert abs(b.loss.item() - math.log(2)) <= 4 * U32


def test_preference_extremes():
    """Large margins saturate without overflow; an impossible label makes the loss infinite."""
    logits, labels, off, ref = packed(7, [6, 6], 64, prompt=False)
    b = check_preference(logits, labels, off, ref - 500.0 * (torch.arange(12, device=DEV) < 6),
                         beta=1.0)
    assert b.loss.item() == 0.0
    b = check_preference(logits, labels, off, ref + 500.0 * (torch.arange(12, device=DEV) < 6),
                         beta=1.0, smoothing=0.1)
    assert math.isfinite(b.loss.item())
    logits[0, labels[0]] = -INF
    b = run_preference(logits, labels, off, ref)
    assert b.loss.item() == INF


def test_preference_gradient_against_differences():
    """Loss and dlogits together, by central differences along random directions of the
    logits.  The loss's third derivative along |d| <= 1 is bounded through its chain by the
    counted tokens' number times 8 beta; the loss's FP32 error by beta times theirs."""
    logits, labels, off, ref = packed(8, [9, 7, 5, 6], 130)
    kw = dict(beta=0.2, label_smoothing=0.1)
    b = run_preference(logits, labels, off, ref, **kw)
    grad = torch.empty_like(logits)
    fa.fa_token_logprobs_gradient(logits, labels, b.lse, b.dlogp, grad)
    n, h = int((labels >= 0).sum()), 2.0 ** -5
    for seed in range(4):
        d = randn(gen(200 + seed), *logits.shape)
        d = d / d.abs().amax()
        at = [run_preference((logits.double() + s * h * d.double()).float(), labels, off, ref,
                             **kw).loss.double() for s in (1, -1)]
        slope = ((at[0] - at[1]) / (2 * h)).item()
        want = (grad.double() * d.double()).sum().item()
        slack = 0.2 * n * 2  # |dz/dx . d| <= beta n 2
        bound = h * h / 6 * (slack ** 3 / 8 + slack * 8) + (0.2 * n * 60 * U32 + 16 * U32) / h
        assert abs(slope - want) <= bound, (slope, want, bound)


def run_policy(logits, labels, old, adv, grad=True, in_place=False, **kw):
    b = fa.policy_buffers(logits.shape[0], DEV)
    for t in b:
        t.fill_(NAN)
    d = (logits if in_place else torch.full_like(logits, NAN)) if grad else None
    fa.fa_policy_loss(logits, labels, old, adv, b, dlogits=d, **kw)
    return b, d


def check_policy(logits, labels, old, adv, ref=None, weights=None, lo=0.2, hi=0.28, kl=0.0,
                 denominator=0.0, scale=1.0, grad_scale=1.0, in_place=False, off_edge=1e-4):
    vocab = logits.shape[1]
    ok = R.counted(labels, vocab)
    logp, p = R.logprobs(logits, labels, scale)
    r = torch.exp(logp - old.double())
    # a ratio within FP32 error of the clip's edge may fall either way: moved off it
    for edge in (1 - lo, 1 + hi):
        old = torch.where((r / edge - 1).abs() < off_edge, old + 3 * off_edge, old)
    want = R.policy(logp, ok, old, adv, ref, weights, lo, hi, kl, denominator)
    dlogits = R.logprobs_gradient(logits, labels, p, want["dlogp"] * grad_scale, scale)
    err = logp_error(logits, scale) if logits.numel() else torch.zeros(logits.shape[0], device=DEV)
    err = err + 3 * U32 * (logp.abs() + old.abs() + (ref.abs() if ref is not None else 0.0))
    b, d = run_policy(logits, labels, old, adv, in_place=in_place, ref_logp=ref, weights=weights,
                      clip_low=lo, clip_high=hi, kl_coef=kl, denominator=denominator,
                      logit_scale=scale, grad_scale=grad_scale)
    assert_close(b.logp, logp, err, "logp")
    r = torch.exp(logp - old.double())
    dd = torch.zeros_like(r) if ref is None else ref.double() - logp
    slope_kl = torch.expm1(dd).abs()
    kl_err = slope_kl * err + 8 * U32 * want["token_kl"].abs() + 2 * U32 * dd.abs() * slope_kl
    kl_err = kl_err + torch.exp(dd) * err * err
    tok_err = (err + 6 * U32) * r * adv.double().abs() + kl * kl_err
    zero = torch.zeros_like(r)
    assert_close(b.token_kl, want["token_kl"], torch.where(ok, kl_err, zero), "token kl")
    assert_close(b.token_loss, want["token_loss"],
                 torch.where(ok, tok_err + 2 * U32 * want["token_loss"].abs(), zero), "token loss")
    w = weights.double().abs() if weights is not None else torch.ones_like(r)
    denom = denominator if denominator else max(1, want["count"])
    n = max(1, want["count"])
    total = (w * torch.where(ok, tok_err + 3 * U32 * want["token_loss"].abs(), zero)).sum() / denom
    assert_close(b.loss, want["loss"].reshape(1), total + 2 * U32 * want["loss"].abs(), "loss")
    assert_close(b.kl, want["kl"].reshape(1),
                 torch.where(ok, kl_err, zero).sum() / n + 2 * U32 * want["kl"], "kl")
    assert_close(b.clip_fraction, want["clip_fraction"].reshape(1), 2 * U32, "clip fraction")
    assert b.count.item() == want["count"]
    assert torch.equal(b.summary, torch.cat([b.loss, b.kl, b.clip_fraction, b.count]))
    coef = want["dlogp"].abs() * grad_scale * scale
    coef_err = (w / denom * grad_scale * scale) * ((err + 8 * U32) * r * adv.double().abs() +
                                                   kl * (torch.exp(dd) * err + 8 * U32 * slope_kl))
    fp = coef[:, None] * (p * (2 * err[:, None] + 10 * U32)) + coef_err[:, None]
    y = torch.where(ok, labels, torch.zeros_like(labels)).long()[:, None]
    fp.scatter_add_(1, y, (coef * 8 * U32)[:, None])
    assert_close(d, dlogits, torch.where(ok[:, None], fp, torch.zeros_like(fp)), "dlogits")
    return b, d


def rollout(seed, tokens, vocab, dtype="f32", hidden=0.1):
    g = gen(seed)
    logits = randn(g, tokens, vocab, dtype=DTYPES[dtype], sigma=2.0)
    labels = torch.randint(0, vocab, (tokens,), device=DEV, generator=g)
    labels[torch.rand(tokens, device=DEV, generator=g) < hidden] = -100
    logp = R.logprobs(logits, labels, 1.0)[0].float()
    old, ref = logp + randn(g, tokens, sigma=0.3), logp + randn(g, tokens, sigma=0.5)
    return logits, labels, old, randn(g, tokens), ref, torch.rand(tokens, device=DEV, generator=g)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 9, 130, 1003, 8192, 32000, 65552])
def test_policy_sizes_and_types(dt, vocab):
    logits, labels, old, adv, ref, w = rollout(vocab, 23, vocab, dt)
    check_policy(logits, labels, old, adv, ref, kl=0.05)
    check_policy(logits, labels, old, adv, ref, w, kl=0.1, denominator=5.0,
                 grad_scale=1024.0, in_place=True)


@pytest.mark.parametrize("vocab", [100_003, 131_072, 262_147, 400_009])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_policy_wide_rows(dt, vocab):
    logits, labels, old, adv, ref, w = rollout(vocab, 3, vocab, dt, hidden=0.0)
    check_policy(logits, labels, old, adv, ref, kl=0.05)
    check_policy(logits, labels, old, adv, ref, kl=0.05, in_place=True)


@pytest.mark.parametrize("tokens", [1, 2, 151, 1023, 1025, 5000])
def test_policy_lengths(tokens):
    logits, labels, old, adv, ref, w = rollout(tokens, tokens, 67)
    check_policy(logits, labels, old, adv, ref, kl=0.05)
    check_policy(logits, labels, old, adv)              # no KL term
    check_policy(logits, labels, old, adv, ref)         # watched, not added
    check_policy(logits, labels, old, adv, None, w, denominator=float(tokens))
    check_policy(logits, labels.to(torch.int32), old, adv, lo=0.0, hi=0.0, off_edge=1e-3)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tokens,vocab", [(4865, 1), (5003, 67), (5003, 1003), (4866, 4096)])
def test_policy_many_rows(dt, tokens, vocab):
    logits, labels, old, adv, ref, w = rollout(tokens + vocab, tokens, vocab, dt)
    check_policy(logits, labels, old, adv, ref, kl=0.05)
    check_policy(logits, labels, old, adv, ref, w, kl=0.1, denominator=float(tokens),
                 in_place=True)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("vocab", [5, 1003, 4096])
def test_policy_layouts(dt, layout, vocab):
    logits, labels, old, adv, ref, w = rollout(1, 8, vocab, dt)
    view, _ = placed(logits, *layout)
    plain, d0 = run_policy(logits, labels, old, adv, ref_logp=ref, kl_coef=0.1)
    b = fa.policy_buffers(8, DEV)
    out, buf = placed(torch.zeros_like(logits), *layout)
    fa.fa_policy_loss(view, labels, old, adv, b, ref_logp=ref, kl_coef=0.1, dlogits=out)
    assert outside_is_nan(out, buf)
    # the cut of a row for 16-byte accesses changes the order of its sum
    for x, y in ((out.double(), d0.double()), (b.summary, plain.summary), (b.logp, plain.logp)):
        unit = R.UNIT[DTYPES[dt]] if x.dtype == torch.float64 else 0.0
        assert bool(((x - y).abs() <= (2 * unit + 200 * U32) * (y.abs() + y.abs().max() * 1e-3)
                     ).all())


def test_policy_without_a_gradient_and_with_nothing():
    logits, labels, old, adv, ref, w = rollout(2, 40, 300)
    full, _ = run_policy(logits, labels, old, adv, ref_logp=ref, kl_coef=0.1)
    only, _ = run_policy(logits, labels, old, adv, grad=False, ref_logp=ref, kl_coef=0.1)
    assert torch.equal(full.summary, only.summary) and torch.equal(full.logp, only.logp)
    b, d = run_policy(logits, torch.full_like(labels, -1), old, adv)
    assert b.summary.tolist() == [0.0, 0.0, 0.0, 0.0] and not d.any() and not b.logp.any()
    e = logits[:0]
    b, _ = run_policy(e, labels[:0], old[:0], adv[:0])
    assert b.summary.tolist() == [0.0, 0.0, 0.0, 0.0]


def test_policy_masks_and_bad_rows():
    """Masked logits have no gradient; rows not counted may hold anything; a NaN row makes its
    own loss and gradient NaN (which the gradient statistics then count)."""
    logits, labels, old, adv, ref, w = rollout(3, 12, 500, "bf16", hidden=0.0)
    logits[0, 100:] = -INF
    labels[0] = 5
    logits[1] = torch.finfo(torch.bfloat16).min
    labels[2] = -100
    logits[2] = NAN
    old = R.logprobs(logits, labels, 1.0)[0].float() + 0.05
    check_policy(logits, labels, old, adv, old - 0.3, kl=0.1)
    logits[3, 7] = NAN
    b, d = run_policy(logits, labels, old, adv, ref_logp=old, kl_coef=0.1)
    assert math.isnan(b.loss.item()) and bool(torch.isnan(d[3]).all())
    keep = [0, 1, 4, 5, 6, 7, 8, 9, 10, 11]
    assert bool(torch.isfinite(d[keep]).all()) and not d[2].any()


def test_policy_gradient_against_differences():
    """By central differences along random directions, with no ratio near a clip edge."""
    logits, labels, old, adv, ref, w = rollout(4, 30, 90)
    logp = R.logprobs(logits, labels, 1.0)[0]
    r = torch.exp(logp - old.double())
    for edge in (0.8, 1.28):
        old = torch.where((r / edge - 1).abs() < 0.1, (logp - 0.0).float(), old)
    kw = dict(ref_logp=ref, clip_low=0.2, clip_high=0.28, kl_coef=0.1)
    b, grad = run_policy(logits, labels, old, adv, **kw)
    h = 2.0 ** -7
    for seed in range(4):
        d = randn(gen(300 + seed), *logits.shape)
        d = d / d.abs().amax()
        at = [run_policy((logits.double() + s * h * d.double()).float(), labels, old, adv, grad=False,
                         **kw)[0].loss.double() for s in (1, -1)]
        slope = ((at[0] - at[1]) / (2 * h)).item()
        want = (grad.double() * d.double()).sum().item()
        # per token |third derivative| <= 27 r |A| + kl (27 e^d); the mean of them over the tokens
        rr = torch.exp(logp - old.double()) * adv.double().abs() * 1.1
        third = 27 * (rr.mean() + 0.1 * torch.exp(ref.double() - logp).mean() * 1.1 + 0.1).item()
        bound = h * h / 6 * third * 1.2 + 80 * U32 * (rr.mean().item() + 1) / h
        assert abs(slope - want) <= bound, (slope, want, bound)


# ---- gated activation -----------------------------------------------------------------

def act_terms(g, kind):
    """Magnitudes that bound the FP32 error of the activation and its derivative: the
    argument of the exponential carries 4 roundings, the rest a dozen."""
    z = g.abs() if kind == "silu" else 1.6 * (g.abs() + 0.0447 * g.abs() ** 3)
    return (12 + 6 * z.clamp(max=90.0)) * U32


def check_gated(gate, up, dh, kind, out_layout=(0, 0), recompute=True):
    dt = gate.dtype
    rows, cols = gate.shape
    h, hbuf = placed(torch.full((rows, cols), NAN, dtype=dt, device=DEV), *out_layout)
    ck = fa.checkpoint_buffer(rows, cols, DEV)
    ck.codes.fill_(99)
    ck.scales.fill_(99.0)
    fa.fa_gated_forward(gate, up, h, ck, kind)
    g64, u64 = gate.double(), up.double()
    value, _ = R.act(g64, kind)
    assert_close(h, value * u64, ((value.abs() + 1e-30) * u64.abs() * act_terms(g64, kind)
                                  ).nan_to_num(posinf=0.0), "h")
    assert outside_is_nan(h, hbuf)
    plain = torch.full_like(h, NAN)
    fa.fa_gated_forward(gate, up, plain, None, kind)
    assert torch.equal(plain.nan_to_num(5.0), h.nan_to_num(5.0))
    # the checkpoint is exactly the stated FP32 rule's
    back = []
    for k, x in enumerate((gate, up)):
        codes, scales = R.quantise(x)
        assert torch.equal(ck.scales[k].nan_to_num(-1.0), scales.nan_to_num(-1.0))
        live = ~torch.isnan(scales).repeat_interleave(128, 1)
        assert torch.equal(ck.codes[k][live], codes[live])
        back.append(R.stored(codes, scales, cols))
    assert torch.equal(ck.values()[0].nan_to_num(5.0), back[0].nan_to_num(5.0))
    gq, uq = back[0].double(), back[1].double()
    a, da = R.act(gq, kind)
    d64 = dh.double()
    dx, dbuf = placed(torch.full((rows, 2 * cols), NAN, dtype=dt, device=DEV), *out_layout)
    again = torch.full_like(h, NAN) if recompute else None
    fa.fa_gated_backward(ck, dh, dx[:, :cols], dx[:, cols:], again, kind)
    t = act_terms(gq, kind)
    assert_close(dx[:, :cols], d64 * uq * da, ((d64 * uq).abs() * (1.2 + gq.abs()) * t).nan_to_num(),
                 "dgate")
    assert_close(dx[:, cols:], d64 * a, (d64.abs() * (a.abs() + 1e-30) * t).nan_to_num(), "dup")
    assert outside_is_nan(dx, dbuf)
    if recompute:
        assert_close(again, a * uq, ((a.abs() + 1e-30) * uq.abs() * t).nan_to_num(), "h again")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 127), (2, 128), (4, 129),
                                       (7, 255), (3, 257), (33, 1403), (16, 5632), (2, 16392)])
def test_gated_sizes_and_types(dt, kind, rows, cols):
    g = gen(rows * cols)
    x = randn(g, rows, 2 * cols, dtype=DTYPES[dt], sigma=2.0)  # halves of one projection
    check_gated(x[:, :cols], x[:, cols:], randn(g, rows, cols, dtype=DTYPES[dt], sigma=0.1), kind)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
def test_gated_layouts(dt, layout):
    g = gen(11)
    d = DTYPES[dt]
    for cols in (264, 515):
        gate, _ = placed(randn(g, 6, cols, dtype=d), *layout)
        up, _ = placed(randn(g, 6, cols, dtype=d), *layout)
        dh, _ = placed(randn(g, 6, cols, dtype=d), *layout)
        check_gated(gate, up, dh, "silu", layout, recompute=layout != (0, 0))


@pytest.mark.parametrize("dt", list(DTYPES))
def test_gated_blocks_of_every_kind(dt):
    """Zero, tiny, huge, one-sided, and non-finite blocks: the latter's gradients are NaN, so
    that a step made of them is skipped; the blocks beside them are not touched."""
    d = DTYPES[dt]
    g = gen(12)
    gate, up = randn(g, 9, 384, dtype=d), randn(g, 9, 384, dtype=d)
    dh = randn(g, 9, 384, dtype=d)
    gate[0] = 0.0
    gate[1, :128] = torch.finfo(d).tiny
    gate[2, 128:256] *= 1e-3
    up[3, :128] = torch.finfo(d).max if d != torch.float32 else 1e30
    gate[3] = 1e-4
    gate[4, 5] = 80.0
    gate[5, 5] = -80.0
    check_gated(gate, up, dh, "silu")
    check_gated(gate, up, dh, "gelu_tanh")
    gate[6, 200] = NAN
    up[7, 10] = INF
    gate[8, 383] = -INF
    ck = fa.checkpoint_buffer(9, 384, DEV)
    h = torch.empty_like(gate)
    fa.fa_gated_forward(gate, up, h, ck)
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    fa.fa_gated_backward(ck, dh, dg, du, None)
    bad = torch.zeros(9, 384, dtype=torch.bool, device=DEV)
    bad[6, 128:256] = bad[7, :128] = bad[8, 256:] = True
    assert torch.equal(torch.isnan(dg), bad)
    bad[3] = True  # its gradient may pass the type's range
    assert bool(torch.isfinite(dg[~bad]).all())


def test_gated_gradient_against_differences():
    """dgate and dup by central differences of the forward at the checkpoint's own values (FP32
    in, so that the perturbed inputs are not quantised)."""
    for kind in ("silu", "gelu_tanh"):
        g = gen(13)
        gate, up = randn(g, 4, 256), randn(g, 4, 256)
        dh = randn(g, 4, 256)
        h = torch.empty_like(gate)
        ck = fa.checkpoint_buffer(4, 256, DEV)
        fa.fa_gated_forward(gate, up, h, ck, kind)
        gq, uq = ck.values()
        dg, du = torch.empty_like(gate), torch.empty_like(gate)
        fa.fa_gated_backward(ck, dh, dg, du, None, kind)
        e = 2.0 ** -6
        for grad, moved in ((dg, 0), (du, 1)):
            at = []
            for s in (1, -1):
                x = [gq.clone(), uq.clone()]
                x[moved] += s * e
                out = torch.empty_like(gate)
                fa.fa_gated_forward(x[0], x[1], out, None, kind)
                at.append(out.double())
            slope = (at[0] - at[1]) / (2 * e) * dh.double()
            # |act'''| < 2.5 for both; h's FP32 error
            other = uq.double().abs() if moved == 0 else 0.0
            bound = dh.double().abs() * (e * e / 6 * 2.5 * other + 40 * U32 / e *
                                         (1 + at[0].abs()) + 8 * U32 / e)
            assert bool(((slope - grad.double()).abs() <= bound).all())


# ---- streams, graphs, sizes past 32 bits -------------------------------------------------

def test_on_a_side_stream_and_in_a_graph():
    """Every operator in one captured graph on a side stream: replays read the inputs anew."""
    g = gen(14)
    table = randn(g, 100, 64, dtype=torch.bfloat16)
    ids = torch.randint(0, 100, (9000,), device=DEV, generator=g)
    out = torch.empty(9000, 64, dtype=torch.bfloat16, device=DEV)
    dtable = torch.empty_like(table)
    scratch = fa.embedding_scratch(9000, 100, 64, DEV)
    logits, labels, off, ref = packed(15, [30, 20, 10, 40], 100)
    pref = fa.preference_buffers(100, 2, DEV)
    pol = fa.policy_buffers(100, DEV)
    old, adv = ref.clone(), randn(g, 100)
    dl, dl2 = torch.empty_like(logits), torch.empty_like(logits)
    gate, up, dh = (randn(g, 5, 200) for _ in range(3))
    h, dg, du = (torch.empty_like(gate) for _ in range(3))
    ck = fa.checkpoint_buffer(5, 200, DEV)

    def step():
        fa.fa_embedding_lookup(ids, table, out)
        fa.fa_embedding_gradient(ids, out, dtable, scratch)
        fa.fa_preference_loss(logits, labels, off, ref, pref)
        fa.fa_token_logprobs_gradient(logits, labels, pref.lse, pref.dlogp, dl)
        fa.fa_policy_loss(logits, labels, old, adv, pol, ref_logp=ref, kl_coef=0.1, dlogits=dl2)
        fa.fa_gated_forward(gate, up, h, ck)
        fa.fa_gated_backward(ck, dh, dg, du)

    results = [out, dtable, *pref, dl, *pol, dl2, h, dg, du]
    stream = torch.cuda.Stream(DEV)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for k in range(3):
        logits.mul_(-0.9)
        gate.mul_(1.1)
        table.mul_(-1)
        ids.copy_(ids.roll(7))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in results]
        step()
        torch.cuda.synchronize()
        for a, b in zip(replayed, results):
            assert torch.equal(a, b)


def test_lookup_and_gradient_past_32_bits():
    """2^31 and more elements: the last tokens' rows and gradients are right."""
    tokens, dim = 600_007, 4096
    ids = torch.arange(tokens, device=DEV, dtype=torch.int32) % 1000
    table = randn(gen(16), 1000, dim, dtype=torch.bfloat16)
    out = torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV)
    fa.fa_embedding_lookup(ids, table, out)
    for a in (0, 2 ** 31 // dim - 3, tokens - 10):
        assert torch.equal(out[a:a + 10], table[ids[a:a + 10].long()])
    # each row's gradient: count times the row (sums of equal BF16 values; exact bound below)
    dtable = torch.empty(1000, dim, device=DEV)
    scratch = fa.embedding_scratch(tokens, 1000, dim, DEV)
    fa.fa_embedding_gradient(ids, out, dtable, scratch)
    count = torch.bincount(ids.long(), minlength=1000).double()[:, None]
    want = table.double() * count
    assert_close(dtable, want, 610 * U32 * want.abs(), "gradient past 32 bits")


def test_logits_past_32_bits():
    tokens, vocab = 68_000, 32_000
    logits = torch.zeros(tokens, vocab, dtype=torch.bfloat16, device=DEV)
    labels = torch.full((tokens,), -100, device=DEV)
    rows = [0, 67_107, 67_108, 67_109, tokens - 1]  # around element 2^31 and at the end
    some = randn(gen(17), len(rows), vocab, dtype=torch.bfloat16, sigma=2.0)
    logits[rows] = some
    labels[rows] = 17
    lab = torch.full((len(rows),), 17, device=DEV)
    want, p = R.logprobs(some, lab, 1.0)
    b = fa.policy_buffers(tokens, DEV)
    zero = torch.zeros(tokens, device=DEV)
    old = zero.clone()
    old[rows] = want.float()
    adv = torch.ones(tokens, device=DEV)
    fa.fa_policy_loss(logits, labels, old, adv, b, dlogits=logits, clip_low=1.0, clip_high=10.0)
    assert b.count.item() == len(rows)
    grad = R.logprobs_gradient(some, lab, p, torch.full((len(rows),), -1 / len(rows), device=DEV), 1.0)
    assert_close(logits[rows], grad, 100 * U32 * grad.abs() + 10 * U32 * (grad.abs() > 0.01), "dlogits")
    assert not logits[1].any() and not logits[-2].any()


def test_gated_past_32_bits():
    rows, cols = 70_000, 32_768
    gate = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    h = torch.empty_like(gate)
    ck = fa.checkpoint_buffer(rows, cols, DEV)
    gate[-1] = 2.0
    gate[65_536] = 3.0
    fa.fa_gated_forward(gate, gate, h, ck)
    for r, x in ((0, 1.0), (65_535, 1.0), (65_536, 3.0), (rows - 1, 2.0)):
        want = torch.tensor(x * x / (1 + math.exp(-x))).to(torch.bfloat16).item()
        assert bool((h[r] == want).all())
    del gate
    dg = torch.empty_like(h)
    dh = torch.ones_like(h)
    fa.fa_gated_backward(ck, dh, dg, h)
    s = 1 / (1 + math.exp(-2.0))
    want = torch.tensor(2 * s * (1 + 2 * (1 - s))).to(torch.bfloat16).item()
    assert abs(dg[-1, 5].item() - want) <= 2 ** -7 * want and bool((dg[-1] == dg[-1, 0]).all())
    assert abs(h[-1, 5].item() - 2 * s) <= 2 ** -7 * 2 * s


# ---- refusals that need a device ----------------------------------------------------------

def test_refusals_on_the_device():
    x = torch.zeros(8, 16, device=DEV)
    ids = torch.zeros(8, dtype=torch.int64, device=DEV)

    def refused(status, call, *args, **kw):
        with pytest.raises(fa.FusedAdamWError) as e:
            call(*args, **kw)
        assert e.value.status == status

    refused(5, fa.fa_embedding_lookup, ids, x, x)                       # output is the table
    both = torch.zeros(8, 32, device=DEV)
    fa.fa_embedding_lookup(ids, both[:, :16], both[:, 16:])             # halves: no overlap
    refused(5, fa.fa_embedding_lookup, ids, both[:, :16], both[:, 8:24])
    scratch = fa.embedding_scratch(8, 8, 16, DEV)
    refused(3, fa.fa_embedding_gradient, ids, x, both[:, :16], scratch[:16])
    refused(7, fa.fa_embedding_gradient, ids, x, both[:, :16],
            torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[1:])
    lse, f = torch.zeros(8, 2, device=DEV), torch.zeros(8, device=DEV)
    refused(5, fa.fa_token_logprobs, x, ids, f, x.view(-1)[:16].view(8, 2))
    refused(5, fa.fa_token_logprobs_gradient, both[:, :16], ids, lse, f, both[:, 1:17])
    refused(4, fa.fa_token_logprobs, x, ids, f, lse, 0.0)
    b = fa.policy_buffers(8, DEV)
    refused(1, fa.fa_policy_loss, x, ids, f, f, b, kl_coef=0.1)         # no reference model
    refused(4, fa.fa_policy_loss, x, ids, f, f, b, clip_low=1.5)
    refused(5, fa.fa_policy_loss, x, ids, b.logp, f, b)                 # an output as an input
    p = fa.preference_buffers(8, 1, DEV)
    off = torch.tensor([0, 4, 8], device=DEV)
    refused(4, fa.fa_preference_loss, x, ids, off, f, p, beta=0.0)
    refused(4, fa.fa_preference_loss, x, ids, off, f, p, label_smoothing=0.6)
    ck = fa.checkpoint_buffer(8, 16, DEV)
    refused(5, fa.fa_gated_forward, x, x, x, ck)
    refused(5, fa.fa_gated_backward, ck, x, both[:, :16], both[:, :16], None)
    # on the host: refused, not computed
    host = torch.zeros(8, 16)
    with pytest.raises((fa.FusedAdamWError, ValueError)):
        fa.fa_embedding_lookup(ids, host, x)
    torch.cuda.synchronize()
    assert not x.any()
