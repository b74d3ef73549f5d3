"""The paths that large and odd sizes take through the model-side operators, against 64 bits.

Embedding gradients of tables above 16 MB (rows without a token are found by a claim per id),
of tokens that need a full cluster or several chunks, of vocabularies that take a third digit;
lookups and gradients of rows at any address in every pair of types; policy rows that a cluster
shares while the labels are counted by a kernel of their own.  Each runs through the normal and
the bounds-checked library.  Tolerances are those of the operators' other tests.
"""

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import model_reference as R
import test_gpu_model_ops as M
from amsgrad_optimizer_step_gb300 import _lib, build
from model_reference import DTYPES, U32, assert_close
from test_gpu_model_ops import DEV, NAN, gen, placed, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=["normal", "checked"], autouse=True)
def library(request):
    build.build()
    if request.param == "normal":
        yield request.param
        return
    lib = _lib.open_library(build.build(variant="checked"))
    with _lib.using(lib):
        yield request.param


@pytest.fixture(autouse=True)
def no_access_out_of_range(library):
    if library == "checked":
        fa.fa_bounds_check_report(clear=True)
    yield
    if library == "checked":
        torch.cuda.synchronize()
        assert fa.fa_bounds_check_report() == (True, 0)


# ---- embedding gradient --------------------------------------------------------------

def gradient(ids, dout, vocab, tdt, words, padding=-1, layout=(0, 0)):
    """The gradient into a table of NaN, with a scratch that holds ``words`` (32-bit)."""
    dtable, buf = placed(torch.full((vocab, dout.shape[1]), NAN, dtype=tdt, device=DEV), *layout)
    scratch = fa.embedding_scratch(ids.numel(), vocab, dout.shape[1], DEV)
    scratch[:scratch.numel() // 4 * 4].view(torch.int32).fill_(words)
    fa.fa_embedding_gradient(ids, dout, dtable, scratch, 0.5, padding)
    assert M.outside_is_nan(dtable, buf)
    return dtable


def check_gradient(ids, dout, vocab, tdt, words=0, padding=-1, layout=(0, 0)):
    got = gradient(ids, dout, vocab, tdt, words, padding, layout)
    want, mag, count = R.embedding_gradient(ids, dout, vocab, 0.5, padding)
    assert_close(got, want, (count[:, None] + 2) * U32 * mag, "embedding gradient")
    assert not got[count == 0].any()
    return got


def skewed(seed, tokens, vocab, outside=0.05):
    """Zipf ids, a few of them outside the table on either side."""
    g = gen(seed)
    ids = M.zipf(g, tokens, vocab)
    u = torch.rand(tokens, device=DEV, generator=g)
    ids[u < outside] = vocab + 3
    ids[u < outside / 2] = -100
    return ids


# Above 16 MB: min(tokens, vocab) * dim * element size > 2^24
LARGE = [("bf16", 9001, 20011, 1024), ("f16", 16800, 17011, 515), ("f32", 4501, 6007, 1032),
         ("bf16", 70_001, 9001, 1000)]


@pytest.mark.parametrize("dt,tokens,vocab,dim", LARGE)
@pytest.mark.parametrize("layout", [(0, 0), (8, 8), (3, 1)])
def test_large_tables(dt, tokens, vocab, dim, layout):
    """Dense, padded and misaligned tables; every stale word a scratch may hold: 0, a token that
    exists, the last one, one past it, all bits."""
    assert min(tokens, vocab) * dim * DTYPES[dt].itemsize > 2 ** 24
    ids = skewed(tokens, tokens, vocab)
    dout = randn(gen(1), tokens, dim, dtype=DTYPES[dt])
    for words in (0, 17, tokens - 1, tokens, -1):
        check_gradient(ids, dout, vocab, DTYPES[dt], words, layout=layout)


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_large_tables_leave_the_padding_row_zero(itype):
    """A padding id that occurs often, its stale claim included: no gradient, and zeros."""
    ids = skewed(2, 9001, 20011).to(itype)
    ids[::3] = 20010
    ids[5::7] = 0
    dout = randn(gen(3), 9001, 1024, dtype=torch.bfloat16)
    dout[::3] = NAN
    got = check_gradient(ids, dout, 20011, torch.bfloat16, words=3, padding=20010)
    assert not got[20010].any()


def test_large_tables_with_one_id_or_none():
    dout = randn(gen(4), 9001, 1024, dtype=torch.bfloat16)
    same = torch.full((9001,), 20010, device=DEV)
    check_gradient(same, dout, 20011, torch.bfloat16)
    got = gradient(torch.full_like(same, -1), dout, 20011, torch.bfloat16, 5)
    assert not got.any()
    got = gradient(same, dout, 20011, torch.bfloat16, 5, padding=20010)
    assert not got.any()


def test_large_tables_again_in_the_same_scratch():
    """Batch after batch in one scratch and one captured graph: the claims that an earlier batch
    left, of ids that the next one has not, count for nothing."""
    tokens, vocab, dim = 9001, 20011, 1024
    ids = skewed(5, tokens, vocab)
    dout = randn(gen(6), tokens, dim, dtype=torch.bfloat16)
    dtable = torch.empty(vocab, dim, dtype=torch.bfloat16, device=DEV)
    scratch = fa.embedding_scratch(tokens, vocab, dim, DEV)
    run = lambda: fa.fa_embedding_gradient(ids, dout, dtable, scratch, 0.5)  # noqa: E731
    stream = torch.cuda.Stream(DEV)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for seed in range(3):
        ids.copy_(skewed(10 + seed, tokens, vocab))
        dtable.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, mag, count = R.embedding_gradient(ids, dout, vocab, 0.5)
        assert_close(dtable, want, (count[:, None] + 2) * U32 * mag, "embedding gradient")


KINDS = {"zipf": lambda g, n, v: skewed(n, n, v), "same": lambda g, n, v: torch.full((n,), v - 1,
                                                                                     device=DEV),
         "spread": lambda g, n, v: torch.randint(-3, v + 3, (n,), device=DEV, generator=g),
         "falling": lambda g, n, v: (v - 1 - torch.arange(n, device=DEV) % v)}


@pytest.mark.parametrize("tokens", [32_769, 36_865, 53_249, 65_535, 65_536, 65_537, 131_072,
                                    131_075, 200_003])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("vocab", [1009, 131_072])
def test_many_tokens(tokens, kind, vocab):
    """Clusters of 9 to 16 CTAs, and several chunks (the last one of a few tokens too), with a
    row of its own for every token; 64-bit items above 65535 ids."""
    g = gen(tokens + vocab)
    ids = KINDS[kind](g, tokens, vocab)
    dout = randn(g, tokens, 24, dtype=torch.bfloat16)
    before = randn(g, vocab, 24)
    M.check_embedding_grad(ids, dout, vocab, torch.float32, scale=0.5)
    M.check_embedding_grad(ids, dout, vocab, torch.float32, scale=0.5, padding=vocab // 2,
                           before=before)


@pytest.mark.parametrize("vocab", [262_143, 262_144, 300_007])
@pytest.mark.parametrize("tokens", [33, 9000, 70_001])
def test_vocabularies_of_three_digits(vocab, tokens):
    g = gen(vocab + tokens)
    ids = torch.randint(0, vocab, (tokens,), device=DEV, generator=g)
    ids[:4] = torch.tensor([0, vocab - 1, vocab - 1, 0], device=DEV)
    ids[9::11] = -1
    M.check_embedding_grad(ids, randn(g, tokens, 8), vocab, torch.float32)
    M.check_embedding_grad(M.zipf(g, tokens, vocab), randn(g, tokens, 12), vocab, torch.float32)


@pytest.mark.parametrize("ddt", list(DTYPES))
@pytest.mark.parametrize("tdt", list(DTYPES))
@pytest.mark.parametrize("dim", [1, 67, 515])
@pytest.mark.parametrize("layout", [(0, 0), (3, 1)])
def test_gradients_of_odd_rows_in_all_types(ddt, tdt, dim, layout):
    g = gen(dim)
    ids = skewed(dim, 900, 61)  # long runs as well
    dout, _ = placed(randn(g, 900, dim, dtype=DTYPES[ddt]), *layout)
    before = randn(g, 61, dim, dtype=DTYPES[tdt])
    M.check_embedding_grad(ids, dout, 61, DTYPES[tdt], layout=layout)
    M.check_embedding_grad(ids, dout, 61, DTYPES[tdt], layout=layout, before=before, padding=5)


# ---- lookup ----------------------------------------------------------------------------

@pytest.mark.parametrize("tdt", list(DTYPES))
@pytest.mark.parametrize("odt", list(DTYPES))
@pytest.mark.parametrize("dim", [1, 5, 12, 67, 515, 2047])
@pytest.mark.parametrize("layouts", [((0, 0), (0, 0)), ((3, 1), (0, 0)), ((0, 0), (5, 3)),
                                     ((1, 2), (3, 1))])
def test_lookups_at_any_address_in_all_types(tdt, odt, dim, layouts):
    g = gen(dim)
    table, _ = placed(randn(g, 50, dim, dtype=DTYPES[tdt]), *layouts[0])
    ids = torch.randint(-2, 52, (37,), device=DEV, generator=g, dtype=torch.int32)
    ids[:2] = torch.tensor([0, 49], device=DEV)
    out, buf = placed(torch.full((37, dim), NAN, dtype=DTYPES[odt], device=DEV), *layouts[1])
    fa.fa_embedding_lookup(ids, table, out, 3.3)
    want = R.lookup(ids, table, 3.3)
    assert_close(out, want, 2 * U32 * want.abs(), f"{tdt}->{odt}")
    assert M.outside_is_nan(out, buf)


# ---- policy loss ------------------------------------------------------------------------

@pytest.mark.parametrize("dt,tokens,vocab", [
    ("f32", 2050, 16_400),   # two CTAs a row, more than eight labels a thread
    ("f32", 2051, 16_403),
    ("bf16", 2050, 32_776),
    ("f32", 290, 2_060),     # two CTAs of one warp
    ("f16", 297, 4_111),
])
def test_rows_of_a_cluster_with_counted_labels(dt, tokens, vocab):
    """The divisor comes from the kernel before the rows', which clusters of CTAs share; in
    place, and for a gradient taken later, too."""
    logits, labels, old, adv, ref, w = M.rollout(tokens + vocab, tokens, vocab, dt)
    M.check_policy(logits, labels, old, adv, ref, kl=0.05)
    M.check_policy(logits.clone(), labels, old, adv, ref, w, kl=0.1, in_place=True)
    # the gradient taken later, from a pass that splits the rows otherwise
    logp, p = R.logprobs(logits, labels, 1.0)
    ratio = torch.exp(logp - old.double())
    for edge in (0.8, 1.28):  # a ratio at the clip's edge may fall either way: moved off it
        old = torch.where((ratio / edge - 1).abs() < 1e-4, old + 3e-4, old)
    ratio, slope = torch.exp(logp - old.double()), torch.exp(ref.double() - logp)
    ok = R.counted(labels, vocab)
    want = R.policy(logp, ok, old, adv, ref, w, 0.2, 0.28, 0.1, 0.0)
    lse = torch.full((tokens, 2), NAN, device=DEV)
    dlogp = torch.full((tokens,), NAN, device=DEV)
    b, _ = M.run_policy(logits, labels, old, adv, grad=False, ref_logp=ref, kl_coef=0.1,
                        weights=w, clip_high=0.28, lse=lse, dlogp=dlogp)
    out = torch.full_like(logits, NAN)
    fa.fa_token_logprobs_gradient(logits, labels, lse, dlogp, out)
    # a log-probability's error, with the roundings of its differences, through both slopes
    err = M.logp_error(logits, 1.0) + 3 * U32 * (logp.abs() + old.abs() + ref.abs())
    coef_err = w / want["count"] * ((err + 8 * U32) * ratio * adv.abs() + 0.1 * (
        slope * err + 8 * U32 * (slope - 1).abs()))
    coef_err = torch.where(ok, coef_err.double(), 0.0)
    assert_close(b.logp, logp, err, "logp")
    assert_close(dlogp, want["dlogp"], coef_err, "dlogp")
    grad = R.logprobs_gradient(logits, labels, p, want["dlogp"], 1.0)
    c = want["dlogp"].abs()
    fp = c[:, None] * p * (2 * err[:, None] + 10 * U32) + coef_err[:, None]
    y = torch.where(ok, labels, 0).long()[:, None]
    fp.scatter_add_(1, y, 8 * U32 * c[:, None])
    assert_close(out, grad, torch.where(ok[:, None], fp, 0.0), "dlogits")
