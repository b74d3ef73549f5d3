"""The model-side operators without a GPU: sizes and refusals of the C ABI and of the binding,
and the tests' 64-bit reference pinned to torch's own functions.  No kernel is launched."""

import ctypes
import math

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import model_reference as R
from amsgrad_optimizer_step_gb300 import _lib, build
from amsgrad_optimizer_step_gb300._lib import FaLogits, FaPolicy, FaPreference

NAN, INF = math.nan, math.inf
FAKE = 0x10000  # never dereferenced: host checks come first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


# ---- sizes ---------------------------------------------------------------------------

def test_checkpoint_size():
    assert fa.fa_checkpoint_size(0, 100) == (0, 0)
    assert fa.fa_checkpoint_size(3, 1) == (2 * 3 * 128, 2 * 3)
    assert fa.fa_checkpoint_size(16384, 5632) == (2 * 16384 * 5632, 2 * 16384 * 44)
    for rows, cols in ((-1, 4), (4, -1), (2 ** 40, 2 ** 40)):
        with pytest.raises(fa.FusedAdamWError) as e:
            fa.fa_checkpoint_size(rows, cols)
        assert e.value.status == 3


def test_embedding_scratch_grows_with_its_arguments():
    sizes = [fa.fa_embedding_scratch(t, 32000, 2048) for t in (0, 1, 31, 33, 4096, 65536, 65537)]
    assert sizes == sorted(sizes)
    # the partial sums dominate: two FP32 rows for each 32 tokens
    assert sizes[5] < 65536 * (2048 * 4 * 2 / 32 + 24) + 32000 * 8
    for bad in ((-1, 10, 10), (10, -1, 10), (10, 10, -1), (2 ** 31, 10, 10), (10, 2 ** 31, 10)):
        with pytest.raises(fa.FusedAdamWError) as e:
            fa.fa_embedding_scratch(*bad)
        assert e.value.status == 3


# ---- refusals, in the library ------------------------------------------------------------

def lookup(lib, tokens=4, idt=1, tdt=0, vocab=8, dim=16, ld=16, scale=1.0, odt=0, out_ld=16):
    return lib.fa_embedding_lookup(tokens, FAKE, idt, FAKE, tdt, vocab, dim, ld, scale, FAKE, odt,
                                   out_ld, None)


def gradient(lib, tokens=4, idt=1, ddt=0, ld=16, scale=1.0, acc=0, tdt=0, vocab=8, dim=16,
             table_ld=16, scratch_bytes=1 << 30):
    return lib.fa_embedding_gradient(tokens, FAKE, idt, FAKE, ddt, ld, scale, -1, acc, FAKE, tdt,
                                     vocab, dim, table_ld, FAKE, scratch_bytes, None)


@pytest.mark.parametrize("call", [lookup, gradient])
def test_embedding_refusals(lib, call):
    assert call(lib, idt=2) == 2 and call(lib, tdt=3) == 2
    assert call(lib, tokens=-1) == 3 and call(lib, vocab=-1) == 3 and call(lib, dim=-1) == 3
    assert call(lib, ld=15) == 3
    assert call(lib, scale=NAN) == 4 and call(lib, scale=INF) == 4 and call(lib, scale=1e39) == 4
    assert call(lib, tokens=2 ** 31) == 3
    assert call(lib, dim=2 ** 23, **{"ld": 2 ** 23, ("out_ld" if call is lookup else "table_ld"):
                                     2 ** 23}) == 3


def test_embedding_empty_calls_launch_nothing(lib):
    assert lookup(lib, tokens=0) == 0 and lookup(lib, dim=0) == 0
    assert gradient(lib, vocab=0) == 0 and gradient(lib, dim=0) == 0
    assert gradient(lib, tokens=0, acc=1) == 0
    assert gradient(lib, acc=2) == 4
    assert gradient(lib, scratch_bytes=10) == 3


def record(**kw):
    base = dict(tokens=4, vocab=8, logits=FAKE, dtype=0, ld=8, labels=FAKE, ltype=1,
                logit_scale=1.0)
    base.update(kw)
    return FaLogits(**base)


BAD_LOGITS = [(dict(dtype=5), 2), (dict(ltype=2), 2), (dict(tokens=-1), 3), (dict(vocab=0), 3),
              (dict(ld=7), 3), (dict(tokens=2 ** 31), 3), (dict(logit_scale=0.0), 4),
              (dict(logit_scale=-1.0), 4), (dict(logit_scale=NAN), 4), (dict(logit_scale=1e5), 4),
              (dict(logit_scale=1e-5), 4)]


@pytest.mark.parametrize("bad,status", BAD_LOGITS)
def test_logits_refusals(lib, bad, status):
    x = ctypes.byref(record(**bad))
    p = FaPreference(pairs=1, seq_offsets=FAKE, ref_logp=FAKE, beta=0.1, loss=FAKE)
    q = FaPolicy(old_logp=FAKE, advantages=FAKE, clip_low=0.2, clip_high=0.2, grad_scale=1.0)
    assert lib.fa_token_logprobs(x, FAKE, FAKE, None) == status
    assert lib.fa_token_logprobs_gradient(x, FAKE, FAKE, 1.0, None, FAKE, 8, None) == status
    assert lib.fa_preference_loss(x, ctypes.byref(p), None) == status
    assert lib.fa_policy_loss(x, ctypes.byref(q), None) == status


def test_logits_records_may_not_be_missing(lib):
    x = ctypes.byref(record())
    assert lib.fa_token_logprobs(None, FAKE, FAKE, None) == 1
    assert lib.fa_preference_loss(x, None, None) == 1
    assert lib.fa_policy_loss(x, None, None) == 1
    empty = ctypes.byref(record(tokens=0, vocab=0, ld=0))
    assert lib.fa_token_logprobs(empty, None, None, None) == 0
    assert lib.fa_token_logprobs_gradient(x, FAKE, FAKE, 1.0, None, FAKE, 7, None) == 3
    assert lib.fa_token_logprobs_gradient(x, FAKE, FAKE, INF, None, FAKE, 8, None) == 4


@pytest.mark.parametrize("bad,status", [
    (dict(pairs=-1), 3), (dict(beta=0.0), 4), (dict(beta=NAN), 4), (dict(beta=INF), 4),
    (dict(label_smoothing=-0.1), 4), (dict(label_smoothing=0.6), 4),
    (dict(label_smoothing=NAN), 4), (dict(average=2), 4)])
def test_preference_refusals(lib, bad, status):
    kw = dict(pairs=1, seq_offsets=FAKE, ref_logp=FAKE, beta=0.1, loss=FAKE)
    kw.update(bad)
    assert lib.fa_preference_loss(ctypes.byref(record()), ctypes.byref(FaPreference(**kw)),
                                  None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(clip_low=-0.1), 4), (dict(clip_low=1.1), 4), (dict(clip_low=NAN), 4),
    (dict(clip_high=-1.0), 4), (dict(clip_high=INF), 4), (dict(kl_coef=-1.0), 4),
    (dict(kl_coef=NAN), 4), (dict(denominator=-1.0), 4), (dict(denominator=1e-60), 4),
    (dict(grad_scale=INF), 4), (dict(kl_coef=0.1, ref_logp=None), 1),
    (dict(dlogits=FAKE, dlogits_ld=7), 3)])
def test_policy_refusals(lib, bad, status):
    kw = dict(old_logp=FAKE, advantages=FAKE, ref_logp=FAKE, clip_low=0.2, clip_high=0.2,
              grad_scale=1.0, summary=FAKE)
    kw.update(bad)
    assert lib.fa_policy_loss(ctypes.byref(record()), ctypes.byref(FaPolicy(**kw)), None) == status


def test_gated_refusals(lib):
    def forward(rows=4, cols=8, ld=8, dtype=0, act=0, codes=FAKE, scales=FAKE):
        return lib.fa_gated_forward(rows, cols, FAKE, ld, FAKE, 8, dtype, act, FAKE, 8, codes,
                                    scales, None)

    def backward(rows=4, cols=8, ld=8, dtype=0, act=0, h=FAKE, h_ld=8):
        return lib.fa_gated_backward(rows, cols, FAKE, FAKE, act, FAKE, ld, dtype, FAKE, 8, FAKE, 8,
                                     h, h_ld, None)

    for call in (forward, backward):
        assert call(dtype=3) == 2 and call(act=2) == 4
        assert call(rows=-1) == 3 and call(cols=-1) == 3 and call(ld=7) == 3
        assert call(rows=0) == 0 and call(cols=0, ld=0) == 0  # nothing launched
    assert forward(codes=None) == 1 and forward(scales=None) == 1
    assert backward(h_ld=7) == 3
    assert backward(rows=0, h=None, h_ld=0) == 0


def test_host_memory_is_refused(lib):
    """CPU tensors reach the library and are refused: there is no CPU fallback."""
    table, out = torch.zeros(4, 8), torch.zeros(2, 8)
    with pytest.raises(fa.FusedAdamWError) as e:
        fa.fa_embedding_lookup(torch.zeros(2, dtype=torch.int64), table, out, stream=0)
    assert e.value.status in (6, 9)  # not device memory / no CUDA device here


# ---- refusals, in the binding -------------------------------------------------------------

def test_binding_refusals():
    table, out = torch.zeros(4, 8), torch.zeros(2, 8)
    ids = torch.zeros(2, dtype=torch.int64)
    bad = [
        lambda: fa.fa_embedding_lookup(ids, table, torch.zeros(3, 8), stream=0),
        lambda: fa.fa_embedding_lookup(ids, table, torch.zeros(2, 16)[:, ::2], stream=0),
        lambda: fa.fa_embedding_lookup(ids, table, torch.zeros(8).expand(2, 8), stream=0),
        lambda: fa.fa_embedding_lookup(torch.zeros(4, dtype=torch.int64)[::2], table, out, stream=0),
        lambda: fa.fa_embedding_lookup(ids, torch.zeros(8), out, stream=0),
        lambda: fa.fa_gated_forward(out, torch.zeros(2, 9), out, None, stream=0),
        lambda: fa.fa_gated_forward(out, out, out, None, "relu", stream=0),
        lambda: fa.fa_gated_backward(fa.checkpoint_buffer(2, 9, "cpu"), out, out, out, stream=0),
        lambda: fa.fa_token_logprobs(out, torch.zeros(3, dtype=torch.int64), out[:, 0], stream=0),
        lambda: fa.fa_token_logprobs(out, ids, torch.zeros(3), stream=0),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    wrong_type = [
        lambda: fa.fa_embedding_lookup(ids.float(), table, out, stream=0),
        lambda: fa.fa_embedding_lookup(ids, table.double(), out, stream=0),
        lambda: fa.fa_gated_forward(out, out.half(), out, None, stream=0),
        lambda: fa.fa_token_logprobs(out, ids, torch.zeros(2).double(), stream=0),
        lambda: fa.fa_token_logprobs_gradient(out, ids, torch.zeros(2, 2), torch.zeros(2),
                                              out.half(), stream=0),
    ]
    for call in wrong_type:
        with pytest.raises(TypeError):
            call()


def test_layers_refuse_odd_shapes():
    from amsgrad_optimizer_step_gb300 import layers
    with pytest.raises(ValueError):
        layers.gated_activation(torch.zeros(2, 7))
    with pytest.raises(ValueError):
        layers.preference_loss(torch.zeros(2, 7), torch.zeros(2, dtype=torch.int64),
                               torch.zeros(2, dtype=torch.int64), torch.zeros(2))


# ---- the 64-bit reference, pinned ---------------------------------------------------------

def test_reference_losses_are_torch_functions():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 17, generator=g, dtype=torch.float64)
    y = torch.randint(0, 17, (9,), generator=g)
    logp, p = R.logprobs(x, y, 0.7)
    assert torch.allclose(logp, -torch.nn.functional.cross_entropy(0.7 * x, y, reduction="none"),
                          rtol=1e-13)
    xg = x.clone().requires_grad_()
    w = torch.randn(9, generator=g, dtype=torch.float64)
    (torch.log_softmax(0.7 * xg, 1).gather(1, y[:, None])[:, 0] * w).sum().backward()
    assert torch.allclose(R.logprobs_gradient(x, y, p, w, 0.7), xg.grad, rtol=1e-12, atol=1e-15)

    ok = torch.rand(9, generator=g) < 0.8
    ref = torch.randn(9, generator=g, dtype=torch.float64)
    lp = torch.randn(9, generator=g, dtype=torch.float64).requires_grad_()
    for average in (False, True):
        loss, _, rewards, dlogp = R.preference(lp.detach(), ref, ok, [0, 2, 5, 5, 9], 0.4, 0.1,
                                               average)
        ratio = (lp - ref) * ok
        s = [ratio[a:b].sum() / (max(1, int(ok[a:b].sum())) if average else 1)
             for a, b in ((0, 2), (2, 5), (5, 5), (5, 9))]
        z = 0.4 * torch.stack([s[0] - s[1], s[2] - s[3]])
        want = (-0.9 * torch.nn.functional.logsigmoid(z) -
                0.1 * torch.nn.functional.logsigmoid(-z)).mean()
        assert torch.allclose(loss, want)
        assert torch.allclose(dlogp, torch.autograd.grad(want, lp)[0], rtol=1e-12)

    old, adv = lp.detach() + 0.3 * torch.randn(9, generator=g, dtype=torch.float64), w
    out = R.policy(lp.detach(), ok, old, adv, ref, w.abs(), 0.2, 0.3, 0.1, 2.0)
    r, d = torch.exp(lp - old), ref - lp
    per = -torch.minimum(r * adv, r.clamp(0.8, 1.3) * adv) + 0.1 * (torch.exp(d) - d - 1)
    want = (w.abs() * per * ok).sum() / 2.0
    assert torch.allclose(out["loss"], want)
    assert torch.allclose(out["dlogp"], torch.autograd.grad(want, lp)[0], rtol=1e-10, atol=1e-14)


def test_reference_activations_are_torch_functions():
    x = torch.linspace(-12, 12, 401, dtype=torch.float64).requires_grad_()
    for kind, f in (("silu", torch.nn.functional.silu),
                    ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh"))):
        value, slope = R.act(x.detach(), kind)
        y = f(x)
        assert torch.allclose(value, y, rtol=1e-9, atol=1e-14)
        assert torch.allclose(slope, torch.autograd.grad(y.sum(), x)[0], rtol=1e-9, atol=1e-12)


def test_reference_quantisation_obeys_its_bound():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 300, generator=g) * torch.exp(3 * torch.randn(5, 1, generator=g))
    x[0, :128] = 0.0
    x[1, :128] = 1e-38
    x[2, 130] = INF
    codes, scales = R.quantise(x)
    assert codes.shape == (5, 384) and scales.shape == (5, 3)
    assert not codes[0, :128].any() and scales[0, 0] == 0 and scales[1, 0] == 0
    assert torch.isnan(scales[2, 1]) and not codes[:, 300:].any()
    back = R.stored(codes, scales, 300)
    top = torch.nn.functional.pad(x, (0, 84)).view(5, 3, 128).abs().amax(2).repeat_interleave(128, 1)
    fine = torch.isfinite(back) & (top[:, :300] >= 2.0 ** -100)
    err = (back - x).abs()[fine]
    assert bool((err <= top[:, :300][fine] * (1 / 254 + 2.0 ** -21)).all())


def test_reference_embedding_is_torch_embedding():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(11, 6, generator=g, dtype=torch.float64).requires_grad_()
    ids = torch.randint(0, 11, (40,), generator=g)
    y = torch.nn.functional.embedding(ids, w, padding_idx=4) * 2.5
    assert torch.equal(R.lookup(ids, w.detach(), 2.5), y.detach())
    dy = torch.randn(40, 6, generator=g, dtype=torch.float64)
    grad, mag, count = R.embedding_gradient(ids, dy, 11, 2.5, 4)
    assert torch.allclose(grad, torch.autograd.grad(y, w, dy)[0])
    assert count[4] == 0 and int(count.sum()) == int((ids != 4).sum())
