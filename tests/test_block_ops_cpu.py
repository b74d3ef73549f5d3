"""The residual blocks' operators without a GPU: sizes and refusals of the C ABI and of the binding,
and the tests' 64-bit reference pinned to published vectors and to torch's own functions.  No
kernel is launched."""

import ctypes
import math

import numpy as np
import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import block_reference as B
from amsgrad_optimizer_step_gb300 import _lib, build
from amsgrad_optimizer_step_gb300._lib import (FaDropoutKey, FaJoin, FaJoinGradient, FaRouter,
                                               FaRouting)

NAN, INF = math.nan, math.inf
FAKE = 0x10000  # never dereferenced: host checks come first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


# ---- sizes ---------------------------------------------------------------------------

def test_scratch_sizes():
    assert fa.fa_block_join_scratch(0, 512, 1) == 0 and fa.fa_block_join_scratch(5, 0, 1) == 0
    # the columns' sums of a CTA are FP32 rows, twice as many with a gate
    assert fa.fa_block_join_scratch(1, 512, 0) == 2 * 512 * 4
    assert fa.fa_block_join_scratch(1, 513, 1) == 4 * 520 * 4
    assert fa.fa_block_join_scratch(10 ** 6, 2048, 1) < 16 << 20
    for bad in ((-1, 8, 1), (8, -1, 1), (8, 8, -1), (2 ** 31, 8, 1), (8, 16385, 1)):
        with pytest.raises(fa.FusedAdamWError) as e:
            fa.fa_block_join_scratch(*bad)
        assert e.value.status == 3
    assert fa.fa_route_scratch(1, 64) <= fa.fa_route_scratch(10 ** 6, 64) < 1 << 20
    for bad in ((-1, 8), (8, -1), (2 ** 31, 8), (8, 1025)):
        with pytest.raises(fa.FusedAdamWError) as e:
            fa.fa_route_scratch(*bad)
        assert e.value.status == 3


# ---- refusals, in the library ------------------------------------------------------------

def dropout(lib, rows=4, cols=8, ld=8, dtype=0, p=0.1, key=True, out_ld=8):
    k = FaDropoutKey(p, 1, 2, None)
    return lib.fa_dropout(rows, cols, FAKE, ld, dtype, ctypes.byref(k) if key else None, FAKE,
                          out_ld, None)


def test_dropout_refusals(lib):
    assert dropout(lib, dtype=3) == 2
    assert dropout(lib, rows=-1) == 3 and dropout(lib, cols=-1) == 3
    assert dropout(lib, ld=7) == 3 and dropout(lib, out_ld=7) == 3
    assert dropout(lib, rows=2 ** 31) == 3
    for p in (-0.1, 1.1, NAN, INF):
        assert dropout(lib, p=p) == 4
    assert dropout(lib, key=False) == 1
    assert dropout(lib, rows=0) == 0 and dropout(lib, cols=0) == 0  # nothing launched


def record(**kw):
    base = dict(rows=4, cols=8, dtype=2, stream_dtype=2, weight_dtype=2, post_norm=1, branch=FAKE,
                branch_ld=8, post_weight=FAKE, pre_weight=FAKE, gate=FAKE, gate_ld=8, groups=2,
                residual_scale=1.0, branch_scale=1.0, eps=1e-6, weight_offset=0.0, dropout=None)
    base.update(kw)
    return FaJoin(**base)


BAD_JOINS = [
    (dict(dtype=3), 2), (dict(stream_dtype=1), 2), (dict(weight_dtype=1), 2),
    (dict(dtype=0, stream_dtype=2, weight_dtype=0), 2), (dict(rows=-1), 3), (dict(cols=-1), 3),
    (dict(rows=2 ** 31), 3), (dict(cols=16385, branch_ld=16385, gate_ld=16385), 3),
    (dict(branch_ld=7), 3), (dict(gate_ld=7), 3), (dict(groups=3), 3), (dict(groups=0), 3),
    (dict(post_norm=2), 4), (dict(eps=0.0), 4), (dict(eps=-1.0), 4), (dict(eps=NAN), 4),
    (dict(eps=1e-60), 4), (dict(eps=INF), 4), (dict(residual_scale=NAN), 4),
    (dict(branch_scale=INF), 4), (dict(weight_offset=1e39), 4)]


@pytest.mark.parametrize("bad,status", BAD_JOINS)
def test_join_refusals(lib, bad, status):
    j = record(**bad)
    g = FaJoinGradient(dout=FAKE, dout_ld=2 ** 20, dresidual=FAKE, dresidual_ld=2 ** 20)
    assert lib.fa_block_join(ctypes.byref(j), FAKE, 2 ** 20, FAKE, 2 ** 20, None, 0, None, None,
                             None) == status
    assert lib.fa_block_join_gradient(ctypes.byref(j), ctypes.byref(g), None) == status


def test_join_records_and_results(lib):
    j = ctypes.byref(record())
    call = lib.fa_block_join
    assert call(None, FAKE, 8, FAKE, 8, FAKE, 8, None, None, None) == 1
    assert call(j, FAKE, 7, FAKE, 8, FAKE, 8, None, None, None) == 3
    assert call(j, FAKE, 8, FAKE, 7, FAKE, 8, None, None, None) == 3
    assert call(j, FAKE, 8, FAKE, 8, FAKE, 7, None, None, None) == 3
    key = FaDropoutKey(2.0, 0, 0, None)
    dropped = record(dropout=ctypes.addressof(key))
    assert call(ctypes.byref(dropped), FAKE, 8, FAKE, 8, FAKE, 8, None, None, None) == 4
    empty = ctypes.byref(record(rows=0, gate=None))
    assert call(empty, None, 8, None, 8, None, 8, None, None, None) == 0  # nothing launched

    def gradient(j=None, **kw):
        return lib.fa_block_join_gradient(ctypes.byref(record(**(j or {}))),
                                          ctypes.byref(FaJoinGradient(**kw)), None)

    assert lib.fa_block_join_gradient(j, None, None) == 1
    # a gradient of what is not there
    assert gradient(dict(branch=None), dbranch=FAKE, dbranch_ld=8) == 1
    assert gradient(dict(post_weight=None), dpost_weight=FAKE) == 1
    assert gradient(dict(post_norm=0), dpost_weight=FAKE) == 1
    assert gradient(dpre_weight=FAKE) == 1  # without dnormed there is no second norm
    assert gradient(dict(gate=None), dgate=FAKE, dgate_ld=8) == 1
    for name in ("out", "dout", "dnormed", "dresidual", "dbranch", "dgate"):
        assert gradient(**{name: FAKE, name + "_ld": 7}) == 3
    assert gradient(dgate=FAKE, dgate_ld=8, scratch=FAKE, scratch_bytes=10) == 3
    assert gradient(dict(cols=0, branch_ld=0, gate_ld=0)) == 0


def router(**kw):
    base = dict(tokens=4, experts=8, logits=FAKE, dtype=0, ld=8, counted=None, top_k=2,
                renormalise=1, weight_scale=1.0, balance_coef=0.01, z_coef=0.0)
    base.update(kw)
    return FaRouter(**base)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=4), 2), (dict(tokens=-1), 3), (dict(tokens=2 ** 31), 3), (dict(experts=0, ld=8), 3),
    (dict(experts=1025, ld=1025), 3), (dict(ld=7), 3), (dict(top_k=0), 3), (dict(top_k=9), 3),
    (dict(experts=64, ld=64, top_k=33), 3), (dict(renormalise=2), 4), (dict(weight_scale=0.0), 4),
    (dict(weight_scale=NAN), 4), (dict(weight_scale=INF), 4), (dict(weight_scale=1e-40), 4),
    (dict(balance_coef=-1.0), 4), (dict(balance_coef=NAN), 4), (dict(z_coef=-1.0), 4),
    (dict(z_coef=INF), 4)])
def test_router_refusals(lib, bad, status):
    x = ctypes.byref(router(**bad))
    r = FaRouting(chosen=FAKE, weights=FAKE, lse=FAKE, counts=FAKE, mean_prob=FAKE, summary=FAKE,
                  scratch=FAKE, scratch_bytes=1 << 30)
    assert lib.fa_route(x, ctypes.byref(r), None) == status
    assert lib.fa_route_gradient(x, ctypes.byref(r), None, None, FAKE, 2 ** 20, None) == status


def test_router_records(lib):
    x = ctypes.byref(router())
    part = FaRouting(chosen=FAKE, weights=FAKE, summary=FAKE)  # all that a loss needs, or nothing
    small = FaRouting(chosen=FAKE, weights=FAKE, lse=FAKE, counts=FAKE, mean_prob=FAKE,
                      summary=FAKE, scratch=FAKE, scratch_bytes=8)
    assert lib.fa_route(None, ctypes.byref(part), None) == 1
    assert lib.fa_route(x, None, None) == 1
    assert lib.fa_route(x, ctypes.byref(part), None) == 1
    assert lib.fa_route(x, ctypes.byref(small), None) == 3
    assert lib.fa_route_gradient(x, None, None, None, FAKE, 8, None) == 1
    assert lib.fa_route_gradient(x, ctypes.byref(small), None, None, FAKE, 7, None) == 3
    none = ctypes.byref(router(tokens=0))
    assert lib.fa_route(none, ctypes.byref(FaRouting()), None) == 0
    assert lib.fa_route_gradient(none, ctypes.byref(FaRouting()), None, None, None, 8, None) == 0


def test_host_memory_is_refused(lib):
    """CPU tensors reach the library and are refused: there is no CPU fallback."""
    x = torch.zeros(4, 8)
    calls = [lambda: fa.fa_dropout(x, torch.zeros(4, 8), fa.Dropout(0.1), stream=0),
             lambda: fa.fa_block_join(None, x, x.clone(), torch.zeros(4, 8), stream=0),
             lambda: fa.fa_route(x, fa.route_buffers(4, 8, 2, "cpu"), stream=0)]
    for call in calls:
        with pytest.raises(fa.FusedAdamWError) as e:
            call()
        assert e.value.status in (6, 9)  # not device memory / no CUDA device here


# ---- refusals, in the binding -------------------------------------------------------------

def test_binding_refusals():
    x, out, w = torch.zeros(2, 8), torch.zeros(2, 8), torch.ones(8)
    half = out.half()
    b = fa.route_buffers(2, 8, 2, "cpu")
    bad = [
        lambda: fa.fa_dropout(x, torch.zeros(3, 8), fa.Dropout(0.1), stream=0),
        lambda: fa.fa_dropout(x, torch.zeros(8).expand(2, 8), fa.Dropout(0.1), stream=0),
        lambda: fa.fa_dropout(torch.zeros(8), out, fa.Dropout(0.1), stream=0),
        lambda: fa.fa_dropout(x, out, fa.Dropout(0.1, counter=torch.zeros(2, dtype=torch.int64)),
                              stream=0),
        lambda: fa.fa_block_join(None, x, torch.zeros(2, 9), out, stream=0),
        lambda: fa.fa_block_join(None, x, out, torch.zeros(2, 16)[:, ::2], stream=0),
        lambda: fa.fa_block_join(None, x, out, out, post_weight=torch.ones(9), stream=0),
        lambda: fa.fa_block_join(None, x, out, out, gate=w, stream=0),
        lambda: fa.fa_block_join(None, x, out, out, out, pre_rstd=torch.ones(3), stream=0),
        lambda: fa.fa_block_join_gradient(None, None, None, None, None, None, None, None, stream=0),
        lambda: fa.fa_block_join_gradient(None, None, x, torch.zeros(2, 9), None, out, None, None,
                                          stream=0),
        lambda: fa.fa_route(torch.zeros(2, 9), b, stream=0),
        lambda: fa.fa_route(x, b, counted=torch.ones(3, dtype=torch.bool), stream=0),
        lambda: fa.fa_route_gradient(x, b, torch.zeros(2, 9), stream=0),
        lambda: fa.fa_route_gradient(x, fa.route_buffers(2, 8, 2, "cpu", loss=False), out, stream=0),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    wrong_type = [
        lambda: fa.fa_dropout(x, half, fa.Dropout(0.1), stream=0),
        lambda: fa.fa_dropout(x, out, fa.Dropout(0.1, counter=torch.zeros(1)), stream=0),
        lambda: fa.fa_block_join(None, x, out, half, stream=0),
        lambda: fa.fa_block_join(None, x, out, out, post_weight=w, pre_weight=w.half(), stream=0),
        lambda: fa.fa_block_join(None, x, half, out, out, stream=0),
        lambda: fa.fa_block_join_gradient(None, x, x, out, out, half, None, None, stream=0),
        lambda: fa.fa_route(x.double(), b, stream=0),
        lambda: fa.fa_route(x, b, counted=torch.ones(2, dtype=torch.int64), stream=0),
        lambda: fa.fa_route_gradient(x, b, half, stream=0),
        lambda: fa.fa_route_gradient(x, b, out, dweights=torch.zeros(2, 2).half(), stream=0),
    ]
    for call in wrong_type:
        with pytest.raises(TypeError):
            call()


def test_layers_refuse_odd_shapes():
    from amsgrad_optimizer_step_gb300 import layers
    with pytest.raises(ValueError):
        layers.block_join(torch.zeros(2, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        layers.dropout(torch.zeros(()), 0.1, 1)
    with pytest.raises(ValueError):
        layers.norm(torch.zeros(()))
    with pytest.raises(ValueError):
        layers.route(torch.zeros(8), 2)


# ---- the 64-bit reference, pinned ---------------------------------------------------------

@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_reference_generator_has_the_published_answers(counter, key, want):
    got = B.philox([np.array([c], dtype=np.uint64) for c in counter], key)
    assert tuple(int(x[0]) for x in got) == want


def test_reference_dropout():
    a = B.kept(3, 11, 0.25, 7, 5, "cpu")
    assert a.shape == (3, 11) and 0 < int(a.sum()) < 33
    assert torch.equal(a, B.kept(3, 11, 0.25, 7, 5, "cpu"))
    assert torch.equal(a[:, :8], B.kept(3, 16, 0.25, 7, 5, "cpu")[:, :8])  # rows of two blocks
    assert not torch.equal(a, B.kept(3, 11, 0.25, 7, 6, "cpu"))
    assert not torch.equal(a, B.kept(3, 11, 0.25, 8, 5, "cpu"))
    assert B.kept(3, 11, 0.0, 7, 5, "cpu").all() and not B.kept(3, 11, 1.0, 7, 5, "cpu").any()
    assert B.keep_scale(0.5) == 2.0 and B.keep_scale(0.0) == 1.0


def test_reference_join_is_autograd():
    g = torch.Generator().manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64).requires_grad_()

    r, y, w1, w2, gate = randn(6, 10), randn(6, 10), randn(10), randn(10), randn(2, 10)
    mask = torch.rand(6, 10, generator=g) < 0.7
    for post in (True, False):
        out, _, rstd = B.join(r, y, w1, gate, post, 0.9, 0.7, 1e-3, 1.0, mask, 1.4)
        normed, _, pre_rstd = B.norm(out, w2, 1e-3, 1.0)
        dout, dn = randn(6, 10).detach(), randn(6, 10).detach()
        leaves = [r, y, gate, w2] + ([w1] if post else [])
        names = ["dresidual", "dbranch", "dgate", "dpre_weight", "dpost_weight"]
        b = torch.nn.functional.rms_norm(y, (10,), w1 + 1, 1e-3) if post else y
        x = 0.9 * r + 0.7 * gate.repeat_interleave(3, 0) * 1.4 * b.masked_fill(~mask, 0.0)
        want = torch.autograd.grad([x, torch.nn.functional.rms_norm(x, (10,), w2 + 1, 1e-3)],
                                   leaves, [dout, dn])
        assert torch.allclose(out, x, rtol=1e-12)
        got = B.join_gradient(out.detach(), y.detach(), dout, dn,
                              rstd.detach()[:, 0] if post else None, pre_rstd.detach()[:, 0],
                              w1.detach(), w2.detach(), gate.detach(), post, 0.9, 0.7, 1.0, mask,
                              1.4)
        for name, x in zip(names, want):
            assert torch.allclose(got[name][0], x, rtol=1e-9, atol=1e-12), name


def test_reference_router():
    x = torch.tensor([[1.0, 3.0, 3.0, -INF], [0.0, -0.0, NAN, INF], [2.0, 2.0, 2.0, 2.0]])
    assert B.chosen(x, 3, None).tolist() == [[1, 2, 0], [2, 3, 0], [0, 1, 2]]
    counted = torch.tensor([True, False, True])
    assert B.chosen(x, 2, counted).tolist() == [[1, 2], [-1, -1], [0, 1]]
    even = B.route(torch.zeros(8, 4, dtype=torch.float64), 4, None, True, 1.0, 2.0, 3.0)
    assert abs(even["balance"].item() - 1.0) < 1e-12
    assert abs(even["z"].item() - math.log(4) ** 2) < 1e-12
    assert torch.allclose(even["weights"], torch.full((8, 4), 0.25, dtype=torch.float64))
