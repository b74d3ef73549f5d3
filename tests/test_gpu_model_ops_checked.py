"""The model-side operators through the bounds-checked build of the library: their own tests,
with every access outside its array counted and skipped; the count must stay zero, and the
results are the normal build's."""

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import test_gpu_model_ops as M
from amsgrad_optimizer_step_gb300 import _lib, build

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def checked():
    build.build()
    lib = _lib.open_library(build.build(variant="checked"))
    with _lib.using(lib):
        enabled, _ = fa.fa_bounds_check_report(clear=True)
    assert enabled
    return lib


CASES = [
    ("lookup", lambda: [M.test_lookup_types("bf16", "f32"), M.test_lookup_types("f32", "f16")]
        + [M.test_lookup_layouts(d, lay) for d in (1, 12, 515, 2048) for lay in M.LAYOUTS]),
    ("embedding gradient lengths", lambda: [
        M.test_embedding_gradient_lengths(t, k) for t in (0, 1, 31, 33, 65, 4097, 8193, 20011)
        for k in ("zipf", "same", "distinct")]),
    ("embedding gradient widths and types", lambda: [
        M.test_embedding_gradient_widths(d, lay) for d in (1, 100, 515, 4104)
        for lay in ((0, 0), (3, 1))] + [M.test_embedding_gradient_types("bf16", "f32", True),
                                        M.test_embedding_gradient_types("f32", "f16", False)]),
    ("embedding gradient vocabularies", lambda: [
        M.test_embedding_gradient_vocabularies(v) for v in (1, 2, 255, 65536, 131072)]),
    ("log-probabilities", lambda: [
        M.test_logprobs_sizes_and_types(dt, v) for dt in ("f32", "bf16")
        for v in (1, 7, 127, 2049, 32000)] + [
        M.test_logprobs_layouts("f16", v, lay) for v in (5, 1003) for lay in M.LAYOUTS]),
    ("wide rows", lambda: [M.test_logprobs_wide_rows("bf16", 131_072),
                           M.test_policy_wide_rows("f32", 100_003),
                           M.test_policy_wide_rows("bf16", 400_009)]),
    ("preference", lambda: [M.test_preference(lens, 0.1, True) for lens in
                            ([1, 1], [0, 0, 3, 4], [17, 16] * 20, [257, 1025])]
        + [M.test_preference_offsets_that_leave_tokens_out()]),
    ("policy", lambda: [M.test_policy_sizes_and_types("bf16", v) for v in (1, 130, 8192, 32000)]
        + [M.test_policy_lengths(t) for t in (1, 151, 5000)]
        + [M.test_policy_layouts("f32", lay, v) for lay in M.LAYOUTS for v in (5, 1003)]),
    ("gated", lambda: [M.test_gated_sizes_and_types(dt, "silu", r, c) for dt in ("f32", "f16")
                       for r, c in ((1, 1), (3, 8), (4, 129), (33, 1403), (16, 5632))]
        + [M.test_gated_layouts("bf16", lay) for lay in M.LAYOUTS]),
]


@pytest.mark.parametrize("name,run", CASES, ids=[c[0] for c in CASES])
def test_no_access_out_of_range(checked, name, run):
    with _lib.using(checked):
        fa.fa_bounds_check_report(clear=True)
        run()
        torch.cuda.synchronize()
        assert fa.fa_bounds_check_report() == (True, 0)


def test_checked_build_gives_the_same_bits(checked):
    logits, labels, old, adv, ref, w = M.rollout(5, 50, 1003, "bf16")
    want, d0 = M.run_policy(logits, labels, old, adv, ref_logp=ref, kl_coef=0.1)
    with _lib.using(checked):
        got, d1 = M.run_policy(logits, labels, old, adv, ref_logp=ref, kl_coef=0.1)
    assert torch.equal(d0, d1) and torch.equal(want.summary, got.summary)
