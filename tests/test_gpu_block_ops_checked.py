"""The residual blocks' operators through the bounds-checked build of the library: their own tests,
with every access outside its array counted and skipped; the count must stay zero, and the
results are the normal build's."""

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
import test_gpu_block_ops as T
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
    ("dropout", lambda: [T.test_dropout_sizes_and_types(dt, shape, 0.3) for dt in ("f32", "bf16")
                         for shape in ((1, 1), (5, 64), (4, 65), (33, 515), (7, 1408))]
        + [T.test_dropout_layouts("f16", lay, c) for lay in T.LAYOUTS for c in (5, 64, 1003)]),
    ("join types and parts", lambda: [
        T.test_join_types_and_parts(k, f, s) for k in T.KINDS[1:5] for f in T.FLAGS
        for s in ((700, 264), (3, 515))]),
    ("join widths", lambda: [T.test_join_widths(c, T.KINDS[4]) for c in (
        1, 9, 257, 2048, 4104, 6152, 8200, 16384)]),
    ("join layouts", lambda: [T.test_join_layouts(lay, T.KINDS[2]) for lay in T.LAYOUTS]),
    ("join groups", lambda: [T.test_join_groups(*s) for s in (
        (6, 6, 40), (1368, 24, 2048), (11001, 3667, 24), (40, 8, 8200), (304, 19, 515))]),
    ("router", lambda: [T.test_route_sizes_and_types(dt, e) for dt in ("f32", "f16")
                        for e in (1, 9, 60, 129, 520, 1024)]
        + [T.test_route_layouts(lay, "bf16") for lay in T.LAYOUTS]
        + [T.test_route_lengths(t) for t in (0, 1, 33, 5000)]),
]


@pytest.mark.parametrize("name,run", CASES, ids=[c[0] for c in CASES])
def test_no_access_out_of_range(checked, name, run):
    with _lib.using(checked):
        fa.fa_bounds_check_report(clear=True)
        run()
        torch.cuda.synchronize()
        assert fa.fa_bounds_check_report() == (True, 0)


def test_checked_build_gives_the_same_bits(checked):
    c = T.Case(300, 1032, "bf16", groups=3, p=0.1)
    c.forward(check=False)
    want = [c.out, c.normed, *c.backward(check=False).values()]
    with _lib.using(checked):
        c.forward(check=False)
        got = [c.out, c.normed, *c.backward(check=False, draw=False).values()]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
