"""Joins of rows that begin anywhere in their 16-byte lines, as contiguous matrices of odd widths
have them: enough rows for the paths that take them in the lines that memory has, against the
formulas in 64 bits, in themselves and beside rows that are not finite; and rows that are wider
than one CTA holds."""

import pytest
import torch

import amsgrad_optimizer_step_gb300 as fa
from amsgrad_optimizer_step_gb300 import _lib
from test_gpu_block_ops import FLAGS, KINDS, NAN, Case, _built  # noqa: F401
from test_gpu_block_ops_checked import checked  # noqa: F401

pytestmark = pytest.mark.gpu


def many_rows(cols, more=0):
    """At least a row for each CTA that fits an SM at this width, whatever the type."""
    warps = ((cols + 14) // 8 + 31) // 32
    return 152 * max(1, 24 // warps) + more


# one run and a few, the last column of a run, the runs one more than the columns ask for (2042 and
# 2047: in some rows only), the widest that the paths hold and the first beyond
@pytest.mark.parametrize("cols", [15, 17, 33, 515, 1003, 2042, 2047, 3081, 4101, 5119, 6131, 6137,
                                  6145, 8191, 16370, 16371, 16383])
@pytest.mark.parametrize("kind", [KINDS[2], KINDS[4], KINDS[0]])
def test_widths(cols, kind):
    c = Case(many_rows(cols, 5), cols, *kind, p=0.1, seed=cols)
    c.forward()
    c.backward()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("flags", FLAGS)
def test_types_and_parts(kind, flags):
    c = Case(1500, 515, *kind, **flags)
    c.forward()
    c.backward()


@pytest.mark.parametrize("more", [-9, -1, 0, 1, 7, 8, 455, 456, 3000])
def test_lengths(more):
    """A row a CTA and fewer, and rows that the teams of a CTA share unevenly."""
    c = Case(many_rows(1026, more), 1026, "bf16", p=0.1)
    c.forward()
    c.backward()


@pytest.mark.parametrize("pad", [1, 2, 3, 6, 8, 13])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_a_wider_matrix(pad, dt):
    """Row distances odd and even, equal to the width or not; what lies between is left alone."""
    for cols in (515, 1024):
        c = Case(1300, cols, dt, p=0.1, layout=(pad, 0))
        c.forward()
        c.backward()


@pytest.mark.parametrize("kind", [KINDS[1], KINDS[3], KINDS[0]])
def test_rows_keep_to_themselves(kind):
    """Lines that two rows share: what is not finite in one changes nothing in the other."""
    c = Case(1300, 515, *kind, p=0.1)
    c.forward(check=False)
    want = c.backward(check=False)
    want = dict(out=c.out, normed=c.normed, dresidual=want["dresidual"], dbranch=want["dbranch"])
    bad = torch.zeros(c.rows, dtype=torch.bool, device=c.out.device)
    bad[[0, 7, 8, 600, c.rows - 2]] = True
    for t in (c.residual, c.branch, c.dout, c.dnormed):
        t[bad] = NAN
    c.forward(check=False)
    got = c.backward(check=False, draw=False)
    got = dict(out=c.out, normed=c.normed, dresidual=got["dresidual"], dbranch=got["dbranch"])
    for name in want:
        assert torch.equal(got[name][~bad], want[name][~bad]), name


def test_the_same_elements_are_dropped_as_of_even_rows():
    """The columns of a matrix keep their elements of the generator whatever lies behind them."""
    for cols in (515, 1029):
        c = Case(1300, cols, "f32", post=False, pre=False, groups=0, p=0.5, alpha=0.0)
        c.branch.fill_(1.0)
        c.residual.zero_()
        c.forward(check=False)
        assert torch.equal(c.out != 0, c.mask)


def test_in_place_and_again():
    c = Case(2000, 1003, "bf16", p=0.1)
    c.forward(check=False)
    x, normed = c.residual.clone(), torch.empty_like(c.normed)
    fa.fa_block_join(c.record, x, c.branch, x, normed, None, None, c.post_weight, c.pre_weight,
                     c.gate)
    assert torch.equal(x, c.out) and torch.equal(normed, c.normed)
    first = c.backward(check=False)
    again = c.backward(check=False, draw=False)
    assert all(torch.equal(first[k], again[k]) for k in first)


def test_no_access_out_of_range(checked):  # noqa: F811
    """Through the bounds-checked build, with the normal build's bits."""
    for kind in (KINDS[0], KINDS[2], KINDS[3]):
        for cols, layout in ((17, (0, 0)), (515, (0, 0)), (2042, (3, 0)), (6131, (0, 0))):
            c = Case(many_rows(cols, 11), cols, *kind, p=0.1, layout=layout)
            c.forward(check=False)
            want = [c.out, c.normed, *c.backward(check=False).values()]
            with _lib.using(checked):
                fa.fa_bounds_check_report(clear=True)
                c.forward(check=False)
                got = [c.out, c.normed, *c.backward(check=False, draw=False).values()]
                torch.cuda.synchronize()
                assert fa.fa_bounds_check_report() == (True, 0)
            assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows,groups", [(1400, 700), (1400, 7), (1400, 1400), (1401, 3), (4000, 2)])
@pytest.mark.parametrize("kind", [KINDS[2], KINDS[3], KINDS[0]])
def test_gates_of_several_groups(rows, groups, kind):
    for cols in (515, 1003):
        c = Case(rows, cols, *kind, groups=groups, p=0.1)
        c.forward()
        c.backward()


# rows that a cluster of two or four CTAs holds, at their first and last widths, and those (6160 FP32)
# whose row a CTA holds but no two
@pytest.mark.parametrize("cols", [6160, 8200, 12288, 12296, 16376, 16384])
@pytest.mark.parametrize("kind", KINDS)
def test_wide_rows(cols, kind):
    for rows, groups, p in ((1, 1, 0.0), (3, 3, 0.1), (77, 1, 0.1), (160, 4, 0.0)):
        c = Case(rows, cols, *kind, groups=groups, p=p)
        c.forward(check=False)
        c.backward()


@pytest.mark.parametrize("flags", FLAGS)
def test_wide_rows_of_all_parts(flags):
    for cols in (8200, 16384):
        c = Case(90, cols, "bf16", "f32", "f32", **flags)
        c.forward(check=False)
        c.backward()


def test_wide_rows_through_the_checked_build(checked):  # noqa: F811
    for dt, cols in (("bf16", 8200), ("f32", 16384)):
        c = Case(100, cols, dt, p=0.1, groups=2)
        c.forward(check=False)
        want = list(c.backward(check=False).values())
        with _lib.using(checked):
            fa.fa_bounds_check_report(clear=True)
            got = list(c.backward(check=False, draw=False).values())
            torch.cuda.synchronize()
            assert fa.fa_bounds_check_report() == (True, 0)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_captured_gradient_that_is_replayed():
    """Both new kinds of rows in a graph, on inputs that change between the replays."""
    cases = [Case(1300, 515, "bf16", p=0.1), Case(20, 16384, "bf16", p=0.1), Case(20, 8200, "f32")]
    for c in cases:
        c.forward(check=False)
        c.draw()
        scratch = fa.join_scratch(c.rows, c.cols, c.groups, c.out.device)
        outs = [torch.empty_like(t) for t in (c.residual, c.branch, c.post_weight, c.pre_weight,
                                              c.gate)]

        def run():
            fa.fa_block_join_gradient(c.record, c.out, c.branch, c.dout, c.dnormed, outs[0],
                                      outs[1], scratch, c.post_rstd, c.pre_rstd, c.post_weight,
                                      c.pre_weight, c.gate, *outs[2:])

        graph = torch.cuda.CUDAGraph()
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        c.dout.mul_(-2)
        for t in outs:
            t.fill_(NAN)
        graph.replay()
        replayed = [t.clone() for t in outs]
        run()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs))


@pytest.mark.parametrize("cols", [4096, 5120, 5632, 6144, 8192])
def test_rows_of_which_a_cta_holds_one(cols):
    for rows, groups in ((5, 1), (400, 4)):
        for kind in (KINDS[0], KINDS[3]):
            c = Case(rows, cols, *kind, groups=groups, p=0.1)
            c.forward(check=False)
            c.backward()


def test_the_norm_can_be_taken_again():
    for cols, dt, st in ((515, "bf16", "bf16"), (1003, "f32", "f32"), (2042, "f16", "f32")):
        c = Case(1300, cols, dt, st, p=0.1)
        c.forward(check=False)
        again = torch.empty_like(c.normed)
        fa.fa_block_join(fa.Join(False, eps=c.eps), c.out, None, None, again,
                         pre_weight=c.pre_weight)
        assert torch.equal(again, c.normed)
