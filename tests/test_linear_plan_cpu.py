"""The dense layers' choice of kernels, on the CPU: what it launches at the
largest sizes, and that the forms which the GPU tests run are all there are."""
import pytest

import linear_plan as plan
from linear_cases import FORMS, line
from dense_gemm_optimisation_row_amd import binding as b

pytestmark = pytest.mark.skipif(plan.hipcc() is None, reason="needs hipcc")

BLOCKS = 2 ** 22   # of 128 x 64: matrices of as many are refused


def sizes():
    """(rows, columns) of matrices just below the limit, and at it."""
    for rows in (1, 3, 64, 128, 129, 4096, 2 ** 20 + 1, 2 ** 28):
        cols = (BLOCKS // -(-rows // 128)) * 64
        while -(-rows // 128) * -(-cols // 64) >= BLOCKS:
            cols -= 64
        yield rows, cols, False
        yield rows, cols + 64 * -(-BLOCKS // -(-rows // 128)), True


def calls(rows, cols):
    """Every call with a matrix of these sizes, on and off 16 bytes, the third
    size small."""
    for fmt in ("bf16", "f16"):
        for small in (1, 8, 72):
            for t in (False, True):
                for shift in (0, 2):
                    for m, n, k in ((rows, cols, small), (rows, small, cols), (small, rows, cols), (small, cols, rows)):
                        yield plan.linear(fmt, m, n, k, t, x=shift, w=shift)
                        yield plan.gated(fmt, m, n, k, t, x=shift, w=shift)
                        yield plan.linear_backward(fmt, m, n, k, t, act="silu", x=shift, w=shift)
                        yield plan.linear_backward(fmt, m, n, k, t, x=shift, w=shift, dy=shift)
                        yield plan.gated_backward(fmt, m, n, k, t, x=shift, w=shift)


@pytest.mark.parametrize("rows,cols,over", list(sizes()))
def test_launches_hold_fewer_than_2_to_32_threads(rows, cols, over):
    if cols >= 2 ** 31 - 64:
        pytest.skip("not an int")
    lines = list(calls(rows, cols))
    for line, (status, _, launches) in zip(lines, plan.launches(lines)):
        if over:
            assert status == b.GEMM_ERR_INVALID_DIM and not launches, line
            continue
        assert status == 0 or (status == b.GEMM_ERR_INVALID_DIM and not launches), (line, status)
        for launch in launches:
            assert 0 <= launch.get("threads", 0) < 2 ** 32, (line, launch)


RING = ["256x256", "256x128", "128x128", "128x64", "64x64"]


def forms(lines):
    """(kernel, tile, layout, whether split, matrices summed, terms, batches) of
    every product that these calls launch."""
    found = set()
    for status, _, launches in plan.launches(lines):
        assert status == 0
        found |= {(v["kind"], v["tile"], v["layout"], v["splits"] > 1, v["segments"] // v["terms"], v["terms"],
                   v["batches"]) for v in launches if v["kind"] in ("ring", "pair", "tile")}
    return found


def every_form():
    for kind, tiles in (("ring", RING), ("pair", RING[2:]), ("tile", ["64x64"])):
        for tile in tiles:
            for split in (False, True):
                if kind != "pair":
                    for layout in ("gated_KxN", "gated_NxK"):
                        yield kind, tile, layout, split, 1, 1, 1
                for terms in (1, 2, 3):
                    for n in (1, 2):
                        yield kind, tile, "KxM", split, 1, terms, n
                        for layout in ("KxN", "NxK"):
                            yield kind, tile, layout, split, n, terms, 1


def test_the_tested_forms_are_all_that_calls_take():
    # 256 x 128 loads half lines of weights as N x K, and is slower than 256 x 256
    # or 128 x 128 at every size; the plain tile gets no operands opened into
    # terms, which are copies at 16 bytes
    taken = {f for f in every_form() if not (f[1] == "256x128" and f[2].endswith("NxK")) and not
             (f[0] == "tile" and f[5] == 3)}
    assert forms([line(c) for c in FORMS]) == taken
