"""That each operand of the orthogonalised update's products has both of its terms, in
every way in which it runs.

On blocks (``update_terms.py``) the result is held, entry by entry, to a bound that no
operand keeps without its lower term.  On full matrices it is held to three times the error
of the same steps with products in FP32: two terms are off by 2^-23 of a value where FP32
is by 2^-24, and the sums of both round alike; 16 x 2^-24 of the result are allowed
beside, for an FP32 error that is small by chance."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
import update_terms as terms
from helpers import say
from test_orthogonalize_gpu import COEFFICIENTS, exact, matrix, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# batch, rows, columns (rows the fewer): one launch; strips of one to four blocks of 32
# rows; the three products on each tile, as whole tiles and as runs
SIZES = [(1, 1, 1), (3, 7, 9), (1, 61, 90), (5, 64, 64), (1, 24, 3000), (1, 60, 1000), (1, 90, 1300), (8, 128, 256),
         (1, 127, 1001), (30, 100, 2000), (1, 128, 5000), (1, 200, 300), (1, 130, 4099), (1, 777, 1033), (1, 1033, 1500),
         (2, 1500, 1501), (1, 2002, 2002), (1, 3001, 3001), (5, 1700, 1702), (1, 4070, 4099)]
FULL = [(1, 40, 60), (1, 30, 3000), (1, 64, 900), (1, 95, 1300), (1, 128, 1024), (30, 100, 2000), (1, 200, 300),
        (1, 777, 1033), (1, 2002, 2002), (5, 1700, 1702), (1, 4070, 4099)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_blocks(size):
    blocks = terms.Blocks(*size, size[1] + size[2], "cpu")
    g = blocks.dense(blocks.values)
    for last in terms.LAST:
        each = terms.steps_for(size[1], last)
        ref, err = terms.exact_and_error(blocks.values, each)
        want = blocks.dense(ref)
        tol = blocks.dense(err + terms.U * (ref.abs() + err))
        for turned in (False, True):
            say("orthogonalize terms", size, last, turned)
            x = (g.mT if turned else g).contiguous().cuda()
            got = dg.orthogonalize(x, steps=len(each), coefficients=each, eps=0.0).cpu()
            off = ((got.mT if turned else got).double() - want).abs()
            assert bool((off <= tol).all()), (last, turned, float((off / tol.clamp_min(1e-300)).max()))


def fp32(g, coefficients, eps=1e-7):
    x = g / (g.double().square().sum((-2, -1), keepdim=True).sqrt() + eps).float()
    for a, b, c in coefficients:
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


@pytest.mark.parametrize("kind", ["normal", "spread"])
@pytest.mark.parametrize("size", FULL, ids=lambda s: "x".join(map(str, s)))
def test_full_matrices(size, kind):
    batch, M, N = size
    say("orthogonalize terms", size, kind)
    g = torch.stack([matrix(M, N, M + N + i, torch.float32, kind) for i in range(batch)])
    each = [COEFFICIENTS] * 5
    got = dg.orthogonalize(g)
    for i in {0, batch // 2, batch - 1}:
        ref = exact(g[i], each)
        own, other = (float((t.double() - ref).norm()) for t in (got[i], fp32(g[i], each)))
        tol = 3 * other + 16 * terms.U * float(ref.norm())
        say(f"  {own / float(ref.norm()):.2e}, FP32 {other / float(ref.norm()):.2e}")
        assert own <= tol, f"{i}: {own / tol:.3g} of the bound"
