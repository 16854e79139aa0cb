"""The orthogonalised update where the polynomial's terms are far larger than the
polynomial: P's entries are bounded by the coefficients' steps, b A's are not, and what
stands beside P in its padded rows must be neither.

Exact: the first row (or column) and the last are equal, 2^(2 k - 1) entries of +-1
each, and all else is zero.  With eps 0 the norm is 2^k, A's four entries are 1 / 2,
and one step with whole coefficients is small integers over powers of two."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from test_orthogonalize_gpu import exact, gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# batch, M, N, k: rows (the shorter side) that are no multiple of 8, on the three
# products' tiles of 64 x 64 (with and without sums apart), 128 x 128 and 256 x 256,
# as whole tiles and as runs; in strips and in one launch
SIZES = [(1, 130, 300, 4), (1, 300, 131, 4), (1, 777, 1033, 5), (1, 2049, 1500, 5), (30, 100, 2000, 4), (1, 2002, 2002, 5),
         (5, 1700, 1702, 5), (1, 3001, 3001, 5), (1, 4070, 4099, 5), (1, 100, 1000, 4), (8, 75, 300, 4), (1, 61, 70, 3)]
# (1, -8, 8) is at most 1 over [0, 1], its b A 4; (5, -20, 16), a Chebyshev polynomial, 5 and 10
COEFFICIENTS = [(1.0, -8.0, 8.0), (5.0, -20.0, 16.0)]


def two_rows(batch, M, N, k, seed):
    m, n = min(M, N), max(M, N)
    g = torch.zeros(batch, m, n, device="cuda")
    for i in range(batch):
        at = torch.randperm(n, generator=gen(seed + i), device="cuda")[:2 ** (2 * k - 1)]
        row = torch.zeros(n, device="cuda")
        row[at] = torch.randint(0, 2, (len(at),), generator=gen(seed + 50 + i), device="cuda").float() * 2 - 1
        g[i, 0] = g[i, -1] = row
    return g if M <= N else g.mT.contiguous()


@pytest.mark.parametrize("coefficients", COEFFICIENTS, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s[:3])))
def test_terms_past_the_polynomial(size, coefficients):
    batch, M, N, k = size
    say("orthogonalize padding", size, coefficients)
    g = two_rows(batch, M, N, k, M + N)
    got = dg.orthogonalize(g, steps=1, coefficients=coefficients, eps=0.0)
    want = exact(g[0], [coefficients], 0.0)
    assert not bool(torch.isnan(got).any()), f"{int(torch.isnan(got).sum())} NaN of {got.numel()}"
    assert torch.equal(got[0], want.float())
    assert torch.equal(got[-1], exact(g[-1], [coefficients], 0.0).float())


def test_later_steps_whose_terms_pass_the_polynomial():
    """1 stays 1 under (1, -8, 8) and (1, 0, 0): exact through all steps."""
    for M, N, k in ((130, 300, 4), (777, 1033, 5), (2002, 2002, 5)):
        for each in ([COEFFICIENTS[0]] * 3, [(1.0, 0.0, 0.0), COEFFICIENTS[0]]):
            say("orthogonalize padding", M, N, each)
            g = two_rows(1, M, N, k, 3)[0]
            got = dg.orthogonalize(g, steps=len(each), coefficients=each, eps=0.0)
            assert torch.equal(got, exact(g, each, 0.0).float())
