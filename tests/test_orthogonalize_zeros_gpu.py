"""The orthogonalised update of zeros, whatever eps, and of norms that eps does not touch."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from test_orthogonalize_gpu import DTYPES, gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# in one launch, in strips, in three products a step; also turned round
SIZES = [(1, 1), (40, 60), (70, 20), (128, 256), (3000, 30), (300, 200), (520, 777)]


@pytest.mark.parametrize("eps", [0.0, 5e-324, 1e-310, 1e-30, 1e-7, float("inf")])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_zeros_stay_zeros(size, eps):
    for dtype in DTYPES.values():
        say("orthogonalize zeros", size, eps, dtype)
        z = torch.zeros(size, device="cuda", dtype=dtype)
        assert bool((dg.orthogonalize(z, eps=eps) == 0).all())
        # next to another matrix of a stack, whose result stays its own
        g = torch.stack((z, torch.randn(size, generator=gen(1), device="cuda").to(dtype)))
        out = dg.orthogonalize(g, eps=eps)
        assert bool((out[0] == 0).all()) and not bool(torch.isnan(out).any())
        assert torch.equal(out[1], dg.orthogonalize(g.flip(0).contiguous(), eps=eps)[0])


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_one_entry_without_eps(size):
    """A single entry is its own norm: a + b + c times its sign after a step, exactly."""
    for v in (-3.0, 2.0 ** -149, 2.0 ** -120, 2.0 ** 127):
        say("orthogonalize one entry", size, v)
        g = torch.zeros(size, device="cuda")
        g[size[0] // 2, size[1] // 2] = v
        out = dg.orthogonalize(g, steps=1, coefficients=(2.0, -1.0, 3.0), eps=0.0)
        assert torch.equal(out, 4.0 * g.sign())
