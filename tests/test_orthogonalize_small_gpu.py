"""The orthogonalised update under coefficients whose steps shrink the singular values:
operands are held relative to the steps' bounds.

One step of (a, 0, 0), undone by the scale, is G / |G|: the factor and the scale round by
2^-24 each, X and P are two terms (2 x 2^-24), their product leaves out lo lo
(4 x 2^-24) and rounds up to twice in each of three instructions (the other products of
the sum are zeros), and the result rounds once: 20 x 2^-24 of a value, and 2^-39 of the
largest where X's terms end, 2^-38 with room for its product's."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from test_orthogonalize_gpu import exact, gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(40, 60), (128, 256), (3000, 30), (300, 200), (777, 1033)]


@pytest.mark.parametrize("a", [1.0, 1e-3, 1e-6, 1e-9, 2.0 ** -35])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_small_multiples(size, a):
    say("orthogonalize small", size, a)
    g = torch.randn(size, generator=gen(size[0]), device="cuda")
    got = dg.orthogonalize(g, steps=1, coefficients=(a, 0.0, 0.0), scale=1 / a).double()
    ref = exact(g, [(a, 0.0, 0.0)], scale=1 / a)
    assert bool(((got - ref).abs() <= 20 * 2.0 ** -24 * ref.abs() + 2.0 ** -38).all()), \
        float(((got - ref).abs() / (20 * 2.0 ** -24 * ref.abs() + 2.0 ** -38)).max())


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_step_on_small_values(size):
    """X shrunk to 1e-6 and then a step of 1.5 s - 0.5 s^3 on its 1e6-fold: A is off by up
    to 160 x 2^-24 of |X|_F^2 = 1 (its sums' roundings, 5 in each of up to 32 instructions),
    P by half of that, P X by as much again, and all of it by less than 1000 x 2^-24."""
    say("orthogonalize small", size)
    g = torch.randn(size, generator=gen(size[0]), device="cuda")
    each = [(1e-6, 0.0, 0.0), (1.5, -0.5e12, 0.0)]
    got = dg.orthogonalize(g, steps=2, coefficients=each, scale=1e6).double()
    ref = exact(g, each, scale=1e6)
    assert bool((got - ref).norm() <= 1000 * 2.0 ** -24 * ref.norm()), float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("c", [1e-17, -1e-17, 0.0])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_cubic_whose_largest_value_is_inside(size, c):
    """24 s - 27 s^3 is 8.7 at 0.54 and 3 at 1: two equal singular values of 0.7, and of
    0.54 from an entry of 2^-1.3 of the norm, neither lost nor past the range."""
    say("orthogonalize cubic", size, c)
    for first, second in ((1.0, 1.0), (0.65, 1.0)):
        g = torch.zeros(size, device="cuda")
        g[0, 1], g[-1, 0] = first, second
        got = dg.orthogonalize(g, steps=1, coefficients=(24.0, -27.0, c), eps=0.0).double()
        ref = exact(g, [(24.0, -27.0, c)], 0.0)
        # one product a sum: A is off by 18 x 2^-24 of itself, P by 27 times that and 6 x 2^-24 of
        # its terms, P X by 15 x 2^-24 of itself and s times P's error: together below 570 x 2^-24
        assert bool(((got - ref).abs() <= 600 * 2.0 ** -24).all())
