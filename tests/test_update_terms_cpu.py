"""That the bounds of the orthogonalised update's blocks hold for its arithmetic in two
terms, and for no operand that has lost its lower term: on the CPU, with the loss planted
in a simulation."""
import pytest
import torch

import update_terms as terms


def worst(blocks, each, drop=None):
    ref, err = terms.exact_and_error(blocks.values, each)
    tol = err + terms.U * (ref.abs() + err)
    return float(((terms.simulate(blocks.values, each, drop).double() - ref).abs() / tol).max())


@pytest.mark.parametrize("m", [1, 2, 24, 64, 130, 777, 2002, 4070])
def test_the_simulation_is_within_the_bounds(m):
    blocks = terms.Blocks(2, m, m + 3, m, "cpu")
    for last in terms.LAST:
        for each in ([last], terms.steps_for(m, last)):
            assert worst(blocks, each) <= 1


@pytest.mark.parametrize("drop", terms.OPERANDS)
@pytest.mark.parametrize("m", [24, 64, 130, 777, 2002, 4070])
def test_a_lost_lower_term_is_not(m, drop):
    blocks = terms.Blocks(2, m, m + 3, m, "cpu")
    assert max(worst(blocks, terms.steps_for(m, last), drop) for last in terms.LAST) > 4
