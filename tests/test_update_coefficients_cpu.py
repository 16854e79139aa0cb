"""The powers of two at which the orthogonalised update holds its operands, on the CPU (a
host build of the plan, ``cpp/update_plan.cpp``): for drawn coefficients the largest
values that the steps allow, found by following singular values over [0, 1], stay
below what binary16 holds, and use its range."""
import os
import random
import subprocess

import numpy as np
import pytest

import linear_plan
from dense_gemm_optimisation_row_amd import binding as b
from dense_gemm_optimisation_row_amd import layers

ROOT = linear_plan.ROOT
pytestmark = pytest.mark.skipif(linear_plan.hipcc() is None, reason="needs hipcc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("update") / "plan")
    subprocess.run([linear_plan.hipcc(), "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                    f"-I{ROOT}/include", f"-I{ROOT}/dense_gemm_optimisation_row_amd/csrc", "-x", "hip",
                    os.path.join(ROOT, "tests", "cpp", "update_plan.cpp"), "-o", exe], check=True, capture_output=True)

    def ask(calls):
        """(status, [(x, gram, poly) of each step]) of each (steps' triples, scale)."""
        lines = "\n".join(f"{scale!r} {len(each)} " + " ".join(repr(float(v)) for t in each for v in t)
                          for each, scale in calls)
        out = subprocess.run([exe], input=lines + "\n", capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(calls)
        found = []
        for line in out:
            rc, *e = (int(v) for v in line.split())
            found.append((rc, [tuple(e[i:i + 3]) for i in range(0, len(e), 3)]))
        return found
    return ask


# The values come from 20001 points; the plan's bounds are of all singular values up to
# the largest of the step before, of which the first steps reach each one.
S = np.linspace(0, 1, 20001)


def largest(each):
    """(r, p) before and in each step: the largest value, and what it multiplies at most."""
    r, out = 1.0, []
    for a, bb, c in each:
        s = S * r
        t = s * s
        p = np.abs(a + t * (bb + t * c))
        out.append((r, float(p.max())))
        r = float((s * p).max())
    return out


def held(found, each):
    rc, steps = found
    assert rc == b.GEMM_OK
    for (x, gram, poly), (r, p) in zip(steps, largest(each)):
        for bound, e in ((r, x), (r * r, gram), (p, poly)):
            # (half of the range or more; 1e-6 for the points)
            assert bound == 0 or 30000 * (1 - 1e-6) <= bound * 2.0 ** e <= 60000 * (1 + 1e-6), (each, bound, e)


def drawn(rng):
    """One to five steps, as fits give them: odd polynomials of one to five, of any size
    that the steps allow."""
    each = []
    r = 1.0
    for _ in range(rng.randint(1, 5)):
        most = 2.0 ** rng.uniform(-6, 6)
        a, bb, c = (rng.uniform(-1, 1) for _ in range(3))
        bb, c = bb / r ** 2 * rng.choice([0, 1, 4]), c / r ** 4 * rng.choice([0, 0, 1, 4])
        t = (S * r) ** 2
        p = float(np.abs(a + t * (bb + t * c)).max())
        if p == 0:
            continue
        step = tuple(v * most / p for v in (a, bb, c))
        nxt = largest(each + [step, (1.0, 0.0, 0.0)])[-1][0]
        if not 2.0 ** -34 < nxt < 250:
            continue
        each.append(step)
        r = nxt
    return each or [(1.5, -0.5, 0.0)]


def test_drawn_coefficients_stay_within_binary16_and_use_its_range(plan):
    rng = random.Random(3)
    calls = [drawn(rng) for _ in range(2000)]
    calls += [[(3.4445, -4.7750, 2.0315)] * 5, [(1.0, -8.0, 8.0)], [(5.0, -20.0, 16.0)], [(1e-3, 0, 0)] * 3,
              [(1e-9, 0, 0)], [(1e-6, 0, 0), (1.5, -0.5e12, 0)], [(1e-5, 0, 0), (3.4445, -4.7750e10, 2.0315e20)] + [
                  (250.0, 0.0, 0.0)] * 2]
    for found, each in zip(plan([(each, 1.0) for each in calls]), calls):
        held(found, each)


def test_polynomials_of_nearly_lower_degree(plan):
    """A leading coefficient that is left over from rounding, as fits give it: the largest
    value is inside [0, 1], where the cubic or the line has it."""
    calls = []
    for c in (1e-16, -1e-16, 1e-17, -1e-17, 1e-20, -1e-30, 1e-300, 0.0, -0.0):
        calls += [[(24.0, -27.0, c)], [(3.0, -4.0, c)], [(24.0, -27.0, c), (1.5, -0.02, 0.0)], [(-6.0, 7.0, c)]]
        calls += [[(2.0, c, -3.0)], [(2.0, c, 3.0)], [(c, -4.0, 5.0)], [(2.0, c, c)], [(c, c, 1.0)], [(c, 2.0, c)]]
    for found, each in zip(plan([(each, 1.0) for each in calls]), calls):
        held(found, each)


def test_coefficients_that_leave_the_range(plan):
    ok = [[(0, 0, 0)], [(0, 0, 0), (1.5, -0.5, 0)], [(2.0 ** -35, 0, 0)], [(1e-6, 0, 0), (1e-4, 0, 0)], [(256.0, 0, 0)]]
    bad = [[(1e-11, 0, 0)], [(1e-13, 0, 0), (1.5, -0.5, 0)], [(1e-6, 0, 0), (1e-5, 0, 0)], [(1e-300, 0, 0)],
           [(0, 1e-12, 1e-13)], [(257.0, 0, 0)]]
    for found, each in zip(plan([(e, 1.0) for e in ok + bad]), ok + bad):
        assert found[0] == (b.GEMM_OK if each in ok else b.GEMM_ERR_INVALID_COEFFICIENTS), each


def test_scales_that_leave_fp32(plan):
    default = [(3.4445, -4.7750, 2.0315)] * 5
    ok = [0.0, -0.0, 1e-20, -1e-25, 0.02, 2.0 ** 100, float("inf"), float("nan")]
    bad = [1e-32, -1e-37, 1e-300, 5e-324, 1e300, -1e200]
    for found, scale in zip(plan([(default, s) for s in ok + bad]), ok + bad):
        assert found[0] == (b.GEMM_OK if any(scale is s for s in ok) else b.GEMM_ERR_INVALID_COEFFICIENTS), scale
    for small in ([(2.0 ** -35, 0, 0)], [(256.0, 0, 0)]):
        assert all(rc == b.GEMM_OK for rc, _ in plan([(small, 2.0 ** -26), (small, 2.0 ** 100)]))


def test_steps_out_of_range_are_refused_before_their_coefficients_are_made():
    for steps in (0, -1, 33, 10 ** 12):   # (10^12 triples are 8 TB)
        with pytest.raises(ValueError, match="steps must be"):
            layers._step_coefficients((3.4445, -4.775, 2.0315), steps)
