"""The bounds of ``test_gradients_by_differences_gpu``, in 64 bits on the CPU:
the formula's gradient is within them, and gradients that are zero, of the
other sign or without the activation's slope are far outside."""
import pytest
import torch

from layer_reference import act_value, difference_bound, linear_grads

STEP, HALF, ULP = 2.0 ** -6, 2.0 ** -11, 2.0 ** -24


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("size", [(24, 40, 64), (130, 72, 136)], ids=str)
def test_wrong_gradients_are_rejected(size, act, seed):
    M, N, K = size
    torch.manual_seed(seed)
    x, w, dy = (torch.randn(M, K, dtype=torch.float64), torch.randn(K, N, dtype=torch.float64) * K ** -0.5,
                torch.randn(M, N, dtype=torch.float64))
    z = x @ w
    dx, dw, _ = linear_grads(act, dy, x, w, z)
    bare = linear_grads("none", dy, x, w, z)
    sums = (K + 1) * ULP * ((x.abs() + STEP) @ (w.abs() + STEP))
    for right, without_slope, f, q in ((dx, bare[0], lambda t, v: act_value(act, (x + t * v) @ w), lambda v: v @ w),
                                       (dw, bare[1], lambda t, v: act_value(act, x @ (w + t * v)), lambda v: x @ v)):
        v = right.sign()
        d = float(((f(STEP, v) - f(-STEP, v)) * dy).sum()) / (2 * STEP)

        def share(g):   # of the bound
            own = float((HALF * g.abs() + 2.0 ** -25).sum())
            return abs(float((g * v).sum()) - d) / (difference_bound(act, dy, z, q(v), STEP, sums, HALF) + own)
        assert share(right) < 1
        for wrong in (torch.zeros_like(right), -right, without_slope):
            assert share(wrong) > 2
