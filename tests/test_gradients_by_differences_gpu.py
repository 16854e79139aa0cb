"""The dense layer's gradients along a direction that they point in (their own
signs, from the formula) against differences of the kernels' own forward pass,
in FP32.  ``test_differences_cpu`` shows that the bounds reject a gradient of
zero, of the other sign and without the activation's slope."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from layer_reference import difference_bound, linear_grads

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -6       # exact in the inputs, which are multiples of 2^-6 below 8
HALF = 2.0 ** -11      # half a step of float16
ULP = 2.0 ** -24


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("size", [(24, 40, 64), (130, 72, 136)], ids=str)
def test_linear(size, act):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")
    say("by differences", size, act)
    M, N, K = size
    T = torch.float16
    g = torch.Generator(device="cuda").manual_seed(M)

    def grid(rows, cols, scale):
        return ((torch.randn(rows, cols, generator=g, device="cuda") * scale).clamp(-7, 7) * 64).round().div(64).to(T)
    x, w, dy = grid(M, K, 1.0), grid(K, N, K ** -0.5), grid(M, N, 1.0)
    pre = dg.linear(x, w, activation=act, save_pre=True)[1]
    dx, dw, _ = dg.linear_backward(dy, x, w, pre=pre, activation=act)
    X, W, D = x.double(), w.double(), dy.double()
    Z = X @ W
    want = linear_grads(act, D, X, W, Z)
    sums = (K + 1) * ULP * ((X.abs() + STEP) @ (W.abs() + STEP))
    for got, formula, moves, q in ((dx, want[0], lambda v, s: (x + s * v, w), lambda v: v.double() @ W),
                                   (dw, want[1], lambda v, s: (x, w + s * v), lambda v: X @ v.double())):
        v = formula.sign().to(T)
        f = [(dg.linear(*moves(v, s), activation=act, out_dtype=torch.float32).double() * D).sum()
             for s in (STEP, -STEP)]
        d = float(f[0] - f[1]) / (2 * STEP)
        along = float((got.double() * v.double()).sum())
        own = float((HALF * got.double().abs() + 2.0 ** -25).sum())     # the gradient's own rounding
        assert abs(along - d) <= difference_bound(act, D, Z, q(v), STEP, sums, HALF) + own
