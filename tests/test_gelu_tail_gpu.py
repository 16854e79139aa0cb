"""GELU's lower tail keeps its relative accuracy: z Phi(z) against the normal
distribution in 64 bits, z from -8 on, through the identity weight (whose
product is z itself).  In binary32 the value is held to (16 + 1.5 z^2) 2^-24 of
itself: the tail's fit and its evaluation, 8 units; the products by t, by a half
of the exponential and by z, a few more; and of the exponential of z^2 / 2 that
of its argument, which is off by 1.25 z^2 units."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say

pytestmark = pytest.mark.gpu
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_lower_tail_is_relatively_accurate(dtype):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")
    T = DTYPES[dtype]
    say("gelu tail", dtype)
    eye = torch.eye(64, dtype=T, device="cuda")
    sweep = torch.linspace(-8, 8, 64 * 96, device="cuda").view(96, 64).to(T)
    for rows in (sweep[:1], sweep[:24], sweep):            # the few-row kernel and the tiles
        Z = rows.double()
        ref = Z * 0.5 * torch.special.erfc(-Z * 0.5 ** 0.5)   # (ndtr is 1 + erf here: no tail below 1e-16)
        bound = (16 + 1.5 * Z.square()) * 2.0 ** -24 * ref.abs()
        y = dg.linear(rows, eye, activation="gelu", out_dtype=torch.float32).double()
        assert bool(((y - ref).abs() <= bound).all()), float(((y - ref).abs() / bound).max())
        y = dg.linear(rows, eye, activation="gelu").double()
        half = torch.where(ref.abs() >= torch.finfo(T).tiny, STEP[T] * (ref.abs() + bound), torch.finfo(T).tiny * STEP[T])
        assert bool(((y - ref).abs() <= bound + half).all())
        # the up projection's gradient is dH act(G): with one row of one at a
        # time it is the weight's gradient too
        one = torch.ones(1, 1, dtype=T, device="cuda")
        w = torch.zeros(1, 64, dtype=T, device="cuda")
        g = rows[:1].contiguous()
        du = dg.gated_backward(torch.ones_like(g), one, w, w, g, torch.ones_like(g), activation="gelu")[2].double()
        assert bool(((du[0] - ref[0]).abs() <= (bound + half + 2.0 ** -17 * ref.abs())[0]).all())
