"""The dense layers of few rows: every count of row blocks, both storages of
the weights, strips that end inside a matrix, sums that end inside a chunk or
are shorter than one, sums over two pairs, unaligned rows.  Small integers:
bit for bit the rounded exact results."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from layer_reference import gated_grads, linear_grads

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEPTHS = [1, 7, 31, 64, 72, 129, 512, 577, 1031, 4096, 4168]
COLUMNS = [1, 9, 16, 40, 257]


@pytest.fixture(autouse=True, scope="module")
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")


def ints(g, rows, cols, dtype, pad=0, low=-2, high=3):
    t = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :cols] = torch.randint(low, high, (rows, cols), generator=g, device="cuda").to(dtype)
    return t[:, :cols]


def weight(g, rows, cols, dtype, transposed, pad=0):
    return ints(g, cols, rows, dtype, pad).t() if transposed else ints(g, rows, cols, dtype, pad)


def same(got, ref, what):
    want = ref.to(got.dtype)
    assert bool((got == want).all()), f"{what}: {int((got != want).sum())} of {got.numel()} differ"


@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 33, 48, 64])
def test_rows(M, dtype, transposed):
    T = DTYPES[dtype]
    for K in DEPTHS:
        for N in COLUMNS + ([8200] if K in (72, 577) else []):
            pad = (K + N) % 4
            say("rows", M, K, N, dtype, transposed, pad)
            g = torch.Generator(device="cuda").manual_seed(K * 31 + N)
            x, w, b = ints(g, M, K, T, pad), weight(g, K, N, T, transposed, pad), ints(g, 1, N, T)[0].contiguous()
            r = ints(g, M, N, torch.float32)
            z = x.double() @ w.double() + b.double()
            y, pre = dg.linear(x, w, bias=b, residual=r, activation="relu", save_pre=True, out_dtype=torch.float32)
            same(pre, z, "pre")
            same(y, z.clamp(min=0) + r.double(), "y")
            dy = ints(g, M, N, T, pad)
            dx = dg.linear_backward(dy, x, w, need_weight=False, need_bias=False)[0]
            same(dx, linear_grads("none", dy.double(), x.double(), w.double(), dy.double())[0], "dx")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 16, 30, 48, 64])
def test_gated_rows(M, dtype, transposed):
    T = DTYPES[dtype]
    for K in DEPTHS:
        for F in COLUMNS:
            pad = (K + F) % 4
            say("gated rows", M, K, F, dtype, transposed, pad)
            g = torch.Generator(device="cuda").manual_seed(K * 31 + F)
            x = ints(g, M, K, T, pad)
            x[:, 300:] = 0                       # the product of both sums stays below 2^24
            wg, wu = weight(g, K, F, T, transposed, pad), weight(g, K, F, T, transposed, pad)
            h, gs, us = dg.gated(x, wg, wu, activation="relu", save_pre=True)
            G, U = x.double() @ wg.double(), x.double() @ wu.double()
            same(gs, G, "g")
            same(us, U, "u")
            same(h, (G.clamp(min=0) * U).float(), "h")
            # the input's gradient: a sum over both pairs, of K gates
            wg, wu = weight(g, F, K, T, transposed, pad), weight(g, F, K, T, transposed, pad)
            dh, g2, u2 = ints(g, M, K, T, pad), ints(g, M, K, T, pad), ints(g, M, K, T, pad)
            x2 = ints(g, M, F, T, pad)
            dx = dg.gated_backward(dh, x2, wg, wu, g2, u2, activation="relu", need_weight=False)[0]
            same(dx, gated_grads("relu", *(t.double() for t in (dh, x2, wg, wu, g2, u2)))[0], "dx")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [65, 130, 300])
def test_tiles_with_narrow_and_cut_operands(M, dtype, transposed):
    """More rows than the strips take, with rows shorter than a 16-byte unit
    or cut by one, of each operand of the three products."""
    T = DTYPES[dtype]
    for K in (1, 3, 7, 8, 9, 15, 63, 65, 130, 329):
        for N in (1, 7, 8, 15, 65, 131):
            pad = (K + N) % 4
            say("narrow", M, K, N, dtype, transposed, pad)
            g = torch.Generator(device="cuda").manual_seed(K * 31 + N)
            x, w, dy = ints(g, M, K, T, pad), weight(g, K, N, T, transposed, pad), ints(g, M, N, T, pad)
            same(dg.linear(x, w, out_dtype=torch.float32), x.double() @ w.double(), "y")
            want = linear_grads("none", dy.double(), x.double(), w.double(), dy.double())
            for got, ref, name in zip(dg.linear_backward(dy, x, w), want, ("dx", "dw", "dbias")):
                same(got, ref, name)
            wu, gs, us = weight(g, K, N, T, transposed, pad), ints(g, M, N, T, pad), ints(g, M, N, T, pad)
            h = dg.gated(x, w, wu, activation="none")
            same(h, ((x.double() @ w.double()) * (x.double() @ wu.double())).float(), "h")
            want = gated_grads("relu", *(t.double() for t in (dy, x, w, wu, gs, us)))
            for got, ref, name in zip(dg.gated_backward(dy, x, w, wu, gs, us, activation="relu"), want,
                                      ("dx", "dwg", "dwu")):
                same(got, ref, name)
