"""The rings of the dense layer and the gated up-projection: every operand
layout on both tiles, with one to several stages, ragged edges in each
direction, sums over two pairs of operands and sums split over k.  Small
integers throughout (products and sums exact in FP32), so results are the
rounded exact ones bit for bit; once more through the library built with LDS
poisoning, where a read that runs ahead of its load or of the barrier that
retires a buffer returns NaN."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import binding, build, layers
from helpers import say
from layer_reference import gated_grads, linear_grads

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
DEPTHS = [8, 32, 40, 64, 72, 96, 136, 264]        # one to nine stages of 32, full and ragged
# rows and outputs: the 128 tile with ragged edges, more of its tiles than two a unit, the 256 tile
SIZES = [(264, 520), (1000, 2056), (4088, 4072)]


@pytest.fixture(scope="module", params=["product", "poisoned"], autouse=True)
def library(request):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")
    if request.param == "product":
        yield request.param
        return
    lib, load, kept = binding.load(build.POISON_LIB), binding.load, dict(layers._functions)
    layers._functions.clear()
    layers._FORMS.clear()
    binding.load = lambda *a: lib
    yield request.param
    binding.load = load
    layers._functions.clear()
    layers._FORMS.clear()
    layers._functions.update(kept)


def ints(g, rows, cols, dtype, low=-3, high=4):
    return torch.randint(low, high, (rows, cols), generator=g, device="cuda").to(dtype)


def weight(g, rows, cols, dtype, transposed):
    return ints(g, cols, rows, dtype).t() if transposed else ints(g, rows, cols, dtype)


def same(got, ref, what):
    want = ref.to(got.dtype)
    assert bool((got == want).all()), f"{what}: {int((got != want).sum())} of {got.numel()} differ"


@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_layer_and_its_gradients(size, dtype, transposed):
    M, N = size
    T = DTYPES[dtype]
    for K in DEPTHS:
        say("ring linear", size, K, dtype, transposed)
        g = torch.Generator(device="cuda").manual_seed(K)
        # K inputs, N outputs; then N inputs summed (dx) and K rows summed (dw)
        x, w, b = ints(g, M, K, T), weight(g, K, N, T, transposed), ints(g, 1, N, T)[0]
        r = ints(g, M, N, T)
        z = x.double() @ w.double() + b.double()
        y, pre = dg.linear(x, w, bias=b, residual=r, activation="relu", save_pre=True)
        same(pre, z, "pre")
        same(y, z.clamp(min=0) + r.double(), "y")
        # outputs M x N over K: the input's gradient of a layer of N inputs and K outputs
        w2, dy, pre2, x2 = weight(g, N, K, T, transposed), ints(g, M, K, T), ints(g, M, K, T), ints(g, M, N, T)
        dx = dg.linear_backward(dy, x2, w2, pre=pre2, activation="relu", need_weight=False, need_bias=False)[0]
        same(dx, linear_grads("relu", dy.double(), x2.double(), w2.double(), pre2.double())[0], "dx")
        # outputs M x N over K rows: the weight's gradient
        dz, x3 = ints(g, K, N, T), ints(g, K, M, T)
        w3 = weight(g, M, N, T, transposed)
        dw = dg.linear_backward(dz, x3, w3, need_input=False, need_bias=False)[1]
        same(dw, x3.double().t() @ dz.double(), "dw")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [(264, 264), (1000, 1032), (4088, 2040)], ids=str)
def test_gated_and_its_gradients(size, dtype, transposed):
    M, F = size
    T = DTYPES[dtype]
    for K in DEPTHS:
        say("ring gated", size, K, dtype, transposed)
        g = torch.Generator(device="cuda").manual_seed(K)
        x, wg, wu = ints(g, M, K, T), weight(g, K, F, T, transposed), weight(g, K, F, T, transposed)
        h, gs, us = dg.gated(x, wg, wu, activation="relu", save_pre=True)
        G, U = x.double() @ wg.double(), x.double() @ wu.double()
        same(gs, G, "g")
        same(us, U, "u")
        same(h, (G.clamp(min=0) * U).float(), "h")
        # K gates: the sum of the input's gradient runs over both pairs
        wg, wu = weight(g, 2 * F, K, T, transposed), weight(g, 2 * F, K, T, transposed)
        dh, g2, u2 = ints(g, M, K, T), ints(g, M, K, T, -1, 2), ints(g, M, K, T, -1, 2)
        x2 = ints(g, M, 2 * F, T)
        dx = dg.gated_backward(dh, x2, wg, wu, g2, u2, activation="relu", need_weight=False)[0]
        want = gated_grads("relu", *(t.double() for t in (dh, x2, wg, wu, g2, u2)))
        same(dx, want[0], "dx")
        # K rows: both weights' gradients
        x3, dh, g3, u3 = ints(g, K, M, T), ints(g, K, F, T), ints(g, K, F, T, -1, 2), ints(g, K, F, T, -1, 2)
        wg, wu = weight(g, M, F, T, transposed), weight(g, M, F, T, transposed)
        got = dg.gated_backward(dh, x3, wg, wu, g3, u3, activation="relu", need_input=False)
        want = gated_grads("relu", *(t.double() for t in (dh, x3, wg, wu, g3, u3)))
        same(got[1], want[1], "dwg")
        same(got[2], want[2], "dwu")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [(136, 264, 1032), (264, 136, 4104), (520, 520, 2000)], ids=str)
def test_sums_split_over_k(size, dtype):
    M, N, K = size
    T = DTYPES[dtype]
    for transposed in (False, True):
        say("ring split", size, dtype, transposed)
        g = torch.Generator(device="cuda").manual_seed(K)
        x, w = ints(g, M, K, T), weight(g, K, N, T, transposed)
        y = dg.linear(x, w, activation="relu", out_dtype=torch.float32)
        same(y, (x.double() @ w.double()).clamp(min=0), "y")
        # both pairs of a gated layer's input gradient, and both weights' gradients
        wg, wu = weight(g, N, K, T, transposed), weight(g, N, K, T, transposed)
        dh, gs, us = (ints(g, M, K, T, -1, 2) for _ in range(3))
        x = ints(g, M, N, T)
        got = dg.gated_backward(dh, x, wg, wu, gs, us, activation="relu")
        want = gated_grads("relu", *(t.double() for t in (dh, x, wg, wu, gs, us)))
        for a, b, name in zip(got, want, ("dx", "dwg", "dwu")):
            same(a, b, name)
        x, dz, w = ints(g, K, M, T, -1, 2), ints(g, K, N, T, -1, 2), weight(g, M, N, T, transposed)
        dw = dg.linear_backward(dz, x, w, need_input=False, need_bias=False)[1]
        same(dw, x.double().t() @ dz.double(), "dw")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [(72, 72, 72), (528, 2752, 792), (377, 6424, 256), (264, 96, 4104), (1016, 1008, 1024),
                                  (1, 64, 8), (3, 1344, 1632), (16, 248, 640), (64, 128, 3520), (3266, 3512, 64),
                                  (496, 1024, 4288)],
                         ids=str)
def test_both_gradients_of_a_pass(size, dtype, transposed):
    # small passes run both products in one launch: each tile, one or both
    # sums split, edges in each direction, and replayed from a graph
    M, K, N = size
    T = DTYPES[dtype]
    say("ring pair", size, dtype, transposed)
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w, dy = ints(g, M, K, T, -1, 2), weight(g, K, N, T, transposed), ints(g, M, N, T, -1, 2)
    dx, dw, db = dg.linear_backward(dy, x, w)
    same(dx, dy.double() @ w.double().t(), "dx")
    same(dw, x.double().t() @ dy.double(), "dw")
    same(db, dy.double().sum(0), "dbias")
    wu, gs, us = weight(g, K, N, T, transposed), ints(g, M, N, T, -1, 2), ints(g, M, N, T, -1, 2)
    want = gated_grads("relu", *(t.double() for t in (dy, x, w, wu, gs, us)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dg.gated_backward(dy, x, w, wu, gs, us, activation="relu")
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, name in zip(got, want, ("dx", "dwg", "dwu")):
            same(a, b, name)
