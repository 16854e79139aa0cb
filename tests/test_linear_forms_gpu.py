"""Every form of the dense layers' products that a call can take (kernel, tile,
layout, whole or split sum, segments, terms, both products in one launch or
not: ``linear_cases``, which ``test_linear_plan_cpu`` holds to its coverage) on
integers whose products and sums are exact in FP32, bit for bit; once more
through the library built with LDS poisoning."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import binding, build, layers
from helpers import say
from layer_reference import gated_grads
from linear_cases import FORMS

pytestmark = pytest.mark.gpu
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


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


class Ints:
    """Integer matrices, a `share` of their elements nonzero, at bases `shift`
    bytes past a 16-byte boundary."""

    def __init__(self, seed, dtype, shift):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.shift = dtype, shift // 2

    def __call__(self, rows, cols, most, share=1.0):
        v = torch.randint(-most, most + 1, (rows, cols), generator=self.g, device="cuda")
        if share < 1:
            v = v * (torch.rand(rows, cols, generator=self.g, device="cuda") < share)
        flat = torch.empty(rows * cols + self.shift, dtype=self.dtype, device="cuda")
        view = flat[self.shift:].view(rows, cols)
        view.copy_(v)
        return view

    def weight(self, rows, cols, transposed, *a):
        return self(cols, rows, *a).t() if transposed else self(rows, cols, *a)


def same(got, ref, what):
    want = ref.to(got.dtype)
    assert bool((got == want).all()), f"{what}: {int((got != want).sum())} of {got.numel()} differ"


@pytest.mark.parametrize("n", range(len(FORMS)))
def test_form(n):
    op, fmt, M, N, K, t, act, shift, need, rounded = FORMS[n]
    say("form", n, FORMS[n])
    T = DTYPES[fmt]
    mk = Ints(n, T, shift)
    if op == "linear":
        x, w = mk(M, K, 2), mk.weight(K, N, t, 2)
        return same(dg.linear(x, w, out_dtype=torch.float32), x.double() @ w.double(), "y")
    if op == "gated":
        x, wg, wu = mk(M, K, 1), mk.weight(K, N, t, 1), mk.weight(K, N, t, 1)
        h, g, u = dg.gated(x, wg, wu, activation="none", save_pre=True)
        G, U = x.double() @ wg.double(), x.double() @ wu.double()
        same(g, G, "g")
        same(u, U, "u")
        return same(h, (G * U).float(), "h")
    # integers of more bits than a term holds, on one side at a time: the
    # gradient's, and where the other operand has terms too, that operand's
    for wide in ("gradient", "other") if fmt == "f16" and not rounded else ("gradient",):
        if op == "linear_backward":
            # silu's slope is a half at 0 and one at 100: exact, yet the gradient
            # of a call that computes it
            most = 1000 if wide == "gradient" and fmt == "f16" else (100 if wide == "gradient" else 1)
            x = mk(M, K, 1 if wide == "gradient" else 1000, 0.25)
            w = mk.weight(K, N, t, 1 if wide == "gradient" else 1000, 0.25)
            dy = mk(M, N, most)
            pre = mk(M, N, 1).abs() * 100 if act != "none" else None
            dz = dy.double() * (torch.where(pre.double() > 0, 1.0, 0.5) if act != "none" else 1.0)
            dx, dw, db = dg.linear_backward(dy, x, w, pre=pre, activation=act, need_input=need[0], need_weight=need[1],
                                            need_bias=need[1])
            if need[0]:
                same(dx, dz @ w.double().t(), "dx")
            if need[1]:
                same(dw, x.double().t() @ dz, "dw")
                same(db, dz.sum(0), "dbias")
            continue
        most = (3 if rounded else 40) if wide == "gradient" else 1
        dh, g, u = mk(M, N, most), mk(M, N, most), mk(M, N, most)
        x = mk(M, K, 1 if wide == "gradient" else 1000, 0.25)
        wg, wu = (mk.weight(K, N, t, 1 if wide == "gradient" else 1000, 0.25) for _ in range(2))
        got = dg.gated_backward(dh, x, wg, wu, g, u, activation="none", need_input=need[0], need_weight=need[1],
                                round_gradient=rounded)
        want = gated_grads("none", *(v.double() for v in (dh, x, wg, wu, g, u)))
        for a, b, name, is_needed in zip(got, want, ("dx", "dwg", "dwu"), (need[0], need[1], need[1])):
            if is_needed:
                same(a, b, name)


@pytest.mark.parametrize("off", ["x", "w", "both"])
@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [136, 520, 1032, 4104])
def test_bases_off_16_bytes_at_strides_on_them(K, dtype, transposed, off):
    """Operands that no ring loads and that are not copied: the plain tile's
    stages, splits and segments, with padded rows and without."""
    T = DTYPES[dtype]
    M, N = 128, 256
    at, on = Ints(K, T, 2), Ints(K + 1, T, 0)
    for pad in (0, 8):
        say("off 16", K, dtype, transposed, off, pad)
        def matrix(mk, rows, cols, most, share=1.0):
            return mk(rows, cols + pad, most, share)[:, :cols]
        def weight(mk, rows, cols, *a):
            return matrix(mk, cols, rows, *a).t() if transposed else matrix(mk, rows, cols, *a)
        mx, mw = at if off != "w" else on, at if off != "x" else on
        x, w = matrix(mx, M, K, 2), weight(mw, K, N, 2)
        same(dg.linear(x, w, out_dtype=torch.float32), x.double() @ w.double(), "y")
        dy = matrix(mx, M, N, 2)
        dx, dw, db = dg.linear_backward(dy, x, w)
        same(dx, dy.double() @ w.double().t(), "dx")
        same(dw, x.double().t() @ dy.double(), "dw")
        same(db, dy.double().sum(0), "dbias")
        x, wg, wu = matrix(mx, M, K, 1), weight(mw, K, N, 1), weight(mw, K, N, 1)
        G, U = x.double() @ wg.double(), x.double() @ wu.double()
        same(dg.gated(x, wg, wu, activation="none"), (G * U).float(), "h")
        # K gates: the input's gradient sums over them
        wg, wu = weight(mw, N, K, 1, 0.25), weight(mw, N, K, 1, 0.25)
        x, dh, g, u = matrix(mx, M, N, 1, 0.25), matrix(on, M, K, 40), matrix(on, M, K, 40), matrix(on, M, K, 40)
        got = dg.gated_backward(dh, x, wg, wu, g, u, activation="none")
        for a, b, name in zip(got, gated_grads("none", *(v.double() for v in (dh, x, wg, wu, g, u))), ("dx", "dwg", "dwu")):
            same(a, b, name)
