"""The dense layer, the gated up-projection and layer norm, forward and
backward, against their formulas in 64 bits.

Small-integer operands (products and sums exact in FP32, no activation or
relu) have to give the rounded exact result bit for bit, whatever kernel,
split or edge a size takes.  Real-valued ones are held to a bound:

* a sum of K products errs by at most K 2^-24 times the sum of their
  magnitudes (FP32 additions, products exact);
* an activation errs by at most 4e-7 |z| beyond its argument's error times its
  largest slope, 1.13 (the normal tail's published 1.5e-7, and a few units of
  2^-24 of the exponential, the reciprocal and the products);
* a slope errs by at most 2e-6, and a value rounded to 16 bits by half a step
  (2^-8 or 2^-11 of it, or half the smallest subnormal).
"""
import numpy as np
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say
from layer_reference import act_slope, act_value, gated_grads, layer_norm_grads, linear_grads

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}
ULP = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]

# rows, outputs, inputs: single elements, odd sizes off every vector, single
# tokens, whole tiles, ragged tiles, sums of one stage and of many
SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 64), (1, 1000, 777), (2, 264, 1032), (16, 128, 512), (33, 100, 72),
          (64, 256, 520), (65, 72, 4096), (129, 130, 131), (200, 1024, 1032), (257, 300, 264), (520, 520, 136)]
LARGE = [(1000, 1032, 1096), (2056, 2176, 200), (4096, 2048, 72)]


@pytest.fixture(autouse=True, scope="module")
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")


class Make:
    """Inputs from a seed: small integers or normal values, as views with
    padded rows (holding NaN) and bases off 16 bytes where asked."""

    def __init__(self, seed, dtype, integer, pad=0, shift=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.integer, self.pad, self.shift = dtype, integer, pad, shift

    def values(self, rows, cols, scale=1.0):
        if self.integer:
            return torch.randint(-4, 5, (rows, cols), generator=self.g, device="cuda").to(self.dtype)
        return (torch.randn(rows, cols, generator=self.g, device="cuda") * scale).to(self.dtype)

    def matrix(self, rows, cols, scale=1.0, dtype=None):
        v = self.values(rows, cols, scale).to(dtype or self.dtype)
        if not self.pad and not self.shift:
            return v
        flat = torch.full((rows * (cols + self.pad) + self.shift,), float("nan"), dtype=v.dtype, device="cuda")
        view = flat[self.shift:].view(rows, cols + self.pad)[:, :cols]
        view.copy_(v)
        return view

    def weight(self, rows, cols, transposed):
        scale = rows ** -0.5
        return self.matrix(cols, rows, scale).t() if transposed else self.matrix(rows, cols, scale)

    def vector(self, n):
        return self.values(1, n)[0].contiguous()


def held(shape, dtype, pad, shift):
    """An output view with padded rows in a larger buffer of a mark, and a
    check that nothing around it was written."""
    rows, cols = shape
    flat = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=dtype, device="cuda")
    view = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def intact():
        rest = flat.clone()
        rest[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = 7.0
        return bool((rest == 7.0).all())
    return view, intact


def exact(got, ref, what):
    want = ref.to(got.dtype)
    assert got.shape == want.shape and bool((got == want).all()), \
        f"{what}: {int((got != want).sum())} of {got.numel()} differ"


def within(got, ref, err, what):
    """|got - ref| at most err (before the rounding to got's type) and half a step."""
    tol = err + (ref.abs() + err) * STEP[got.dtype] + TINY[got.dtype]
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    assert bool((off <= tol).all()), f"{what}: worst {float((off / tol).max()):.3g} of the bound"


def sum_err(a, b):
    """Bound of the error of a @ b summed in FP32."""
    return a.shape[1] * ULP * (a.abs() @ b.abs())


def act_err(act, z, dz):
    return dz if act in ("none",) else 1.13 * dz + 4e-7 * z.abs()


# ------------------------------------------------------------- dense layer --

@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE, ids=str)
def test_linear_is_exact_on_integers(shape, dtype, transposed):
    M, N, K = shape
    T = DTYPES[dtype]
    for case, (act, bias, res, f32, pad, shift) in enumerate([
            ("none", False, False, True, 0, 0), ("relu", True, True, True, 0, 0), ("none", True, True, False, 8, 0),
            ("relu", True, False, False, 3, 1)]):
        say("linear", shape, dtype, transposed, case)
        mk = Make(100 + case, T, True, pad, shift)
        x, w = mk.matrix(M, K), mk.weight(K, N, transposed)
        b = mk.vector(N) if bias else None
        out_t = torch.float32 if f32 else T
        r = mk.matrix(M, N, dtype=out_t) if res else None
        y, intact = held((M, N), out_t, pad, shift)
        z = x.double() @ w.double() + (b.double() if bias else 0)
        got, pre = dg.linear(x, w, bias=b, residual=r, activation=act, out_dtype=out_t, y=y, save_pre=True)
        ref = act_value(act, z) + (r.double() if res else 0)
        exact(got, ref, "y")
        exact(pre, z, "pre")
        assert intact()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 264, 1032), (5, 33, 777), (40, 512, 1000), (300, 520, 264), (1000, 1032, 520)],
                         ids=str)
def test_linear_activations(shape, dtype, act):
    M, N, K = shape
    T = DTYPES[dtype]
    for f32 in (False, True):
        say("linear act", shape, dtype, act, f32)
        mk = Make(7, T, False)
        x, w, b = mk.matrix(M, K, 2.0), mk.weight(K, N, f32), mk.vector(N)
        r = mk.matrix(M, N, dtype=torch.float32 if f32 else T)
        y, pre = dg.linear(x, w, bias=b, residual=r, activation=act, save_pre=True,
                           out_dtype=torch.float32 if f32 else None)
        X, W = x.double(), w.double()
        z = X @ W + b.double()
        dz = sum_err(X, W) + ULP * z.abs()
        within(pre, z, dz, "pre")
        v = act_value(act, z)
        e = act_err(act, z, dz)
        within(y, v + r.double(), e + ULP * (v + r.double()).abs(), "y")


def test_linear_adds_into_its_residual_in_place():
    mk = Make(3, torch.bfloat16, True)
    for M, N, K in ((1, 520, 1032), (70, 136, 72), (700, 1032, 264)):
        say("in place", M, N, K)
        x, w, y = mk.matrix(M, K), mk.weight(K, N, False), mk.matrix(M, N)
        ref = x.double() @ w.double() + y.double()
        assert dg.linear(x, w, residual=y, y=y) is y
        exact(y, ref, "y")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxN", "NxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE[:2], ids=str)
def test_linear_backward_is_exact_on_integers(shape, dtype, transposed):
    M, N, K = shape
    T = DTYPES[dtype]
    for act, pad, shift in (("none", 0, 0), ("relu", 8, 0), ("relu", 5, 1)):
        say("linear backward", shape, dtype, transposed, act, pad)
        mk = Make(11, T, True, pad, shift)
        x, w, dy = mk.matrix(M, K), mk.weight(K, N, transposed), mk.matrix(M, N)
        pre = mk.matrix(M, N) if act != "none" else None
        z = pre.double() if pre is not None else None
        want = linear_grads(act, dy.double(), x.double(), w.double(), torch.zeros_like(dy).double() if z is None else z)
        dx_out, intact = held((M, K), T, pad, shift)
        dx, dw, db = dg.linear_backward(dy, x, w, pre=pre, activation=act, dx=dx_out)
        for got, ref, name in zip((dx, dw, db), want, ("dx", "dw", "dbias")):
            exact(got, ref, name)
        assert intact()
        assert dw.stride() == (w.stride() if not pad else dw.stride()) or min(dw.shape) == 1


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 264, 1032), (77, 520, 131), (520, 264, 1000)], ids=str)
def test_linear_backward_slopes(shape, dtype, act):
    M, N, K = shape
    T = DTYPES[dtype]
    say("linear backward act", shape, dtype, act)
    mk = Make(12, T, False)
    x, w, dy, pre = mk.matrix(M, K), mk.weight(K, N, False), mk.matrix(M, N), mk.matrix(M, N, 3.0)
    X, W, D, Z = x.double(), w.double(), dy.double(), pre.double()
    dx, dw, db = dg.linear_backward(dy, x, w, pre=pre, activation=act)
    want = linear_grads(act, D, X, W, Z)
    slope = act_slope(act, Z)
    e = D.abs() * 2e-6 + ULP * (D * slope).abs()                       # before dZ's rounding
    r = e + ((D * slope).abs() + e) * STEP[T] + TINY[T]                # and after it
    dz = (D * slope).abs() + r
    within(dx, want[0], r @ W.abs().t() + N * ULP * (dz @ W.abs().t()), "dx")
    within(dw, want[1], X.abs().t() @ r + M * ULP * (X.abs().t() @ dz), "dw")
    within(db, want[2], e.sum(0) + M * ULP * dz.sum(0), "dbias")


def test_linear_backward_computes_only_what_is_asked():
    mk = Make(4, torch.float16, True)
    x, w, dy = mk.matrix(40, 72), mk.weight(72, 64, False), mk.matrix(40, 64)
    want = linear_grads("none", dy.double(), x.double(), w.double(), dy.double())
    for need in range(8):
        say("asked", need)
        got = dg.linear_backward(dy, x, w, need_input=bool(need & 1), need_weight=bool(need & 2),
                                 need_bias=bool(need & 4))
        for i in range(3):
            if need >> i & 1:
                exact(got[i], want[i], str(i))
            else:
                assert got[i] is None


def test_linear_of_nothing():
    T = torch.bfloat16
    x = torch.empty(0, 16, dtype=T, device="cuda")
    w = torch.ones(16, 8, dtype=T, device="cuda")
    assert dg.linear(x, w).shape == (0, 8)
    dx, dw, db = dg.linear_backward(torch.empty(0, 8, dtype=T, device="cuda"), x, w)
    assert dx.shape == (0, 16) and bool((dw == 0).all()) and bool((db == 0).all())
    # no inputs: the sum is empty, bias and residual remain
    x, w = torch.empty(5, 0, dtype=T, device="cuda"), torch.empty(0, 8, dtype=T, device="cuda")
    b, r = torch.full((8,), -2.0, dtype=T, device="cuda"), torch.full((5, 8), 3.0, dtype=T, device="cuda")
    assert bool((dg.linear(x, w, bias=b, residual=r, activation="relu") == 3.0).all())
    # no outputs: the input's gradient is zero
    x, w = torch.ones(5, 16, dtype=T, device="cuda"), torch.empty(16, 0, dtype=T, device="cuda")
    dx, dw, db = dg.linear_backward(torch.empty(5, 0, dtype=T, device="cuda"), x, w)
    assert dx.shape == (5, 16) and bool((dx == 0).all()) and dw.shape == (16, 0) and db.shape == (0,)


def test_extreme_values_stay_in_their_place():
    """An infinity or NaN in one row reaches that row's outputs only; the
    largest finite values go through every activation and slope."""
    T = torch.bfloat16
    for M, N, K in ((1, 136, 264), (20, 136, 264), (300, 264, 136)):
        say("extreme", M, N, K)
        mk = Make(9, T, True)
        x, w = mk.matrix(M, K), mk.weight(K, N, False)
        bad = x.clone()
        bad[M - 1, K - 1] = float("nan")
        y = dg.linear(bad, w)
        assert bool(torch.isnan(y[M - 1]).all())
        if M > 1:
            exact(y[:M - 1], (x.double() @ w.double())[:M - 1], "other rows")
    big = torch.finfo(T).max
    z = torch.tensor([[-big, big, -100.0, 100.0, -1e-30, 1e-30, 0.0, -0.0]], dtype=T, device="cuda")
    eye = torch.eye(8, dtype=T, device="cuda")
    for act in ACTS[1:]:
        # the identity weight gives z itself
        y = dg.linear(z, eye, activation=act).double()
        ref = torch.where(z.double() < -50, 0.0, act_value(act, z.double().clamp(-50, 50)))
        ref = torch.where(z.double() > 50, z.double(), ref)
        assert bool(((y - ref).abs() <= ref.abs() * 2.0 ** -7 + 1e-30).all()), (act, y, ref)
        one = torch.ones_like(z)
        dx = dg.linear_backward(one, z, eye, pre=z, activation=act)[0].double()
        slope = torch.where(z.double() > 50, 1.0, torch.where(z.double() < -50, 0.0,
                                                              act_slope(act, z.double().clamp(-50, 50))))
        assert bool(((dx - slope).abs() <= slope.abs() * 2.0 ** -8 + 1e-6).all()), (act, dx, slope)


# ---------------------------------------------------- gated up-projection --

@pytest.mark.parametrize("transposed", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE, ids=str)
def test_gated_is_exact_on_integers(shape, dtype, transposed):
    M, F, K = shape
    T = DTYPES[dtype]
    for act, pad, shift in (("none", 0, 0), ("relu", 8, 0), ("relu", 3, 1)):
        say("gated", shape, dtype, transposed, act, pad)
        mk = Make(21, T, True, pad, shift)
        x = mk.matrix(M, K)
        wg, wu = mk.weight(K, F, transposed), mk.weight(K, F, transposed)
        # inputs past 256 are zero: the product of both sums stays below 2^24
        x[:, 256:] = 0
        out, intact = held((M, F), T, pad, shift)
        g, u = x.double() @ wg.double(), x.double() @ wu.double()
        h, gs, us = dg.gated(x, wg, wu, activation=act, save_pre=True, h=out)
        exact(gs, g, "g")
        exact(us, u, "u")
        exact(h, (act_value(act, g) * u).float(), "h")
        assert intact()


def test_gated_takes_the_halves_of_one_weight():
    mk = Make(5, torch.float16, True)
    for M, F, K in ((1, 264, 136), (50, 136, 72), (600, 520, 136)):
        say("halves", M, F, K)
        x, w = mk.matrix(M, K), mk.matrix(K, 2 * F)
        g, u = x.double() @ w[:, :F].double(), x.double() @ w[:, F:].double()
        exact(dg.gated(x, w[:, :F], w[:, F:], activation="relu"), (g.clamp(min=0) * u).float(), "h")


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 264, 1032), (77, 131, 520), (520, 1032, 264)], ids=str)
def test_gated_activations_and_gradients(shape, dtype, act):
    M, F, K = shape
    T = DTYPES[dtype]
    say("gated act", shape, dtype, act)
    mk = Make(22, T, False)
    x, wg, wu, dh = mk.matrix(M, K), mk.weight(K, F, False), mk.weight(K, F, False), mk.matrix(M, F)
    X, A, B, D = x.double(), wg.double(), wu.double(), dh.double()
    h, g, u = dg.gated(x, wg, wu, activation=act, save_pre=True)
    G, U = X @ A, X @ B
    eg, eu = sum_err(X, A), sum_err(X, B)
    within(g, G, eg, "g")
    within(u, U, eu, "u")
    ev = act_err(act, G, eg)
    v = act_value(act, G)
    within(h, v * U, ev * (U.abs() + eu) + v.abs() * eu + ULP * (v * U).abs(), "h")
    # the gradients are those at the saved, rounded products
    G, U = g.double(), u.double()
    dx, dwg, dwu = dg.gated_backward(dh, x, wg, wu, g, u, activation=act)
    want = gated_grads(act, D, X, A, B, G, U)
    dg_, du = D * U * act_slope(act, G), D * act_value(act, G)
    e1 = (D * U).abs() * 2e-6 + 2 * ULP * dg_.abs()
    e2 = D.abs() * 4e-7 * G.abs() + 2 * ULP * du.abs()
    r1 = e1 + (dg_.abs() + e1) * STEP[T] + TINY[T]
    r2 = e2 + (du.abs() + e2) * STEP[T] + TINY[T]
    m1, m2 = dg_.abs() + r1, du.abs() + r2
    within(dx, want[0], r1 @ A.abs().t() + r2 @ B.abs().t() + 2 * F * ULP * (m1 @ A.abs().t() + m2 @ B.abs().t()),
           "dx")
    within(dwg, want[1], X.abs().t() @ r1 + M * ULP * (X.abs().t() @ m1), "dwg")
    within(dwu, want[2], X.abs().t() @ r2 + M * ULP * (X.abs().t() @ m2), "dwu")


@pytest.mark.parametrize("transposed", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + LARGE[:2], ids=str)
def test_gated_backward_is_exact_on_integers(shape, dtype, transposed):
    M, F, K = shape
    T = DTYPES[dtype]
    for act, pad, shift in (("none", 0, 0), ("relu", 8, 0), ("relu", 5, 1)):
        say("gated backward", shape, dtype, transposed, act, pad)
        mk = Make(23, T, True, pad, shift)
        x, dh, g, u = mk.matrix(M, K), mk.matrix(M, F), mk.matrix(M, F), mk.matrix(M, F)
        wg, wu = mk.weight(K, F, transposed), mk.weight(K, F, transposed)
        want = gated_grads(act, *(t.double() for t in (dh, x, wg, wu, g, u)))
        dx_out, intact = held((M, K), T, pad, shift)
        got = dg.gated_backward(dh, x, wg, wu, g, u, activation=act, dx=dx_out)
        for t, ref, name in zip(got, want, ("dx", "dwg", "dwu")):
            exact(t, ref, name)
        assert intact()


# --------------------------------------------------------------- layer norm --

NORM_SHAPES = [(1, 1), (1, 64), (3, 7), (5, 513), (70, 512), (9, 1000), (130, 1024), (3, 1500), (700, 777),
               (1100, 2048), (4, 4096), (600, 4097), (3, 8000), (2, 16384), (2, 16385), (40, 20001),
               # several turns of each form of the backward kernel
               (300, 9000), (5000, 513), (5000, 200), (700, 8192), (700, 3000)]


@pytest.mark.parametrize("dtype,weight_f32", [("f32", True), ("f16", False), ("f16", True), ("bf16", False),
                                              ("bf16", True)])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_layer_norm_and_its_gradients(shape, dtype, weight_f32):
    M, N = shape
    T = DTYPES[dtype]
    for pad, shift, offset in ((0, 0, 0.0), (3, 1, 20.0)):
        say("layer norm", shape, dtype, weight_f32, pad)
        mk = Make(31, T, False, pad, shift)
        x, dy = mk.matrix(M, N), mk.matrix(M, N)
        x += offset
        wt = torch.float32 if weight_f32 else T
        w, bias = (mk.vector(N).float() + 1).to(wt), mk.vector(N).to(wt)
        out, intact = held((M, N), T, pad, shift)
        y, mean, rstd = dg.layer_norm(x, w, bias, eps=1e-5, save_stats=True, y=out)
        X, W, B, D = x.double(), w.double(), bias.double(), dy.double()
        mu = X.mean(1)
        var = ((X - mu[:, None]) ** 2).mean(1)
        rs = 1 / torch.sqrt(var + 1e-5)
        # a row's sums: 8 V additions of a thread, 64 at most, and 9 of the
        # tree, past 16384 elements N / 2048 times 8 of a thread
        chain = (64 + 10 if N <= 16384 else 8 * (N // 2048 + 1) + 10) * ULP
        e_mu = chain * X.abs().mean(1) + ULP * mu.abs()
        within(mean, mu, e_mu, "mean")
        e_c = e_mu[:, None] + ULP * (X - mu[:, None]).abs()            # of x - mean
        e_var = (2 * e_c * (X - mu[:, None]).abs() + e_c ** 2).mean(1) + chain * var
        e_rs = rs * (e_var * rs ** 2 / 2 + 4 * ULP)
        within(rstd, rs, e_rs, "rstd")
        xh = (X - mu[:, None]) * rs[:, None]
        e_xh = e_c * rs[:, None] + xh.abs() * (e_rs / rs)[:, None] + ULP * xh.abs()
        within(y, xh * W + B, e_xh * W.abs() + 2 * ULP * ((xh * W).abs() + B.abs()), "y")
        assert intact()
        # gradients at the statistics as given
        mu, rs = mean.double(), rstd.double()
        dx_out, intact = held((M, N), T, pad, shift)
        dx, dw, db = dg.layer_norm_backward(dy, x, w, mean, rstd, dx=dx_out)
        want = layer_norm_grads(D, X, W, mu, rs)
        xh = (X - mu[:, None]) * rs[:, None]
        e_xh = 3 * ULP * (xh.abs() + (X.abs() + mu.abs()[:, None]) * rs[:, None])
        t = D * W
        e_t = ULP * t.abs()
        e_1 = (e_t.mean(1) + (chain + ULP) * t.abs().mean(1))[:, None]
        th = (t * xh).abs()
        e_2 = ((e_t * xh.abs() + t.abs() * e_xh).mean(1) + (chain + ULP) * th.mean(1))[:, None]
        c2 = (t * xh).mean(1, keepdim=True).abs()
        mag = t.abs() + t.mean(1, keepdim=True).abs() + xh.abs() * c2
        within(dx, want[0], rs[:, None] * (e_t + e_1 + xh.abs() * e_2 + e_xh * (c2 + e_2) + 5 * ULP * mag), "dx")
        rows = (M // 512 + 1 + 100) * ULP                               # a workgroup's rows, then the join
        if N > 16384:
            rows = (M + 100) * ULP
        within(dw, want[1], (D.abs() * e_xh).sum(0) + rows * (D * xh).abs().sum(0), "dw")
        within(db, want[2], rows * D.abs().sum(0), "db")
        assert intact()


def test_layer_norm_without_weights_and_of_constant_rows():
    x = torch.full((5, 300), 3.0, device="cuda")
    y, mean, rstd = dg.layer_norm(x, save_stats=True)
    assert bool((y == 0).all()) and bool((mean == 3.0).all())
    assert bool(((rstd.double() * 1e-5 ** 0.5 - 1).abs() < 1e-6).all())
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = torch.randn(6, 2, 40, generator=g, device="cuda"), torch.randn(6, 2, 40, generator=g, device="cuda")
    y, mean, rstd = dg.layer_norm(x, save_stats=True)
    assert mean.shape == (6, 2) and y.shape == x.shape
    dx, dw, db = dg.layer_norm_backward(dy, x, None, mean, rstd)
    want = layer_norm_grads(dy.double().view(12, 40), x.double().view(12, 40), None, mean.double().view(-1),
                            rstd.double().view(-1))
    for got, ref in zip((dx.view(12, 40), dw, db), want):
        assert float((got.double() - ref).abs().max()) < 1e-5     # values of order 10, 2^-24 each
    dx, dw, db = dg.layer_norm_backward(dy, x, None, mean, rstd, need_weight=False)
    assert dw is None and db is None
    # no rows: the weight gradients are zero
    e = torch.empty(0, 40, device="cuda")
    dx, dw, db = dg.layer_norm_backward(e, e, torch.ones(40, device="cuda"), e[:, 0].contiguous(),
                                        e[:, 0].contiguous())
    assert dx.shape == (0, 40) and bool((dw == 0).all()) and bool((db == 0).all())


def test_layer_norm_of_nonfinite_rows_leaves_the_others():
    x = torch.randn(9, 700, device="cuda")
    ref = dg.layer_norm(x)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[4, 699] = bad
        y = dg.layer_norm(z)
        assert bool(torch.isnan(y[4]).any())
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(y[keep], ref[keep])


# ------------------------------------------- streams, graphs, determinism --

def _sublayer(p, x, dy):
    """A pre-norm feed-forward sublayer, forward and backward."""
    n, mean, rstd = dg.layer_norm(x, p["nw"], p["nb"], save_stats=True)
    h, g, u = dg.gated(n, p["wg"], p["wu"], save_pre=True)
    y = dg.linear(h, p["wd"], residual=x)
    dh, dwd, _ = dg.linear_backward(dy, h, p["wd"], need_bias=False)
    dn, dwg, dwu = dg.gated_backward(dh, n, p["wg"], p["wu"], g, u)
    dx, dnw, dnb = dg.layer_norm_backward(dn, x, p["nw"], mean, rstd)
    return y, dx + dy, dwd, dwg, dwu, dnw, dnb


def _sublayer_inputs(M, seed=41):
    mk = Make(seed, torch.bfloat16, False)
    K, F = 264, 520
    p = dict(nw=mk.vector(K), nb=mk.vector(K), wg=mk.weight(K, F, False), wu=mk.weight(K, F, False),
             wd=mk.weight(F, K, True))
    return p, mk.matrix(M, K), mk.matrix(M, K)


def test_sublayer_on_another_stream_and_again_gives_the_same_bits():
    p, x, dy = _sublayer_inputs(300)
    first = _sublayer(p, x, dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = _sublayer(p, x, dy)
    s.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    # a stream handed to the call itself
    y = dg.linear(x, p["wg"], stream=s)
    s.synchronize()
    assert torch.equal(y, dg.linear(x, p["wg"]))


@pytest.mark.parametrize("M", [1, 300])
def test_sublayer_in_a_graph_replays_as_it_runs(M):
    p, x, dy = _sublayer_inputs(M)
    _sublayer(p, x, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _sublayer(p, x, dy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _sublayer(p, x, dy)
    for trial in range(4):
        _, nx, ndy = _sublayer_inputs(M, 50 + trial)
        x.copy_(nx)
        dy.copy_(ndy)
        eager = _sublayer(p, x, dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b), trial


def test_gradients_match_differences_of_the_kernels_own_forward():
    """<dx, v> against central differences of <dy, layer(x)> in FP32 outputs:
    the step 2^-4 is exact in float16, the products' third derivatives along v
    are below 10, so the differences err by less than 2 (2^-4)^2 of the terms'
    size, and the FP32 sums by 2^-20 over the step."""
    T = torch.float16
    mk = Make(61, T, False)
    M, N, K = 24, 40, 64
    x, w = (mk.matrix(M, K) * 64).round() / 64, mk.weight(K, N, False)
    v = torch.randint(-1, 2, (M, K), generator=mk.g, device="cuda").to(T)
    dy = mk.matrix(M, N)
    h = 2.0 ** -4
    for act in ("gelu", "gelu_tanh", "silu"):
        say("differences", act)
        pre = dg.linear(x, w, activation=act, save_pre=True)[1]
        dx = dg.linear_backward(dy, x, w, pre=pre, activation=act)[0]
        up = dg.linear(x + h * v, w, activation=act, out_dtype=torch.float32).double()
        down = dg.linear(x - h * v, w, activation=act, out_dtype=torch.float32).double()
        d = ((up - down) * dy.double()).sum() / (2 * h)
        size = float((dy.double().abs() * (v.double().abs() @ w.double().abs()) ** 1).sum())
        assert abs(float((dx.double() * v.double()).sum()) - float(d)) <= (2 * h * h + 2.0 ** -9) * size


# -------------------------------------------------------------- refusals --

def test_refusals():
    T = torch.bfloat16
    x, w = torch.zeros(4, 16, dtype=T, device="cuda"), torch.zeros(16, 8, dtype=T, device="cuda")
    with pytest.raises(ValueError):
        dg.linear(x, w[:8])
    with pytest.raises(TypeError):
        dg.linear(x, w.half())
    with pytest.raises(TypeError):
        dg.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        dg.linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        dg.linear(x, w, bias=torch.zeros(7, dtype=T, device="cuda"))
    with pytest.raises(TypeError):
        dg.linear(x, w, residual=torch.zeros(4, 8, device="cuda"))
    with pytest.raises(TypeError):
        dg.linear(x, w, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        dg.linear(torch.zeros(4, 32, dtype=T, device="cuda")[:, ::2], w)
    with pytest.raises(dg.GemmError):   # a broadcast row: its stride is below its length
        dg.linear(x[:1].expand(4, 16), w)
    with pytest.raises(ValueError):
        dg.linear(x, w, workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        dg.linear_backward(torch.zeros(4, 8, dtype=T, device="cuda"), x, w, activation="gelu")
    with pytest.raises(ValueError):
        dg.gated(x, w, w.t().contiguous().t())
    with pytest.raises(ValueError):
        dg.gated(x, w, w[:, :4])
    with pytest.raises(TypeError):
        dg.layer_norm(x.double())
    with pytest.raises(dg.GemmError):
        dg.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        dg.layer_norm(x, torch.zeros(15, dtype=T, device="cuda"))
    with pytest.raises(ValueError):
        dg.layer_norm_backward(x, x, None, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))
