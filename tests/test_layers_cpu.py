"""CPU-side checks of the layer entry points: argument refusals happen before
anything touches a device, and the formulas the GPU tests compare against
agree with differences.  No kernel is launched here."""
import ctypes

import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import binding as b
from layer_reference import act_slope, act_value, gated_grads, layer_norm_grads, linear_grads

P = 0x1000   # a non-null, 256-byte aligned address that no refused call reads


def linear_params(**kw):
    d = dict(M=4, N=8, K=16, op_w=0, ldx=16, ldw=8, ldy=8, ldr=8, ldp=8, activation=1, y_f32=0)
    d.update(kw)
    return b.LinearParams(*[d[n] for n, _ in b.LinearParams._fields_])


def linear_backward_params(**kw):
    d = dict(M=4, N=8, K=16, op_w=0, lddy=8, ldx=16, ldw=8, ldp=8, lddx=16, lddw=8, activation=1)
    d.update(kw)
    return b.LinearBackwardParams(*[d[n] for n, _ in b.LinearBackwardParams._fields_])


def gated_params(**kw):
    d = dict(M=4, F=8, K=16, op_w=0, ldx=16, ldw=8, ldh=8, ldp=8, activation=4)
    d.update(kw)
    return b.GatedParams(*[d[n] for n, _ in b.GatedParams._fields_])


def gated_backward_params(**kw):
    d = dict(M=4, F=8, K=16, op_w=0, lddh=8, ldx=16, ldw=8, ldp=8, lddx=16, lddw=8, activation=4)
    d.update(kw)
    return b.GatedBackwardParams(*[d[n] for n, _ in b.GatedBackwardParams._fields_])


def norm_params(**kw):
    d = dict(M=4, N=8, ldx=8, ldy=8, lddx=8, weight_f32=0, eps=1e-5)
    d.update(kw)
    return b.LayerNormParams(*[d[n] for n, _ in b.LayerNormParams._fields_])


CALLS = {   # parameters, pointers (workspace and stream apart)
    "gemm_linear": (linear_params, [P] * 6),
    "gemm_linear_backward": (linear_backward_params, [P] * 7),
    "gemm_gated": (gated_params, [P] * 6),
    "gemm_gated_backward": (gated_backward_params, [P] * 9),
    "gemm_layer_norm": (norm_params, [P] * 6),
    "gemm_layer_norm_backward": (norm_params, [P] * 8),
}


def call(stem, params, pointers, kind="bf16", ws=P, ws_bytes=1 << 30):
    args = list(pointers) + ([] if stem == "gemm_layer_norm" else [ws, ws_bytes]) + [None]
    if params is None:
        return int(getattr(b.load(), f"{stem}_{kind}")(None, *args))
    return b.raw_layer(stem, kind, params, *args)


@pytest.mark.parametrize("stem", CALLS)
def test_null_parameters_and_negative_sizes_are_refused(stem):
    make, pointers = CALLS[stem]
    assert call(stem, None, pointers) == b.GEMM_ERR_NULL_PTR
    for name in ("M", "N", "F", "K"):
        if any(name == n for n, _ in type(make())._fields_):
            assert call(stem, make(**{name: -1}), pointers) == b.GEMM_ERR_INVALID_DIM
    if stem.startswith("gemm_layer_norm"):
        return
    assert call(stem, make(M=2 ** 30, N=2 ** 30) if "linear" in stem else make(M=2 ** 30, F=2 ** 30),
                pointers) == b.GEMM_ERR_INVALID_DIM
    for bad in (-1, 2):
        assert call(stem, make(op_w=bad), pointers) == b.GEMM_ERR_INVALID_LAYOUT
    for bad in (-1, 5):
        assert call(stem, make(activation=bad), pointers) == b.GEMM_ERR_INVALID_ACTIVATION


@pytest.mark.parametrize("stem,name,least", [
    ("gemm_linear", "ldx", 16), ("gemm_linear", "ldw", 8), ("gemm_linear", "ldy", 8), ("gemm_linear", "ldr", 8),
    ("gemm_linear", "ldp", 8), ("gemm_linear_backward", "lddy", 8), ("gemm_linear_backward", "ldx", 16),
    ("gemm_linear_backward", "ldw", 8), ("gemm_linear_backward", "ldp", 8), ("gemm_linear_backward", "lddx", 16),
    ("gemm_linear_backward", "lddw", 8), ("gemm_gated", "ldx", 16), ("gemm_gated", "ldw", 8), ("gemm_gated", "ldh", 8),
    ("gemm_gated", "ldp", 8), ("gemm_gated_backward", "lddh", 8), ("gemm_gated_backward", "ldx", 16),
    ("gemm_gated_backward", "ldw", 8), ("gemm_gated_backward", "ldp", 8), ("gemm_gated_backward", "lddx", 16),
    ("gemm_gated_backward", "lddw", 8), ("gemm_layer_norm", "ldx", 8), ("gemm_layer_norm", "ldy", 8),
    ("gemm_layer_norm_backward", "ldx", 8), ("gemm_layer_norm_backward", "ldy", 8),
    ("gemm_layer_norm_backward", "lddx", 8)])
def test_strides_below_the_row_are_refused(stem, name, least):
    make, pointers = CALLS[stem]
    assert call(stem, make(**{name: least - 1}), pointers) == b.GEMM_ERR_INVALID_LAYOUT
    if name in ("ldw", "lddw"):   # the transposed storage's rows hold K
        assert call(stem, make(op_w=1, **{name: 15}), pointers) == b.GEMM_ERR_INVALID_LAYOUT


@pytest.mark.parametrize("stem,required", [
    ("gemm_linear", (0, 1, 4)), ("gemm_linear_backward", (0, 1, 2, 3)), ("gemm_gated", (0, 1, 2, 3, 4, 5)),
    ("gemm_gated_backward", (0, 1, 2, 3, 4, 5, 7, 8)), ("gemm_layer_norm", (0, 3)),
    ("gemm_layer_norm_backward", (0, 1, 3, 4, 5))])
def test_missing_operands_are_refused(stem, required):
    make, pointers = CALLS[stem]
    for i in required:
        p = list(pointers)
        p[i] = None
        assert call(stem, make(ldw=16, lddw=16) if "linear_b" in stem or "gated_b" in stem else make(), p) \
            == b.GEMM_ERR_NULL_PTR, i


@pytest.mark.parametrize("stem", ["gemm_linear", "gemm_linear_backward", "gemm_gated", "gemm_gated_backward",
                                  "gemm_layer_norm_backward"])
def test_workspace_is_checked(stem):
    make, pointers = CALLS[stem]
    # few outputs and a long sum: the forward products are split over k (those
    # of few rows are not, and need none)
    long = dict(M=100, K=4096, ldx=4096, lddx=4096) if "norm" not in stem else dict(M=100)
    if "backward" not in stem and "norm" not in stem:
        long["ldw"] = 8
    names = {n for n, _ in type(make())._fields_}
    params = make(**{k: v for k, v in long.items() if k in names})
    need = b.layer_workspace(stem, params)
    assert need > 0
    for ws, size in ((None, need), (P, need - 1), (P + 64, need)):
        assert call(stem, params, pointers, ws=ws, ws_bytes=size) == b.GEMM_ERR_WORKSPACE
    out = ctypes.c_size_t()
    f = getattr(b.load(), stem + "_workspace")
    assert f(ctypes.byref(params), None) == b.GEMM_ERR_NULL_PTR
    assert f(None, ctypes.byref(out)) == b.GEMM_ERR_NULL_PTR
    with pytest.raises(dg.GemmError):
        b.layer_workspace(stem, make(M=-1))


def test_layer_norm_refuses_a_bad_eps():
    for eps in (-1.0, float("nan")):
        assert call("gemm_layer_norm", norm_params(eps=eps), [P] * 6) == b.GEMM_ERR_INVALID_DIM


def test_empty_calls_launch_nothing():
    """These return GEMM_OK with no GPU present."""
    full = [P] * 9
    assert call("gemm_linear", linear_params(M=0), full[:6]) == 0
    assert call("gemm_linear", linear_params(N=0), full[:6]) == 0
    assert call("gemm_gated", gated_params(M=0), full[:6]) == 0
    assert call("gemm_gated", gated_params(F=0), full[:6]) == 0
    assert call("gemm_layer_norm", norm_params(M=0), full[:6]) == 0
    assert call("gemm_layer_norm_backward", norm_params(N=0), full[:8]) == 0


def test_status_of_an_unknown_activation_has_a_name():
    assert "activation" in dg.status_string(b.GEMM_ERR_INVALID_ACTIVATION)


def test_host_tensors_are_refused():
    x, w = torch.zeros(2, 4, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dg.linear(x, w)
    with pytest.raises(ValueError):
        dg.gated(x, w, w)
    with pytest.raises(ValueError):
        dg.layer_norm(x)


# ------------------------------------- the reference against differences --

def _close_to_differences(f, x, grad, dy):
    """<grad, v> = d/dt <dy, f(x + t v)> by central differences, in 64 bits: at
    step 1e-5 the differences err by the third derivative (below 10 in these
    functions) times 1e-10 and by rounding, 2^-52 / 1e-5, both relative to the
    sum's terms."""
    torch.manual_seed(5)
    v = torch.randn_like(x)
    h = 1e-5
    terms = dy.abs().sum() * 4
    d = ((f(x + h * v) * dy).sum() - (f(x - h * v) * dy).sum()) / (2 * h)
    assert abs((grad * v).sum() - d) <= 1e-8 * terms


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
def test_reference_gradients_match_differences(act):
    torch.manual_seed(1)
    x, w, w2 = (torch.randn(s, dtype=torch.float64) for s in ((5, 7), (7, 6), (7, 6)))
    bias = torch.randn(6, dtype=torch.float64)
    dy = torch.randn(5, 6, dtype=torch.float64)
    z = x @ w + bias
    dx, dw, db = linear_grads(act, dy, x, w, z)
    _close_to_differences(lambda t: act_value(act, t @ w + bias), x, dx, dy)
    _close_to_differences(lambda t: act_value(act, x @ t + bias), w, dw, dy)
    _close_to_differences(lambda t: act_value(act, x @ w + t), bias, db, dy)
    dx, dg_, du = gated_grads(act, dy, x, w, w2, x @ w, x @ w2)
    _close_to_differences(lambda t: act_value(act, t @ w) * (t @ w2), x, dx, dy)
    _close_to_differences(lambda t: act_value(act, x @ t) * (x @ w2), w, dg_, dy)
    _close_to_differences(lambda t: act_value(act, x @ w) * (x @ t), w2, du, dy)
    _close_to_differences(lambda t: act_value(act, t), z, act_slope(act, z) * dy, dy)


def test_reference_layer_norm_gradients_match_differences():
    torch.manual_seed(2)
    x, dy = torch.randn(4, 9, dtype=torch.float64), torch.randn(4, 9, dtype=torch.float64)
    w, bias = torch.randn(9, dtype=torch.float64), torch.randn(9, dtype=torch.float64)

    def norm(x, w, bias):
        return torch.nn.functional.layer_norm(x, (9,), w, bias, 1e-5)
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + 1e-5)
    dx, dw, db = layer_norm_grads(dy, x, w, mean, rstd)
    _close_to_differences(lambda t: norm(t, w, bias), x, dx, dy)
    _close_to_differences(lambda t: norm(x, t, bias), w, dw, dy)
    _close_to_differences(lambda t: norm(x, w, t), bias, db, dy)


def test_a_gradient_is_kept_as_its_weight_is_also_with_one_row():
    from dense_gemm_optimisation_row_amd.layers import _grad_stride
    t = torch.zeros
    assert _grad_stride(t(4, 6), b.GEMM_OP_N, None, "dw") == 6
    assert _grad_stride(t(6, 4).t(), b.GEMM_OP_T, None, "dw") == 4
    assert _grad_stride(t(4, 6), b.GEMM_OP_N, t(4, 9)[:, :6], "dw") == 9
    # a single row, kept N x K with a stride of 3: only such a gradient will do
    w = t(6, 3)[:, :1].t()
    assert w.shape == (1, 6)
    assert _grad_stride(w, b.GEMM_OP_T, t(6, 5)[:, :1].t(), "dw") == 5
    assert _grad_stride(w, b.GEMM_OP_T, t(1, 6), "dw") == 1
    for op, given in ((b.GEMM_OP_N, t(6, 5)[:, :1].t()), (b.GEMM_OP_N, t(6, 4).t()), (b.GEMM_OP_T, t(4, 6))):
        with pytest.raises(ValueError):
            _grad_stride(t(*given.shape), op, given, "dw")
