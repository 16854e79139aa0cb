"""Sizes and strides that a C int does not hold are refused before anything is
allocated or launched; ctypes alone would cut them off.  The tensors are
stand-ins without storage that say they are on the GPU."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import binding, layers

LONG = 2 ** 32 + 4
B16 = torch.bfloat16


class OnGpu:
    """A tensor's shape, strides and type, with a GPU's name for a device."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype=B16, of=None):
        self.t = torch.empty(shape, dtype=dtype, device="meta") if of is None else of

    def __getattr__(self, name):
        return getattr(self.t, name)

    def view(self, *shape):
        return OnGpu(of=self.t.view(*shape))

    def new_empty(self, *args, **kw):
        raise AssertionError("allocated")


def vector(n, dtype=torch.float32):
    return OnGpu(n, dtype=dtype)


CALLS = {
    "linear rows": lambda: dg.linear(OnGpu(LONG, 2), OnGpu(2, 8)),
    "linear folded rows": lambda: dg.linear(OnGpu(2 ** 17, 2 ** 15, 2), OnGpu(2, 8)),
    "linear outputs": lambda: dg.linear(OnGpu(4, 2), OnGpu(2, LONG)),
    "linear inputs": lambda: dg.linear(OnGpu(4, LONG), OnGpu(LONG, 2)),
    "linear backward rows": lambda: dg.linear_backward(OnGpu(LONG, 8), OnGpu(LONG, 2), OnGpu(2, 8)),
    "gated rows": lambda: dg.gated(OnGpu(LONG, 2), OnGpu(2, 8), OnGpu(2, 8)),
    "gated outputs": lambda: dg.gated(OnGpu(4, 2), OnGpu(2, LONG), OnGpu(2, LONG)),
    "gated backward rows": lambda: dg.gated_backward(OnGpu(LONG, 8), OnGpu(LONG, 2), OnGpu(2, 8), OnGpu(2, 8),
                                                     OnGpu(LONG, 8), OnGpu(LONG, 8)),
    "layer norm rows": lambda: dg.layer_norm(OnGpu(LONG, 2)),
    "layer norm columns": lambda: dg.layer_norm(OnGpu(2, LONG)),
    "layer norm backward rows": lambda: dg.layer_norm_backward(OnGpu(LONG, 2), OnGpu(LONG, 2), None, vector(LONG),
                                                               vector(LONG)),
    "product rows": lambda: dg.gemm_bf16_f32acc(OnGpu(LONG, 2), OnGpu(2, 8)),
    "product sum": lambda: dg.gemm_bf16_f32acc(OnGpu(4, LONG), OnGpu(LONG, 8)),
    "product of views, rows": lambda: dg.gemm_bf16_f32acc_ex(OnGpu(LONG, 2), OnGpu(2, 8)),
    "product of views, columns": lambda: dg.gemm_bf16_f32acc_ex(OnGpu(4, 2), OnGpu(2, LONG)),
    "raw product": lambda: binding.raw_gemm("f32", None, LONG, 2, 2, 1, 1, 1, None),
    "raw product of views": lambda: binding.raw_gemm_ex("f32", 0, 0, 2, 2, 2, 1.0, 1, LONG, 1, 2, 0.0, 1, 2, None),
    "plan": lambda: binding.plan("f32", LONG, 2, 2),
    "convolution": lambda: binding.conv_params(LONG, 2, 6, 6, 3, 3, 3),
}


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def refuse(*a, **k):
        raise AssertionError("allocated or launched")
    monkeypatch.setattr(layers, "_run", refuse)
    monkeypatch.setattr(torch, "empty", lambda *a, real=torch.empty, **k: real(*a, **k)
                        if k.get("device") == "meta" else refuse())


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_an_int_are_refused(name):
    with pytest.raises(ValueError, match="2\\^31|out of range"):
        CALLS[name]()


def test_the_largest_sizes_of_an_int_still_have_parameters():
    p = binding.LayerNormParams(2 ** 31 - 1, 2, 2, 2, 2, 0, 1e-5)
    assert p.M == 2 ** 31 - 1


@pytest.mark.parametrize("stem", ["gemm_layer_norm", "gemm_layer_norm_backward"])
def test_layer_norm_rows_that_overflow_a_column_are_refused(stem):
    """The long rows' kernels step 2048 columns past a row's end; the sizes
    that stay an int are taken (an empty batch launches nothing)."""
    address, most = 0x1000, 2 ** 31 - 4096

    def call(M, N):
        params = binding.LayerNormParams(M, N, N, N, N, 0, 1e-5)
        pointers = [address] * 6 + [None] if stem == "gemm_layer_norm" else \
            [address] * 6 + [None, None, address, 2 ** 40, None]
        return binding.raw_layer(stem, "bf16", params, *pointers)
    for N in (most + 1, 2 ** 31 - 2048, 2 ** 31 - 1):
        assert call(1, N) == binding.GEMM_ERR_INVALID_DIM
    assert call(0, most) == 0
