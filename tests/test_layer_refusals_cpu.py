"""What the layers' C entry points refuse and what they leave unread, without a
GPU: refusals come before anything touches a device."""
import pytest

from dense_gemm_optimisation_row_amd import binding as b

P = 0x1000   # a non-null, 256-byte aligned address that no such call reads


@pytest.mark.parametrize("eps", [float("nan"), -1.0, float("-inf")])
def test_the_backward_pass_of_layer_norm_does_not_read_eps(eps):
    p = b.LayerNormParams(0, 8, 8, 8, 8, 0, eps)
    assert b.raw_layer("gemm_layer_norm_backward", "bf16", p, *[P] * 6, None, None, P, 0, None) == b.GEMM_OK
    p = b.LayerNormParams(100, 8, 8, 8, 8, 0, eps)
    assert b.layer_workspace("gemm_layer_norm_backward", p) > 0
    # missing rows are still refused, and the forward pass refuses the eps
    assert b.raw_layer("gemm_layer_norm_backward", "bf16", p, None, *[P] * 5, None, None, P, 0, None) \
        == b.GEMM_ERR_NULL_PTR
    assert b.raw_layer("gemm_layer_norm", "bf16", p, *[P] * 6, None) == b.GEMM_ERR_INVALID_DIM
