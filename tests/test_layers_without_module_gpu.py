"""The 8-bit layers without the extension module: the same results, through Python."""
import warnings

import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import layers
from test_i8_gpu import gen, need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def test_results_are_the_same(monkeypatch):
    g = gen(6)
    x = torch.randn(5, 96, generator=g, device="cuda")
    w, u = (torch.randn(40, 96, generator=g, device="cuda") for _ in range(2))
    r = torch.randn(5, 40, generator=g, device="cuda").to(torch.bfloat16)

    def step():
        (q, s), (a, sa), (b, sb) = (dg.quantize_i8(t) for t in (x, w, u))
        return q, s, dg.linear_i8(q, s, a.t(), sa, residual=r), dg.gated_i8(q, s, a.t(), sa, b.t(), sb)
    first = step()
    assert layers._marshal      # the module is built and in use
    known = step()
    monkeypatch.setattr(layers, "_marshal", False)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for out in (known, step(), step()):
            assert all(torch.equal(p, q) for p, q in zip(first, out))
