"""Race check of the 8-bit rings and of the orthogonalised update's products
through the LDS-poisoning build of the library, as for the other kernels that load
straight into LDS: a read ahead of its load or behind a refill returns all-ones
(-1, a NaN), so exact inputs have to give the exact result, at one to several
stages of every tile, full and ragged."""
import ctypes

import pytest
import torch

from dense_gemm_optimisation_row_amd import binding as b
from dense_gemm_optimisation_row_amd import build
from helpers import say
from test_i8_gpu import codes, gen, powers, product
from test_orthogonalize_gpu import exact, signs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")
    return b.load(build.POISON_LIB)


def space(lib, stem, params):
    need = ctypes.c_size_t()
    assert getattr(lib, stem + "_workspace")(ctypes.byref(params), ctypes.byref(need)) == b.GEMM_OK
    return torch.empty(max(need.value, 256), dtype=torch.uint8, device="cuda"), need.value


# rows and outputs that take each tile, with one to nine stages of 64 k and split sums
I8 = [(70, 70, (16, 64, 128, 144, 576)), (1000, 2100, (64, 1040)), (2056, 2176, (80, 208, 336)),
      (4090, 4090, (64, 528)), (100, 64, (16000,)), (5, 300, (16, 4096))]


@pytest.mark.parametrize("M,N,Ks", I8, ids=lambda v: str(v))
def test_8_bit_products(lib, M, N, Ks):
    for K in Ks:
        say("poison i8", M, N, K)
        g = gen(M + K)
        x, w, u = codes(g, M, K), codes(g, N, K), codes(g, N, K)
        sx, sw, su = powers(g, M), powers(g, N), powers(g, N)
        z, v = (product(x, a.t()) * sx.double()[:, None] * s.double() for a, s in ((w, sw), (u, su)))
        y = torch.full((M, N), 7.0, device="cuda")
        p = b.LinearI8Params(M, N, K, 1, K, K, N, N, 0, 0)
        ws, size = space(lib, "gemm_linear_i8", p)
        rc = lib.gemm_linear_i8_f32(ctypes.byref(p), x.data_ptr(), sx.data_ptr(), w.data_ptr(), sw.data_ptr(), None,
                                    None, y.data_ptr(), ws.data_ptr(), size, None)
        assert rc == b.GEMM_OK and torch.equal(y, z.float())
        p = b.GatedI8Params(M, N, K, 1, K, K, N, 0, 0)
        ws, size = space(lib, "gemm_gated_i8", p)
        rc = lib.gemm_gated_i8_f32(ctypes.byref(p), x.data_ptr(), sx.data_ptr(), w.data_ptr(), sw.data_ptr(),
                                   u.data_ptr(), su.data_ptr(), y.data_ptr(), ws.data_ptr(), size, None)
        assert rc == b.GEMM_OK and torch.equal(y, (z * v).float())


@pytest.mark.parametrize("M,N,k", [(129, 130, 4), (40, 3000, 4), (128, 4100, 4), (777, 1033, 5), (1024, 2500, 5),
                                   (2049, 1500, 5), (3000, 3000, 5), (4100, 4096, 5)])
def test_one_step_of_signs(lib, M, N, k):
    for c in ((2.0, -1.0, 3.0), (0.0, 3.0, 1.0)):
        say("poison orthogonalize", M, N, c)
        g = signs(M, N, k, M + N)[0]
        o = torch.full((M, N), 7.0, device="cuda")
        p = b.OrthogonalizeParams(1, M, N, 0, 0, N, N, 1, 0, 0, 0.0, 1.0)
        p.coefficients[:3] = c
        ws, size = space(lib, "gemm_orthogonalize", p)
        rc = lib.gemm_orthogonalize_f32(ctypes.byref(p), g.data_ptr(), o.data_ptr(), ws.data_ptr(), size, None)
        assert rc == b.GEMM_OK and torch.equal(o, exact(g, [c], 0.0).float())
