"""What the 8-bit layers, their quantisation and the orthogonalised update refuse, and the
workspace that they ask for, without a GPU: refusals come before anything touches a device."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from dense_gemm_optimisation_row_amd import binding as b
from dense_gemm_optimisation_row_amd import layers

P = 0x1000   # a non-null, 256-byte aligned address that no such call reads
KINDS = ("f32", "f16", "bf16")


def linear(M=100, N=64, K=128, op=1, ldx=None, ldw=None, ldy=None, ldr=None, act=0, unaligned=0):
    ldx, ldw, ldy, ldr = (max(d, 1) if ld is None else ld
                          for d, ld in ((K, ldx), (K if op else N, ldw), (N, ldy), (N, ldr)))
    return b.LinearI8Params(M, N, K, op, ldx, ldw, ldy, ldr, act, unaligned)


def run(p, kind="bf16", X=P, xs=P, W=P, ws=P, bias=None, R=None, Y=P, work=None, size=0):
    return b.raw_layer("gemm_linear_i8", kind, p, X, xs, W, ws, bias, R, Y, work, size, None)


@pytest.mark.parametrize("kind", KINDS)
def test_linear_refusals(kind):
    for bad in (linear(M=-1), linear(N=-1), linear(K=-1), linear(K=131072), linear(M=1 << 29, N=1 << 10)):
        assert run(bad, kind) == b.GEMM_ERR_INVALID_DIM
    for bad in (linear(op=2), linear(ldx=127), linear(ldw=100), linear(ldy=63)):
        assert run(bad, kind) == b.GEMM_ERR_INVALID_LAYOUT
    assert run(linear(ldr=63), kind, R=P) == b.GEMM_ERR_INVALID_LAYOUT
    assert run(linear(act=5), kind) == run(linear(act=-1), kind) == b.GEMM_ERR_INVALID_ACTIVATION
    for name in ("X", "xs", "W", "ws", "Y"):
        assert run(linear(), kind, **{name: None}) == b.GEMM_ERR_NULL_PTR
    # off 16 bytes without saying so
    assert run(linear(), kind, X=P + 8) == run(linear(), kind, W=P + 1) == b.GEMM_ERR_INVALID_LAYOUT
    # copies need their workspace
    for p in (linear(K=100), linear(op=0), linear(unaligned=1), linear(ldx=136)):
        need = b.layer_workspace("gemm_linear_i8", p)
        assert need > 0 and need % 256 == 0
        assert run(p, kind) == run(p, kind, work=P, size=need - 1) == run(p, kind, work=P + 16, size=need) \
            == b.GEMM_ERR_WORKSPACE
    assert run(linear(M=0), kind, X=None, xs=None, Y=None) == b.GEMM_OK
    assert run(linear(N=0), kind, W=None, ws=None, Y=None) == b.GEMM_OK


@pytest.mark.parametrize("kind", KINDS)
def test_gated_refusals(kind):
    def call(p, **changed):
        args = dict(X=P, xs=P, G=P, gs=P, U=P, us=P, H=P)
        args.update(changed)
        return b.raw_layer("gemm_gated_i8", kind, p, *args.values(), None, 0, None)

    def params(M=100, F=64, K=128, op=1, ldx=128, ldw=128, ldh=64, act=4, unaligned=0):
        return b.GatedI8Params(M, F, K, op, ldx, ldw, ldh, act, unaligned)
    for bad in (params(M=-1), params(F=-2), params(K=131072, ldx=131072, ldw=131072)):
        assert call(bad) == b.GEMM_ERR_INVALID_DIM
    for bad in (params(op=3), params(ldx=1), params(ldw=64), params(ldh=1)):
        assert call(bad) == b.GEMM_ERR_INVALID_LAYOUT
    assert call(params(act=9)) == b.GEMM_ERR_INVALID_ACTIVATION
    for name in ("X", "xs", "G", "gs", "U", "us", "H"):
        assert call(params(), **{name: None}) == b.GEMM_ERR_NULL_PTR
    assert call(params(), U=P + 4) == b.GEMM_ERR_INVALID_LAYOUT
    assert call(params(unaligned=1)) == b.GEMM_ERR_WORKSPACE
    assert call(params(M=0), X=None) == b.GEMM_OK


@pytest.mark.parametrize("kind", KINDS)
def test_quantize_refusals(kind):
    def call(M, K, ldx, ldq, x=P, q=P, s=P):
        return b.raw_layer("gemm_quantize_i8", kind, b.QuantizeParams(M, K, ldx, ldq), x, q, s, None)
    assert call(-1, 4, 4, 4) == call(4, -1, 4, 4) == call(1, 2 ** 31 - 65536, 2 ** 31 - 1, 2 ** 31 - 1) \
        == b.GEMM_ERR_INVALID_DIM
    assert call(4, 4, 3, 4) == call(4, 4, 4, 3) == call(4, 0, 0, 1) == b.GEMM_ERR_INVALID_LAYOUT
    assert call(4, 4, 4, 4, x=None) == call(4, 4, 4, 4, q=None) == call(4, 0, 1, 1, s=None) == b.GEMM_ERR_NULL_PTR
    assert call(0, 4, 4, 4, None, None, None) == b.GEMM_OK


def ortho(batch=1, M=64, N=96, op_g=0, op_o=0, ldg=None, ldo=None, steps=5, eps=1e-7, scale=1.0,
          coefficients=(3.4445, -4.775, 2.0315)):
    p = b.OrthogonalizeParams(batch, M, N, op_g, op_o, (M if op_g else N) if ldg is None else ldg,
                              (M if op_o else N) if ldo is None else ldo, steps, M * N, M * N, eps, scale)
    values = list(coefficients) * b.GEMM_MAX_STEPS
    p.coefficients[:] = values[:3 * b.GEMM_MAX_STEPS]
    return p


@pytest.mark.parametrize("kind", KINDS)
def test_orthogonalize_refusals(kind):
    def call(p, g=P, o=P, work=None, size=0):
        return b.raw_layer("gemm_orthogonalize", kind, p, g, o, work, size, None)
    for bad in (ortho(batch=-1), ortho(M=-1), ortho(N=-1), ortho(N=1 << 22), ortho(steps=0), ortho(steps=33),
                ortho(eps=-1.0), ortho(eps=float("nan")), ortho(batch=1 << 30, M=1, N=1)):
        assert call(bad) == b.GEMM_ERR_INVALID_DIM
    for bad in (ortho(op_g=2), ortho(op_o=-1), ortho(ldg=95), ortho(op_o=1, ldo=63)):
        assert call(bad) == b.GEMM_ERR_INVALID_LAYOUT
    nan, inf = float("nan"), float("inf")
    # not finite; a singular value of 1 becomes 300; one below 1 grows past 256 within the steps
    for c in ((nan, 0, 0), (1, inf, 0), (300, 0, 0), (4, 0, 0), (0, 0, 300), (1e308, 1e308, 1e308)):
        assert call(ortho(coefficients=c)) == b.GEMM_ERR_INVALID_COEFFICIENTS
    large = ortho(M=300, N=200)
    need = b.layer_workspace("gemm_orthogonalize", large)
    assert call(ortho(), None) == call(large, P, None) == b.GEMM_ERR_NULL_PTR
    assert call(large) == call(large, work=P, size=need - 1) == call(large, work=P + 128, size=need) \
        == b.GEMM_ERR_WORKSPACE
    assert call(ortho(batch=0), None, None) == call(ortho(M=0), None, None) == b.GEMM_OK
    for c in ((1.5, -0.5, 0), (2, -1.5, 0.5), (1.875, -1.25, 0.375), (1, 0, 0), (0, 0, 0)):
        assert b.layer_workspace("gemm_orthogonalize", ortho(M=300, N=200, coefficients=c)) > 0
    # what LDS holds needs none
    assert b.layer_workspace("gemm_orthogonalize", ortho()) == 0


def test_workspaces_do_not_overflow():
    p = ortho(batch=4, M=40000, N=60000)
    assert b.layer_workspace("gemm_orthogonalize", p) > 4 * 4 * (2 * 40000 * 60000 + 2 * 40000 * 40000)
    p = linear(M=1 << 20, N=1 << 13, K=30001, op=0)
    assert b.layer_workspace("gemm_linear_i8", p) > (1 << 20) * 30001


def test_tensors_on_the_cpu_are_refused():
    x, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    for call in (lambda: dg.quantize_i8(torch.zeros(4, 16)), lambda: dg.linear_i8(x, s, x.t(), s),
                 lambda: dg.gated_i8(x, s, x.t(), s, x.t(), s), lambda: dg.orthogonalize(torch.zeros(4, 4))):
        with pytest.raises(ValueError):
            call()


def test_tensors_that_require_grad_are_refused():
    x = torch.zeros(4, 16, requires_grad=True)
    for call in (lambda: dg.quantize_i8(x), lambda: dg.orthogonalize(x)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
    codes, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        dg.linear_i8(codes, s, codes.t(), s)
    with pytest.raises(ValueError, match="requires grad"):
        dg.gated_i8(codes, s, codes.t(), s, codes.t(), s)


def test_coefficients_of_the_wrong_number_are_refused():
    assert layers._step_coefficients((1, 2, 3), 2) == (1.0, 2.0, 3.0, 1.0, 2.0, 3.0)
    assert layers._step_coefficients([(1, 2, 3), (4, 5, 6)], 2) == (1.0, 2.0, 3.0, 4.0, 5.0, 6.0)
    for bad in ((1, 2), [(1, 2, 3)], [(1, 2), (3, 4)], ()):
        with pytest.raises(ValueError):
            layers._step_coefficients(bad, 2)


def test_storage_of_stacks():
    t = torch.empty(2, 3, 5, 7)
    assert layers._matrices(t, "g") == (6, b.GEMM_OP_N, 7, 35)
    assert layers._matrices(t.mT, "g") == (6, b.GEMM_OP_T, 7, 35)
    assert layers._matrices(t[:, :, 1:4, 2:5], "g") == (6, b.GEMM_OP_N, 7, 35)
    assert layers._matrices(t[0, 0], "g") == (1, b.GEMM_OP_N, 7, 0)
    assert layers._matrices(torch.empty(1, 9), "g")[:3] == (1, b.GEMM_OP_N, 9)
    for bad in (t.transpose(0, 1), t[:, :2], t[..., ::2], torch.empty(7).expand(5, 7)):
        with pytest.raises(ValueError):
            layers._matrices(bad, "g")
