"""The orthogonalised update against its definition in 64 bits.

Exact: a matrix of 4^k entries of +-1 and zeros elsewhere has the norm 2^k, so with
eps 0 and small whole coefficients one step is integers over 2^(5 k), which fit the
two terms and FP32 throughout: the result has to be equal, at every size, edge and
storage.

Otherwise the error's 2-norm is held to what the steps' roundings come to.  With f(s) =
a s + b s^3 + c s^5 on the singular values, a step passes an error on by at most L,
the largest of |f'| and |f / s| over them, and adds
  the two terms of its operands: 2^-23 of X, and of A through |b| + 2 |c| |A|,
  of P through P X, each twice (both factors of a product), and lo lo, 2^-24;
  the sums in FP32: rounding errors of both signs in a sum of K products add up to
  6 sqrt(K) 2^-24 of the sum of their magnitudes but with a probability of 2
  exp(-18), and the magnitudes' sum is at most |.|_F of the factors' 2-norms by row
  and column;
and the result is rounded once to its type."""
import pytest
import torch

import dense_gemm_optimisation_row_amd as dg
from helpers import say

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(autouse=True, scope="module")
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU (run the CPU suite with -m 'not gpu')")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def exact(g, coefficients, eps=1e-7, scale=1.0):
    """The definition in 64 bits, a step for each triple, of a matrix or a stack."""
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for a, b, c in coefficients:
        gram = x @ x.mT
        x = a * x + (b * gram + c * gram @ gram) @ x
    return scale * (x.mT if tall else x)


def error_bound(g, coefficients, eps=1e-7):
    """Bound of the error's 2-norm before the result is rounded, of one matrix."""
    u = 2.0 ** -24
    x = g.double()
    x = x.mT if x.shape[0] > x.shape[1] else x
    x = x / (x.norm() + eps)
    err = 2 * u                      # the factor and its product
    for a, b, c in coefficients:
        m, n = x.shape
        s = torch.linalg.svdvals(x)
        top, fro = float(s[0]) + err, float(x.norm()) + err
        t = torch.linspace(0, top, 2001, dtype=torch.float64, device=x.device)
        grows = float((a + 3 * b * t ** 2 + 5 * c * t ** 4).abs().max())
        grows = max(grows, float((a + b * t ** 2 + c * t ** 4).abs().max()))
        # of A: two operands in two terms, lo lo, the sums; then A's own two terms
        rows = float(x.square().sum(1).sum())                 # |.|_F of the outer product of the rows' norms
        d_gram = (4 * u + u) * rows + 6 * n ** 0.5 * u * rows + 2 * u * rows
        gram = x @ x.mT
        fro_a, top_a = float(gram.norm()), top * top
        square = float(gram.square().sum())                   # as `rows`, of A A
        d_poly = (abs(b) + 2 * abs(c) * top_a) * d_gram
        d_poly += abs(c) * (5 * u + 6 * m ** 0.5 * u) * square + 3 * u * (abs(b) * fro_a + abs(c) * square)
        poly = b * gram + c * gram @ gram
        poly.diagonal().add_(a)
        d_poly += 3 * u * float(poly.norm())                  # the diagonal's sum, and P's two terms
        spread = float(poly.norm(dim=1).norm() * x.norm(dim=0).norm())   # magnitudes of P X, by its norms
        step = d_poly * top + (2 * u + u) * grows * fro + 6 * m ** 0.5 * u * spread / 1 + 2 * u * grows * fro
        err = grows * err + step + 2.0 ** -37 * (m * n) ** 0.5
        x = poly @ x
    return err


def matrix(M, N, seed, dtype, kind="spread"):
    g = gen(seed)
    if kind == "normal":
        x = torch.randn(M, N, generator=g, device="cuda")
    else:   # directions that fall off, and little noise under them
        r = min(M, N)
        fall = torch.arange(1, r + 1, device="cuda") ** -1.0
        x = (torch.randn(M, r, generator=g, device="cuda") * fall) @ torch.randn(r, N, generator=g, device="cuda")
        x = x + 0.01 * torch.randn(M, N, generator=g, device="cuda")
    return (0.01 * x).to(dtype)


def near(got, g, coefficients, what, eps=1e-7, scale=1.0):
    ref = exact(g, coefficients, eps, scale)
    err = abs(scale) * error_bound(g, coefficients, eps)
    tol = err + STEP[got.dtype] * (float(ref.norm()) + err) + 2.0 ** -25 * ref.numel() ** 0.5 * (got.dtype == torch.float16)
    off = float((got.double() - ref).norm())
    assert got.shape == g.shape and got.dtype == g.dtype
    assert off <= tol, f"{what}: {off / tol:.3g} of the bound ({off:.3g}, of {float(ref.norm()):.3g})"


def signs(M, N, k, seed, batch=1):
    """4^k entries of +-1 in each of a stack of zeros."""
    out = torch.zeros(batch, M * N, device="cuda")
    for i in range(batch):
        at = torch.randperm(M * N, generator=gen(seed + i), device="cuda")[:4 ** k]
        out[i, at] = torch.randint(0, 2, (4 ** k,), generator=gen(seed + 50 + i), device="cuda").float() * 2 - 1
    return out.view(batch, M, N)


EXACT = [(1, 1, 0), (1, 5, 1), (4, 1, 1), (8, 8, 2), (16, 33, 3), (33, 16, 3), (64, 64, 3), (65, 64, 4), (72, 200, 4),
         (128, 256, 4), (129, 130, 4), (257, 100, 4), (300, 77, 4), (256, 512, 4), (520, 264, 5), (777, 1033, 5),
         (1033, 777, 5), (64, 4096, 4), (2000, 40, 4), (1024, 1024, 5), (2049, 1500, 5), (128, 4100, 4), (96, 96, 3), (40, 300, 4),
         (3000, 3000, 5), (2200, 4400, 5), (4400, 2300, 5), (4100, 4096, 5), (4070, 4200, 5)]


@pytest.mark.parametrize("stored", ["rows", "columns"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", EXACT, ids=lambda s: "x".join(map(str, s[:2])))
def test_one_step_of_signs(size, dtype, stored):
    M, N, k = size
    for batch in (1, 3):
        say("orthogonalize", size, dtype, stored, batch)
        x = signs(M, N, k, M + 2 * N, batch).to(DTYPES[dtype])
        g = x.mT.contiguous().mT if stored == "columns" else x
        for c in ((2.0, -1.0, 3.0), (0.0, 3.0, 1.0), (1.0, 0.0, 0.0), (1.0, 0.0, 2.0)):
            got = dg.orthogonalize(g, steps=1, coefficients=c, eps=0.0, scale=2.0)
            want = exact(x, [c], 0.0, 2.0).to(got.dtype)
            assert got.stride() == g.stride() or min(M, N) == 1
            assert torch.equal(got, want), f"{c}: {int((got != want).sum())} of {got.numel()} differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["normal", "spread"])
@pytest.mark.parametrize("size", [(1, 1), (1, 300), (7, 5), (16, 16), (64, 64), (100, 131), (128, 128), (260, 72),
                                  (192, 2048), (512, 512), (777, 1033), (1500, 400)],
                         ids=lambda s: "x".join(map(str, s)))
def test_steps(size, kind, dtype):
    M, N = size
    g = matrix(M, N, M + N, DTYPES[dtype], kind)
    say("orthogonalize", size, kind, dtype)
    near(dg.orthogonalize(g), g, [COEFFICIENTS] * 5, "five steps")
    near(dg.orthogonalize(g, steps=2, coefficients=(1.5, -0.5, 0.0), scale=-0.3), g, [(1.5, -0.5, 0.0)] * 2, "cubic",
         scale=-0.3)
    each = [(4.0, -6.0, 2.5), COEFFICIENTS, (1.875, -1.25, 0.375)]
    near(dg.orthogonalize(g, steps=3, coefficients=each, eps=1e-3), g, each, "a triple for each step", eps=1e-3)


# more than one, and than two, workgroups a compute unit where a matrix is strips
MANY = [(100, 64, 200), (120, 100, 250), (80, 20, 1500), (75, 500, 128), (40, 2500, 90)]


@pytest.mark.parametrize("size", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_matrices(size):
    batch, M, N = size
    say("orthogonalize", size)
    x = signs(M, N, 4, M + N, batch)
    got = dg.orthogonalize(x, steps=1, coefficients=(2.0, -1.0, 3.0), eps=0.0)
    assert torch.equal(got, exact(x, [(2.0, -1.0, 3.0)], 0.0, 1.0).to(got.dtype))
    g = torch.stack([matrix(M, N, i, torch.float32, "spread") for i in range(batch)])
    got = dg.orthogonalize(g)
    for i in (0, batch // 2, batch - 1):
        near(got[i], g[i], [COEFFICIENTS] * 5, f"{i}")


@pytest.mark.parametrize("size", [(20, 8000), (4090, 64), (96, 2560), (128, 1280), (1, 5000), (100, 1000), (33, 65)],
                         ids=lambda s: "x".join(map(str, s)))
def test_steps_of_few_rows(size):
    M, N = size
    say("orthogonalize", size)
    for dtype in DTYPES.values():
        g = matrix(M, N, M + N, dtype, "spread")
        near(dg.orthogonalize(g), g, [COEFFICIENTS] * 5, "five steps")
        wide = torch.zeros(M + 2, N + 9, device="cuda", dtype=dtype)   # off 16 bytes, rows with gaps
        wide[1:-1, 3:N + 3] = g
        assert torch.equal(dg.orthogonalize(wide[1:-1, 3:N + 3]), dg.orthogonalize(g))
        again = g.clone()
        assert torch.equal(dg.orthogonalize(again, out=again), dg.orthogonalize(g))
        out = torch.full((N + 2, M + 1), 7.0, device="cuda", dtype=dtype)
        dg.orthogonalize(g, out=out[1:-1, :-1].mT)
        assert torch.equal(out[1:-1, :-1].mT, dg.orthogonalize(g))
        assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all()) and bool((out[:, -1] == 7).all())


def test_stacks_and_strides():
    g = gen(4)
    flat = torch.randn(2, 3, 70, 100, generator=g, device="cuda")
    each = dg.orthogonalize(flat)
    assert each.shape == flat.shape
    for i in range(2):
        for j in range(3):
            near(each[i, j], flat[i, j], [COEFFICIENTS] * 5, f"{i} {j}")
            assert torch.equal(each[i, j], dg.orthogonalize(flat[i, j]))
    wide = torch.randn(3, 70, 140, generator=g, device="cuda")
    part = wide[:, 3:60, 5:98]                     # rows and matrices with gaps, off 16 bytes
    got = dg.orthogonalize(part)
    for i in range(3):
        near(got[i], part[i], [COEFFICIENTS] * 5, f"part {i}")
    out = torch.full((3, 70, 140), 7.0, device="cuda")
    dg.orthogonalize(part, out=out[:, 3:60, 5:98])
    assert torch.equal(out[:, 3:60, 5:98], got)
    out[:, 3:60, 5:98] = 7.0
    assert bool((out == 7.0).all())
    turned = torch.empty(3, 93, 57, device="cuda").mT
    assert torch.equal(dg.orthogonalize(part, out=turned), got)
    again = part.clone()
    assert dg.orthogonalize(again, out=again) is again and torch.equal(again, got)   # in place
    for shape in ((0, 4, 5), (3, 0, 5), (3, 4, 0)):
        assert dg.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def test_unusual_values():
    z = torch.zeros(40, 60, device="cuda")
    assert bool((dg.orthogonalize(z) == 0).all())
    for bad in (float("nan"), float("inf"), float("-inf")):
        g = torch.randn(2, 40, 60, generator=gen(2), device="cuda")
        g[0, 3, 5] = bad
        out = dg.orthogonalize(g)
        assert bool(torch.isnan(out[0]).all()) and torch.equal(out[1], dg.orthogonalize(g[1]))
    # norms past FP32's range, and far below the smallest eps
    base = torch.randn(50, 90, generator=gen(3), device="cuda")
    base = base / base.abs().max()
    for by, eps in ((3e38, 1e-7), (1e-30, 0.0), (1e-30, 1e-31)):
        g = base * by
        near(dg.orthogonalize(g, eps=eps), g, [COEFFICIENTS] * 5, f"{by}", eps=eps)
    for shape in ((2, 128, 256), (30, 3000)):   # in strips
        assert bool((dg.orthogonalize(torch.zeros(shape, device="cuda")) == 0).all())
        g = torch.randn(2, *shape[-2:], generator=gen(5), device="cuda")
        g[0, 3, -1] = float("nan")
        out = dg.orthogonalize(g)
        assert bool(torch.isnan(out[0]).all()) and torch.equal(out[1], dg.orthogonalize(g[1]))
    one = torch.zeros(30, 20, device="cuda")
    one[7, 3] = -5.0                       # a single entry
    near(dg.orthogonalize(one), one, [COEFFICIENTS] * 5, "one entry")


def test_graphs_and_streams_share_nothing():
    """Two captured graphs replayed in turn, with eager calls between them and one on a stream of its own."""
    xs = [torch.randn(s, generator=gen(i), device="cuda") for i, s in enumerate(((200, 330), (330, 200)))]
    dg.orthogonalize(xs[0])
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dg.orthogonalize(x))
        graphs.append(graph)
    for turn in range(4):
        for i, x in enumerate(xs):
            x.copy_(torch.randn(x.shape, generator=gen(10 * turn + i), device="cuda"))
        want = [dg.orthogonalize(x.clone()) for x in xs]
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), turn
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dg.orthogonalize(xs[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])


def test_graphs_and_streams_of_few_rows():
    """All steps in one launch and a step in one, captured, replayed in turn and on two streams at once."""
    sizes = [(64, 64), (2, 128, 256), (24, 3000), (100, 90)]
    xs = [torch.randn(s, generator=gen(i), device="cuda") for i, s in enumerate(sizes)]
    for x in xs:
        dg.orthogonalize(x)
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dg.orthogonalize(x))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(4):
        for i, x in enumerate(xs):
            x.copy_(torch.randn(x.shape, generator=gen(10 * turn + i), device="cuda"))
        want = [dg.orthogonalize(x.clone()) for x in xs]
        for graph in graphs:
            graph.replay()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [dg.orthogonalize(x, stream=streams[i % 2]) for _ in range(3) for i, x in enumerate(xs)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), turn
        assert all(torch.equal(a, b) for a, b in zip(got, 3 * want)), turn


def test_a_training_step_and_its_served_weights():
    """A layer's gradient, its orthogonalised update, and the updated weights in 8 bits."""
    g = gen(8)
    M, K, N = 160, 200, 136
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)     # outputs by inputs
    x, dy = (torch.randn(M, d, generator=g, device="cuda").to(torch.bfloat16) for d in (K, N))
    dw = dg.linear_backward(dy, x, w.t(), need_input=False, need_bias=False)[1]            # a transposed view
    update = dg.orthogonalize(dw, scale=0.02)
    near(update, dw, [COEFFICIENTS] * 5, "update", scale=0.02)
    assert update.stride() == dw.stride()
    new = w - update.t()
    q, s = dg.quantize_i8(new)
    xq, sx = dg.quantize_i8(x)
    y = dg.linear_i8(xq, sx, q.t(), s, out_dtype=torch.float32)
    # codes are off by at most half a step each
    exact_y = x.double() @ new.double().t()
    half = 0.5 * (sx.double()[:, None] * new.double().abs().sum(1) + s.double() * x.double().abs().sum(1)[:, None]) \
        + 0.25 * K * sx.double()[:, None] * s.double()
    assert bool(((y.double() - exact_y).abs() <= half * (1 + 1e-6)).all())
