"""Matrices on which the orthogonalised update's errors have tight bounds, and its
arithmetic in two terms, for torch on any device.

Blocks of 2 x 2 entries in rows and columns of their own: a sum of the products has at
most two products that are not zero, and an error stays in its block, so a step's
roundings are followed entry by entry.  With u = 2^-24, what a step adds to an entry is
  of a product: lo lo, which is left out, 4 u; and up to eight roundings of 2 u each (two
  products in three instructions, and sums kept apart), together 20 u of the sum of the
  magnitudes;
  of two terms: 2 u, and 2^-39 of the operand's bound where they end;
  of P: 4 u of its terms' magnitudes, of the factor, the scale and the result's own
  rounding u each.
Dropping a lower term anywhere is an error of up to 2^-11 of an entry, 2^-13 in the mean."""
import torch

U = 2.0 ** -24
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


class Blocks:
    """Blocks of an m x n stack of `batch` matrices, m <= n: (batch, K, 2, 2), and where
    they lie."""

    def __init__(self, batch, m, n, seed, device):
        g = torch.Generator(device=device).manual_seed(seed)
        k = max(m // 2, 1)
        self.shape, self.k = (batch, m, n), k

        def places(size):   # (a single row or column counts as both of its block's)
            at = torch.stack([torch.randperm(size, generator=g, device=device)[:2 * k] for _ in range(batch)])
            return at.expand(batch, 2) if size == 1 else at
        rows, cols = places(m), places(n)
        v = torch.rand(batch, k, 2, 2, generator=g, device=device) * 0.5 + 0.5
        v = v * (torch.randint(0, 2, v.shape, generator=g, device=device) * 2 - 1)
        if m == 1:
            v[..., 1, :] = 0
        if n == 1:
            v[..., :, 1] = 0
        self.values = v
        self.rows, self.cols = rows.view(batch, k, 2, 1), cols.view(batch, k, 1, 2)

    def dense(self, v):
        b, m, n = self.shape
        out = v.new_zeros(b, m * n)
        out.scatter_add_(1, (self.rows * n + self.cols).reshape(b, -1), v.reshape(b, -1))
        return out.view(b, m, n)


def _mm(a, b):
    return torch.matmul(a, b)


def _bounds(each):
    """The largest singular value before each step, and the largest of what multiplies it."""
    s = torch.linspace(0, 1, 4001, dtype=torch.float64)
    r, out = 1.0, []
    for a, b, c in each:
        t = (s * r) ** 2
        p = (a + t * (b + t * c)).abs()
        out.append((r, float(p.max())))
        r = float((s * r * p).max())
    return out


def exact_and_error(values, each, eps=0.0):
    """The steps in 64 bits on blocks, and a bound of the kernels' error before the result
    is rounded, entry by entry."""
    x = values.double()
    x = x / (x.square().sum((1, 2, 3), keepdim=True).sqrt() + eps)
    end = 2.0 ** -39
    e = 3 * U * x.abs() + end
    eye = torch.eye(2, dtype=torch.float64, device=x.device)
    for (a, b, c), (r, p) in zip(each, _bounds(each)):
        ax = x.abs()
        gram, agram = _mm(x, x.mT), _mm(ax, ax.mT)
        eg = _mm(ax, e.mT) + _mm(e, ax.mT) + _mm(e, e.mT) + 20 * U * agram
        eg = eg + 2 * U * (gram.abs() + eg) + end * r * r
        g = gram.abs()
        square = _mm(gram, gram)
        asq = _mm(g, g)
        es = _mm(g, eg) + _mm(eg, g) + _mm(eg, eg) + 20 * U * asq
        poly = a * eye + b * gram + c * square
        ep = abs(b) * eg + abs(c) * es + 4 * U * (abs(a) * eye + abs(b) * g + abs(c) * asq)
        ep = ep + 2 * U * (poly.abs() + ep) + end * p
        y = _mm(poly, x)
        ey = _mm(ep, ax) + _mm(poly.abs(), e) + _mm(ep, e) + 20 * U * _mm(poly.abs(), ax)
        x, e = y, ey + 3 * U * (y.abs() + ey) + end * p * r
    return x, e


def steps_for(m, last):
    """Default steps that bring blocks of an m-row matrix to singular values of about a
    half, then `last`, in which A and A A are all there is."""
    k, s = 0, m ** -0.5
    while 3.4445 * s < 0.6:
        k, s = k + 1, 3.4445 * s
    return [COEFFICIENTS] * k + [last]


LAST = [(0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.0, -1.0, 2.0)]


def two_terms(v, most, keep=True):
    """v (32 bits) in two binary16 terms at the power of two of the bound `most`."""
    by = 2.0 ** torch.floor(torch.log2(torch.tensor(60000.0 / most, dtype=torch.float64))).item()
    y = (v * by).float()
    hi = y.half().float()
    lo = (y - hi).half().float() if keep else torch.zeros_like(y)
    return hi / by, lo / by


def product(a, b):
    """Products of pairs of terms, without lo lo, summed in 32 bits."""
    return a[0] @ b[0] + (a[1] @ b[0] + a[0] @ b[1])


def simulate(values, each, drop=None):
    """The kernels' arithmetic on blocks; `drop` names an operand whose lower term is lost."""
    x = (values.double() / values.double().square().sum((1, 2, 3), keepdim=True).sqrt()).float()
    eye = torch.eye(2, device=x.device)
    for (a, b, c), (r, p) in zip(each, _bounds(each)):
        def x_as(name):
            return two_terms(x, r, drop != name)
        first, second = x_as("X, first of X X^T"), x_as("X, second of X X^T")
        gram = product(first, tuple(t.mT for t in second))
        square = product(two_terms(gram, r * r, drop != "A, first of A A"),
                         tuple(t.mT for t in two_terms(gram, r * r, drop != "A, second of A A")))
        held = sum(two_terms(gram, r * r, drop != "A, in P"))
        poly = (c * square.double() + (b * held.double() + a * eye.double())).float()
        x = product(two_terms(poly, p, drop != "P"), x_as("X, in P X"))
    return x


OPERANDS = ["X, first of X X^T", "X, second of X X^T", "A, first of A A", "A, second of A A", "A, in P", "P", "X, in P X"]
