"""Orthogonalised updates on the GPU at the ends of their numbers, and where one
product can be seen by itself: products of few terms whose leading parts cancel."""
import random

import pytest
import torch

from test_gpu_ortho import check, exact

pytestmark = pytest.mark.gpu
BF, SF = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def test_norms_up_to_the_largest_finite_one(L):
    """A norm that is finite in FP32 gives numbers, up to the type's last value;
    past it, NaN."""
    most = torch.finfo(SF).max
    for dtype, v in ((BF, 3.2e38), (BF, torch.finfo(BF).max), (SF, 3.01e38), (SF, most)):
        x = torch.full((1, 1), v, dtype=dtype, device="cuda")
        check(L.orthogonalize([x])[0], x, 5, L.NEWTON_SCHULZ, 1.0, "%s %g" % (dtype, v))
    for shape in ((60, 90), (300, 400), (90, 60)):
        base = torch.randn(shape, dtype=torch.float64, device="cuda")
        x = (base * (3.3e38 / base.norm())).float()
        assert 3.2e38 < float(x.double().norm()) < most
        check(L.orthogonalize([x])[0], x, 5, L.NEWTON_SCHULZ, 1.0, str(shape))
        x = (base * (3.5e38 / base.norm())).float()
        assert bool(torch.isfinite(x).all()) and float(x.double().norm()) > most
        assert bool(torch.isnan(L.orthogonalize([x])[0]).all())


def test_tiny_and_huge_factors(L):
    """y = s * X, rounded once to BF16, for factors from where the result is a
    subnormal number to where it overflows.  X of a 1 x 1 matrix is one number,
    computed here in 64 bits; the kernel's is off by less than 2^-18 of it (five
    steps' pairs of 22 bits and fp32 sums, each step's error grown by at most the
    slope a)."""
    g = random.Random(5)
    scales = [g.uniform(1, 2) * 2.0 ** e for e in range(-134, -118) for _ in range(8)] + [3e38, 1e38, -2.7e-39, 0.0]
    scales = torch.tensor(scales).double().tolist()      # (as the call holds them)
    xs = [torch.full((1, 1), g.uniform(0.5, 2), device="cuda") for _ in scales]
    ys = [torch.full((1, 1), 7.0, dtype=BF, device="cuda") for _ in scales]
    xl = L.LctMatrices(xs)
    L.lct_list_orthogonalize(xl, L.LctMatrices(ys), L.alloc_orthogonal(xl), scale=scales)
    got = torch.cat(ys).view(-1).double().cpu()
    want = torch.tensor([s * float(exact(x.cpu(), 5, L.NEWTON_SCHULZ)) for s, x in zip(scales, xs)], dtype=torch.float64)
    step = torch.clamp(2.0 ** torch.floor(torch.log2(want.abs() + 1e-300)), min=2.0 ** -126) * 2.0 ** -7
    off = (got - want).abs() - 2.0 ** -18 * want.abs()
    assert bool((off <= step / 2).all()), (off / step).max()


def cancelled(coef, pairs):
    """One step on a matrix that holds a 3 x 3 square of ones and nothing else,
    with the numbers that the kernels hold, relative to X0's 1 / 3: every row of
    the square alike, so one element stands for all."""
    a, b, c = coef
    half = lambda v, s: float(torch.tensor(v * s, dtype=torch.float64).float().half()) / s      # noqa: E731

    def pair(v, s):
        h = half(v, s)
        return h, half(v - h, s)

    xh, xl = pair(1 / (3 + 1e-7), 2.0 ** 15)
    lo = xl if pairs else 0.0
    ah, al = pair(3 * (xh * xh + 2 * xh * lo), 2.0 ** 14)
    bh, bl = pair(b * (ah + al) + c * 3 * (ah * ah + 2 * ah * al), 2.0 ** 13)
    bl = bl if pairs else 0.0
    return a * (xh + xl) + 3 * (bh * xh + bh * lo + bl * xh)


@pytest.mark.parametrize("m,n,coefs", [
    (200, 300, [(2, -3, 1), (1, -1, 0)]), (200, 2049, [(2, -3, 1), (1, -1, 0)]), (256, 1024, [(2, -3, 1), (1, -1, 0)]),
    (300, 400, [(0, -1, 1), (1, -2, 1)]), (400, 257, [(0, -1, 1), (1, -2, 1)]), (777, 2049, [(0, -1, 1), (1, -2, 1)]),
    (5120, 10240, [(0, -1, 1), (1, -2, 1)])])
def test_every_product_of_the_pairs(L, m, n, coefs):
    """Coefficients whose sum is zero: of a matrix with one singular value, one,
    nothing is left but what the numbers held in fewer bits leave, 1e-4 of X and
    more.  So a low part that is missing from a product, or a piece of a product's
    long side, would change the result by 1e-4 of X or more (with a single B its
    rounding hides A's low part unless the terms of B cancel too: a = 0 there).
    The square of ones visits every 32 rows and every 32 columns.

    Tolerance: each of the sums of up to nine products rounds at most nine times,
    its factor and the additions three times more, 2^-24 each, for A (which enters
    with |b|, and with |c| twice), A A, B X and a X: together less than 128 * 2^-24
    of X for these coefficients.  A pair's low part may round the other way, 2^-22,
    six times.  A single B may where it is small, 2^-11 of the result (where it is
    not, it lies a sixth of a step from the border).  And half a BF16 step of
    the result."""
    steps = max((m + 31) // 32, (n + 31) // 32)
    more = []
    if m * n > 1 << 24:       # a large one: fewer places, and short matrices beside it, in large tiles too
        places = [0, 1, 63, 64, 101, 159, 160, 200, 318, 319]
        more = [(200, 2049), (2049, 200)]
    else:
        places = range(steps)
    shapes = [(m, n), *more]
    xs = [torch.zeros(s, dtype=BF, device="cuda") for s in shapes]
    ys = [torch.empty_like(x) for x in xs]
    xl, yl = L.LctMatrices(xs), L.LctMatrices(ys)
    work = L.alloc_orthogonal(xl)
    for k in places:
        at = []
        for x in xs:
            r, c = ([(k * 32 + o) % s for o in (1, 14, 27)] for s in x.shape)
            x.zero_()
            x[torch.tensor(r)[:, None], torch.tensor(c)] = 1.0
            at.append((torch.tensor(r)[:, None], torch.tensor(c)))
        for coef in coefs:
            L.lct_list_orthogonalize(xl, yl, work, steps=1, coef=coef)
            for x, y, i in zip(xs, ys, at):
                short = min(x.shape) <= 256
                want = cancelled(coef, short)
                tol = (128 * 2.0 ** -24 + 6 * 2.0 ** -22) / 3 + (2.0 ** -9 + 2.0 ** -11) * abs(want)
                got = y[i].double()
                assert float((got - want).abs().max()) <= tol, (tuple(x.shape), k, coef, got, want)
                assert int((y != 0).sum()) <= 9


def test_lists_of_matrices_with_a_short_side(L):
    """More than a batch holds with whole tiles' sides, and a side near the
    longest."""
    for shapes in ([(16, 8192)] * 33 + [(8192, 9)], [(1, 300_000)] * 5 + [(3, 7)] + [(300_001, 1)] * 3, [(2, 1 << 22), (5, 5)]):
        xs = [torch.randn(s, device="cuda").to(BF) for s in shapes]
        for k, (x, y) in enumerate(zip(xs, L.orthogonalize(xs))):
            check(y, x, 5, L.NEWTON_SCHULZ, 1.0, "%d: %s" % (k, tuple(x.shape)))


@pytest.mark.parametrize("m,n", [(257, 300), (300, 2100), (1024, 700)])
def test_errors_of_many_steps(L, m, n):
    """The error of many steps is that of the documented roundings: as large as
    the same iteration leaves in 64 bits with them.  They are made anew for each
    element, so the two errors' norms, of m and more directions, differ by chance
    as 1 / sqrt(m), at most a sixteenth; three times that is allowed."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, n, generator=g, device="cuda")
    for steps in (5, 8, 12):
        y = torch.empty(m, n, dtype=BF, device="cuda")
        xl = L.LctMatrices([x])
        L.lct_list_orthogonalize(xl, L.LctMatrices([y]), L.alloc_orthogonal(xl), steps=steps)
        e, r = exact(x, steps, L.NEWTON_SCHULZ), exact(x, steps, L.NEWTON_SCHULZ, rounded=True)
        got, model = float((y.double() - e).norm()), float((r - e).norm())
        assert abs(got - model) <= 3 / 16 * model, (steps, got / float(e.norm()), model / float(e.norm()))
