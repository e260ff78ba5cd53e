"""Orthogonalised updates on the GPU against the definition in 64 bits.

Tolerance.  The kernels document where numbers are rounded to fewer bits: X to a
pair of FP16 numbers of which the products see the first, A to a pair, B to one,
y to BF16; of matrices of at most 256 rows (or columns) the products see pairs
throughout.  ``rounded`` makes the iteration in 64 bits with those roundings.
Beside it the kernels round their sums to fp32: a sum of K products by at most
sqrt(K) * 2^-24 (signs fall either way) of the operands' norms, three sums a
step, and what lies in directions that X hardly has is multiplied by at most a
each step: a^5 * sqrt(3 K) * 2^-24 < 5e-5 * sqrt(K) relative to the result.  The
result's distance from the exact one is that of ``rounded`` and no more than that
besides (norms)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def exact(x, steps, coef, scale=1.0, rounded=False):
    a, b, c = coef
    v = x.double()
    tall = v.shape[0] > v.shape[1]
    v = v.T.contiguous() if tall else v
    v = v / (v.norm() + 1e-7)
    pairs = v.shape[0] <= 256
    h = lambda t, s: (t * s).to(torch.float32).to(HF).double() / s      # noqa: E731
    pair = lambda t, s: h(t, s) + h(t - h(t, s), s)                     # noqa: E731
    for k in range(steps):
        if rounded:
            v = pair(v, 2.0 ** 15)
        w = h(v, 2.0 ** 15) if rounded and not pairs else v
        p = torch.mm(w, w.T.contiguous())
        if rounded:
            p = pair(p, 2.0 ** 14)
        q = b * p + c * torch.mm(p, p)
        if rounded:
            q = (pair if pairs else h)(q, 2.0 ** 13)
        v = a * v + torch.mm(q, w)
    v = scale * (v.T if tall else v)
    return v.to(SF).to(BF).double() if rounded else v


def check(y, x, steps, coef, scale=1.0, what=""):
    e = exact(x, steps, coef, scale)
    r = exact(x, steps, coef, scale, True)
    norm = float(e.norm())
    allowed = float((r - e).norm()) + 5e-5 * math.sqrt(max(x.shape)) * norm
    got = float((y.double() - e).norm())
    assert got <= allowed, "%s: off by %.3g of the norm, %.3g allowed" % (what, got / norm, allowed / norm)


def matrix(m, n, kind, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + m * 1009 + n)
    x = torch.randn(m, n, generator=g, device="cuda")
    if kind == "low":      # a few directions, and next to nothing in the others
        r = min(4, m, n)
        x = torch.randn(m, r, generator=g, device="cuda") @ torch.randn(r, n, generator=g, device="cuda") + 1e-3 * x
    return (x * (1e-3 if dtype != HF else 0.1)).to(dtype)


SHAPES = [(1, 1), (1, 7), (9, 1), (3, 5), (17, 16), (64, 64), (127, 129), (128, 128), (129, 127), (255, 300), (400, 100),
          (256, 1031), (700, 640)]


@pytest.mark.parametrize("kind", ["full", "low"])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_shapes_in_one_list(L, dtype, kind):
    xs = [matrix(m, n, kind, dtype) for m, n in SHAPES]
    ys = [torch.full(x.shape, 7.0, dtype=BF, device="cuda") for x in xs]
    before = [x.clone() for x in xs]
    xl, yl = L.LctMatrices(xs), L.LctMatrices(ys)
    scales = [0.2 * math.sqrt(max(s)) for s in SHAPES]
    L.lct_list_orthogonalize(xl, yl, L.alloc_orthogonal(xl), scale=scales)
    for x, y, s, was in zip(xs, ys, scales, before):
        check(y, x, 5, L.NEWTON_SCHULZ, s, str(tuple(x.shape)))
        assert torch.equal(x, was)


@pytest.mark.parametrize("m,n", [(1024, 2100), (2305, 768)])
def test_larger_matrices(L, m, n):
    for kind in ("full", "low"):
        x = matrix(m, n, kind, BF)
        check(L.orthogonalize([x])[0], x, 5, L.NEWTON_SCHULZ, 1.0, "%d x %d %s" % (m, n, kind))


def test_many_large_matrices(L):
    """Enough of them for the large tiles, in two batches, short ones among
    them."""
    shapes = [(1024, 2048)] * 13 + [(200, 300), (2304, 768), (1, 5)] + [(1024, 2048)] * 13 + [(900, 1300)] * 8
    xs = [matrix(m, n, "full", BF, k) for k, (m, n) in enumerate(shapes)]
    ys = L.orthogonalize(xs)
    for k in (0, 13, 14, 15, 20, len(xs) - 1):
        check(ys[k], xs[k], 5, L.NEWTON_SCHULZ, 1.0, str(tuple(xs[k].shape)))


@pytest.mark.parametrize("steps", [1, 2, 3, 6])
def test_steps_and_coefficients(L, steps):
    for coef in (L.NEWTON_SCHULZ, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0)):
        x = matrix(200, 300, "full", SF)
        y = torch.empty(200, 300, dtype=BF, device="cuda")
        xl = L.LctMatrices([x])
        L.lct_list_orthogonalize(xl, L.LctMatrices([y]), L.alloc_orthogonal(xl), steps=steps, coef=coef)
        check(y, x, steps, coef, 1.0, "%s, %d steps" % (coef, steps))


def test_result_is_near_orthogonal(L):
    """What the operator is for: singular values within the quintic's band."""
    x = matrix(256, 512, "full", BF)
    s = torch.linalg.svdvals(L.orthogonalize([x])[0].cpu().double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


def test_scales_of_values(L):
    """Norms from next to nothing (where the 1e-7 counts) to near the type's
    end; power-of-two scales change nothing else."""
    base = torch.randn(60, 90, device="cuda", dtype=torch.float64)
    for dtype, scale in ((SF, 1e-38), (SF, 1e-9), (SF, 1e-7), (SF, 1e30), (BF, 1e-30), (BF, 1e-6), (BF, 1e35), (HF, 1e-6),
                         (HF, 1e3)):
        x = (base * scale).to(dtype)
        y = L.orthogonalize([x])[0]
        if float(x.double().norm()) < 1e-12:   # values near zero on the whole
            assert float(y.abs().max()) <= 500 * float(x.double().norm()) / 1e-7
            continue
        check(y, x, 5, L.NEWTON_SCHULZ, 1.0, "%s %g" % (dtype, scale))


def test_zeros_and_values_out_of_the_ordinary(L):
    """Zeros give zeros; a NaN or an infinity makes its matrix NaN and touches
    no other."""
    xs = [torch.zeros(70, 130, dtype=BF, device="cuda"), matrix(70, 130, "full", BF), matrix(130, 70, "full", BF),
          matrix(70, 130, "full", BF)]
    xs[1][3, 5] = float("nan")
    xs[2][129, 69] = float("inf")
    ys = L.orthogonalize(xs)
    assert bool((ys[0] == 0).all())
    assert bool(torch.isnan(ys[1]).all()) and bool(torch.isnan(ys[2]).all())
    check(ys[3], xs[3], 5, L.NEWTON_SCHULZ)


def test_stacked_matrices_views_and_empty_ones(L):
    """A tensor of three dimensions is a matrix each; results at odd places of
    one buffer leave what lies beside them; matrices without elements."""
    x = torch.stack([matrix(65, 130, "full", BF, k) for k in range(3)])
    flat = torch.full((3 * 65 * 130 + 20,), 7.0, dtype=BF, device="cuda")
    y = flat[5:5 + x.numel()].view(3, 65, 130)
    empty = torch.empty(0, 5, dtype=BF, device="cuda")
    xl = L.LctMatrices([x, empty])
    assert len(xl) == 4
    L.lct_list_orthogonalize(xl, L.LctMatrices([y, empty.clone()]), L.alloc_orthogonal(xl))
    for k in range(3):
        check(y[k], x[k], 5, L.NEWTON_SCHULZ)
    assert bool((flat[:5] == 7.0).all() and (flat[5 + x.numel():] == 7.0).all())


def test_in_place_repeats_and_bounded_memory(L):
    """In place, the same bits; the working memory holds a guard behind it."""
    xs = [matrix(m, n, "full", BF) for m, n in ((300, 200), (64, 500))]
    want = L.orthogonalize(xs)
    xl = L.LctMatrices(xs)
    work = L.alloc_orthogonal(xl)
    need = work.scratch.numel()
    work.scratch = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    again = [torch.empty_like(x) for x in xs]
    L.lct_list_orthogonalize(xl, L.LctMatrices(again), work)
    L.lct_list_orthogonalize(xl, xl, work)
    for w, a, x in zip(want, again, xs):
        assert torch.equal(w, a) and torch.equal(w, x)
    assert bool((work.scratch[need:] == 0x5A).all())


def test_two_streams_at_once(L):
    cases = []
    for k in range(2):
        xs = [matrix(300 + 50 * k, 400, "full", BF, k)]
        xl, ys = L.LctMatrices(xs), [torch.empty_like(xs[0])]
        cases.append((xl, L.LctMatrices(ys), L.alloc_orthogonal(xl), L.orthogonalize(xs)[0], ys[0], torch.cuda.Stream(), xs))
    torch.cuda.synchronize()
    for _ in range(10):
        for xl, yl, work, _, _, st, _ in cases:
            L.lct_list_orthogonalize(xl, yl, work, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[3], c[4])


def test_replayed_from_a_graph(L):
    xs = [matrix(m, n, "full", BF) for m, n in ((300, 200), (64, 500), (1, 9))]
    ys = [torch.empty_like(x) for x in xs]
    xl, yl = L.LctMatrices(xs), L.LctMatrices(ys)
    work = L.alloc_orthogonal(xl)
    L.lct_list_orthogonalize(xl, yl, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lct_list_orthogonalize(xl, yl, work)
    for rep in range(4):
        for x in xs:
            x.copy_(torch.randn(x.shape, device="cuda"))
        want = L.orthogonalize(xs)
        for y in ys:
            y.zero_()
        work.scratch.fill_(0x7F)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, ys):
            assert torch.equal(a, b), rep
