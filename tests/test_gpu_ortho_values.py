"""Orthogonalised updates on the GPU at the ends of their numbers."""
import math
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
