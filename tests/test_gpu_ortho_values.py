"""Orthogonalised updates on the GPU at the ends of their numbers."""
import math
import random

import pytest
import torch

from test_gpu_ortho import check

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
