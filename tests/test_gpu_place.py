"""Placing spilled bytes: more blocks than one scan group holds, in overflow
regions of every length around what they need, byte for byte against the oracle
where they hold everything, and with a guard behind the region."""
import numpy as np
import pytest
import torch

import synth
from test_gpu_parity import assert_same, check_codebook, dev, host_parts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def heavy(n, sigma, seed):
    """Normal values, a part of the streams spilling in most units and, in some
    blocks, none."""
    g = np.random.default_rng(seed)
    x = g.normal(0.0, sigma, n)
    at = np.arange(n) // 4096 % 5 != 0
    x[at] *= np.exp2(g.integers(-3, 3, at.sum()) * 4.0)
    return synth.to_bf16_bits(x)


@pytest.mark.parametrize("blocks", [200, 300, 2500])
def test_spills_in_regions_of_every_length(L, orc, blocks):
    """200 blocks are settled in one launch, 300 and 2500 scanned and then
    placed; 2500 have more units than the placing waves take at once."""
    n = blocks * 4096 - 1234
    x = heavy(n, 0.02, blocks)
    model = synth.Model(synth.GAUSSIAN, 0.02, 0.0)
    cb, ocb = check_codebook(L, orc, model, x)
    lay, xd = L.layout(4096, 3), dev(x)
    need = orc.encode(ocb, x, 4096, 3).spilled
    assert need > 50 * blocks
    for cap in (need + 777, need, need - 1, need - need // 3, 65, 1):
        ref = orc.encode(ocb, x, 4096, 3, cap)
        ovf = torch.full((cap + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        t = L.alloc_tensor(n, lay, cap, ovf=ovf)
        L.lct_encode(cb, xd, t)
        g = host_parts(t)
        assert g["status"] == (0 if cap >= need else L.ST_OVF_FULL)
        assert np.array_equal(g["obase"], ref.obase)
        if cap >= need:                          # (else the region's contents are not specified)
            assert_same(g, ref, "cap %d of %d" % (cap, need))
        assert bool((ovf[cap:] == 0xA5).all()), "guard behind %d bytes" % cap
