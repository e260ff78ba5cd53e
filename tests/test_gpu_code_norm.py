"""Norms of compressed tensors on the GPU: a tensor read with a codebook that
is not its own, and the bits of the sums."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def values(y):
    torch.cuda.synchronize()
    return y.cpu().double().numpy()


def code_norm(L, cb, t, kind):
    out = L.alloc_norm(nblk=t.sizes.nblk)
    L.lct_tensor_norm(cb, t, out, kind=kind)
    torch.cuda.synchronize()
    return float(out.sum)


@pytest.mark.parametrize("lay", [(65536, 25), (32768, 12), (4096, 25), (16384, 3)])
def test_a_tensor_read_with_another_codebook(L, lay):
    """Its streams run out of bits before they run out of positions: the norm
    then reads zeros, as the decoder does, so it is the norm of what that
    decodes to.  Zeros read as a field whose values outweigh all others' (its
    squares leave the range of fp32 sums), so one field read from elsewhere
    shows in the sum."""
    n = 2 * lay[0] + lay[0] // 3
    x = (torch.randn(n, generator=torch.Generator().manual_seed(n)) * 0.02).to(BF).cuda()
    own = L.lct_codebook_build(L.Model(L.GAUSSIAN, 0.02, 0.0), x)
    t = L.encode(own, x, L.layout(*lay))
    length = np.zeros(256, np.uint8)
    length[97:158] = 6                           # more bits than the streams hold
    length[250] = 5                              # the code of zero bits
    other = L.lct_codebook_from_lengths(length, 6)
    y = values(L.decode(other, t))
    past = (np.abs(y) >= 2.0 ** 123).sum()
    assert np.isfinite(y).all() and (past > n // 4 or lay == (4096, 25))
    v = y.astype(np.longdouble)
    want = float((v * v).sum())
    assert abs(code_norm(L, other, t, L.NORM_L2) - want) <= want * (n + 64) * 2.0 ** -53
    assert code_norm(L, other, t, L.NORM_MAX) == np.abs(y).max()
    # and its own codebook still reads the tensor
    assert code_norm(L, own, t, L.NORM_MAX) == np.abs(values(x)).max()


@pytest.mark.parametrize("lay,heavy", [((65536, 25), False), ((32768, 12), True), ((32768, 11), True),
                                       ((4096, 2), False)])
def test_sums_hold_64_bits(L, lay, heavy):
    """S is summed in 64 bits from the first square on: a square is exact (16
    significant bits), and an addition is off by 2^-53 of a partial sum that
    is at most S.  On its way a square meets one addition for each later
    position of its stream, six joins of the lanes, three of a block's waves
    and six of the blocks' values (38 blocks: one wave; the other waves' zeros
    add exactly)."""
    n = 37 * lay[0] + 1001
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g) * 0.02
    if heavy:                                    # many fields spill
        x *= torch.exp2(torch.randint(-20, 8, (n,), generator=g).float())
    x = x.to(BF).cuda()
    cb = L.lct_codebook_build(L.Model(L.GAUSSIAN, 0.02, 0.0), x)
    t = L.encode(cb, x, L.layout(*lay))
    if heavy:
        assert t.spilled() > 0
    v = values(x).astype(np.longdouble)
    want = (v * v).sum()
    adds = lay[0] // 256 + 6 + 3 + 6
    assert abs(code_norm(L, cb, t, L.NORM_L2) - want) <= want * adds * 2.0 ** -53
    # dense, of the same values: the two sums differ by their order only
    out = L.grad_norm([x])
    assert abs(float(out.sum) - want) <= want * (n + 64) * 2.0 ** -53
