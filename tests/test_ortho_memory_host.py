"""Working memory of orthogonalised updates (no GPU): what long lists and
matrices with a short side take."""
import ctypes as C

import pytest
import torch

from test_norms_host import FakeList


@pytest.fixture(scope="module")
def L():
    import lossless_bf16_tensor_split_amd as L
    return L


ROOM = 17 << 20   # parts of sums, norms


def need(L, shapes):
    ns = [m * n for m, n in shapes]
    x = FakeList(L, ns, [0x1000_0000_0000 + (k << 40) for k in range(len(ns))], [L.BF16] * len(ns))
    out = C.c_uint64(0)
    assert L.lib.lct_orthogonal_scratch(x.ref, (C.c_uint64 * len(ns))(*[m for m, _ in shapes]), C.byref(out)) == L.OK
    return out.value


def most(shape):
    """What a matrix may take, its sides rounded up to 128: 8 bytes an element
    and 6 for each of m * m (12 and 8 for at most 256 rows)."""
    m, n = sorted(shape)
    a, b = (12, 8) if m <= 256 else (8, 6)
    m, n = -(-m // 128) * 128, -(-n // 128) * 128
    return a * m * n + b * m * m


@pytest.mark.parametrize("shapes", [[(16, 8192)] * 32, [(64, 6400)] * 32, [(1, 1 << 22)] * 31, [(1 << 22, 1)],
                                    [(130, 50_000)] * 20])
def test_short_sides_are_rounded_up_to_small_tiles(L, shapes):
    """However many tiles they make: large ones would double the memory and the
    work."""
    assert need(L, shapes) <= sum(most(s) for s in shapes) + ROOM


def test_large_matrices_beside_short_ones(L):
    """Where most of the work is large matrices', the short ones are rounded up
    with them; none takes more than four times its own rounding."""
    shapes = [(2560, 9728)] * 4 + [(100, 9000), (1, 5)]
    assert need(L, shapes) <= sum(most(s) for s in shapes[:4]) + 4 * sum(most(s) for s in shapes[4:]) + ROOM


@pytest.mark.parametrize("shape", [(1, 1 << 22), (1 << 22, 1), (9, 65536), (100, 300_000), (1, 1 << 20), (200, 500_000)])
def test_lists_of_matrices_with_a_short_side(L, shape):
    """A batch gathers at most 2^27 elements with whole tiles' sides (a larger
    matrix is one by itself), however few of them are the matrices' own."""
    one = most(shape)
    m, n = (-(-s // 128) * 128 for s in shape)
    batch = max(1, min(32, (1 << 27) // (m * n)))
    for count in (1, 31, 32, 200):
        assert need(L, [shape] * count) <= min(count, batch) * one + ROOM, count


@pytest.mark.parametrize("shape", [(256, 256), (257, 256), (257, 300), (2560, 9728), (1000, 1000), (4096, 4096), (1, 1)])
def test_memory_of_a_matrix(L, shape):
    """The documented bytes of one matrix, and not much less."""
    bytes = most(shape) if min(shape) < 4096 else most([-(-s // 256) * 256 for s in shape])
    assert bytes <= need(L, [shape]) <= bytes + ROOM
