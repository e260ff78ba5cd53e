"""Host-side refusals of a group's norm (no GPU): the group descriptor is filled
by hand as a bind fills it, over addresses that are never dereferenced."""
import ctypes as C

import pytest

SCR, EACH, OUT, TABLE, BASE = (k << 40 for k in (0x60, 0x70, 0x71, 0x20, 0x10))


@pytest.fixture(scope="module")
def L():
    import lossless_bf16_tensor_split_amd as L
    return L


def fingerprint(ns, lay):
    """A bound group's: FNV-1a over the layout, the count and the sizes, eight
    bytes each."""
    h = 1469598103934665603
    for v in [lay.block_elems, lay.cap_words, len(ns)] + list(ns):
        for b in int(v).to_bytes(8, "little"):
            h = (h ^ b) * 1099511628211 & (1 << 64) - 1
    return h


class Bound:
    """A group of ns elements and its storage."""

    def __init__(self, L, ns, lay):
        self.L, self.arr = L, (C.c_uint64 * len(ns))(*ns)
        self.nblk = sum(-(-n // lay.block_elems) for n in ns)
        sf = sum(-(-n // 256) * 256 for n in ns)
        self.g = L.Group(len(ns), lay, self.nblk, sf, fingerprint(ns, lay), C.cast(self.arr, C.c_void_p), None, TABLE)
        b = C.c_uint64(0)
        assert L.lib.lct_group_table_bytes(len(ns), self.arr, C.byref(lay), C.byref(b)) == L.OK
        self.table_bytes = b.value
        assert L.lib.lct_norm_scratch(0, self.nblk, C.byref(b)) == L.OK
        self.scratch_bytes = b.value
        at = [BASE + (k << 32) for k in range(7)]
        self.all = L._Tensor(sf, lay, *at[:5], 100, at[5], at[6])

    def norm(self, scr=SCR, each=EACH, out=OUT):
        return self.L.lib.lct_group_norm(C.byref(self.g), C.byref(self.all), 0, 1.0, 1.0, C.c_void_p(scr),
                                         C.c_void_p(each), C.c_void_p(out), None)


@pytest.mark.parametrize("ns", [[100000, 0, 77, 70000], [0, 0]])
def test_outputs_on_the_groups_table_are_refused(L, ns):
    """The table holds the codebooks, members and blocks that the norm's
    kernels read while they write their results; the members also where the
    group has no blocks."""
    b = Bound(L, ns, L.layout(65536, 25))
    assert b.norm(out=OUT + 4) == L.EALIGN            # (the descriptor passes for a bound one)
    end = TABLE + b.table_bytes
    for kw in ({"scr": TABLE}, {"scr": TABLE + 256}, {"scr": end - 256}, {"scr": TABLE - b.scratch_bytes + 256},
               {"out": TABLE}, {"out": end - 16}, {"out": TABLE - 8}, {"each": TABLE + 4}, {"each": end - 4},
               {"each": TABLE - 4 * len(ns) + 4}):
        assert b.norm(**kw) == L.EALIAS, kw
    if b.nblk:
        for kw in ({"scr": BASE}, {"out": BASE + (1 << 32)}, {"each": BASE + (2 << 32)}):
            assert b.norm(**kw) == L.EALIAS, kw


def test_another_fingerprint_is_refused(L):
    b = Bound(L, [100000, 77], L.layout(65536, 25))
    b.g.shape_hash ^= 1
    assert b.norm(out=OUT + 4) == L.EINVAL
