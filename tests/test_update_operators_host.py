"""Host-side checks of the mix, the table's rows and gradient, and the
orthogonalisation (no GPU): every refusal of the C calls before anything reaches
a device (addresses are made up and never read), scratch sizes, and the Python
calls' checks of their tensors."""
import ctypes as C

import pytest
import torch

from test_boundary_host import _fake_tensor
from test_norms_host import FakeList

A, B, D, E = 0x1000_0000_0000, 0x2000_0000_0000, 0x3000_0000_0000, 0x4000_0000_0000
SCR = 0x6000_0000_0000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import lossless_bf16_tensor_split_amd as L
    return L


def ptr(v):
    return None if v is None else C.c_void_p(v)


# ------------------------------------------------------------------ mix

def mix(L, t, o, cb, x=E, b=1.0, coef=None, cb_out=None, dense=None, ahead=0):
    return L.lib.lct_mix_step(cb and C.byref(cb), t and C.byref(t), 0.9, ptr(x), b, ptr(coef),
                              C.byref(cb_out if cb_out is not None else cb) if cb else None, o and C.byref(o),
                              ptr(dense), ahead, None)


def test_mix_refusals(L):
    lay, n = L.layout(65536, 25), 100_000
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None)
    t, o = _fake_tensor(L, n, lay, A), _fake_tensor(L, n, lay, B)
    ok = L.EARCH, L.EHIP   # every check passed: only the device is missing here
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a device")
    assert mix(L, t, o, cb) in ok
    assert mix(L, t, o, cb, dense=E, ahead=1) in ok                  # over x itself
    assert mix(L, t, t, cb) == L.EALIAS                              # scratch and overflow are the output's own
    assert mix(L, None, o, cb) == mix(L, t, None, cb) == mix(L, t, o, None) == L.EINVAL
    assert mix(L, t, o, cb, x=None) == L.EINVAL
    assert mix(L, t, o, cb, ahead=1) == L.EINVAL                     # nowhere to look ahead to
    assert mix(L, t, o, cb, cb_out=L.Codebook()) == L.EINVAL         # a codebook that was never built
    assert mix(L, t, _fake_tensor(L, n + 1, lay, B), cb) == L.EINVAL
    assert mix(L, t, _fake_tensor(L, n, L.layout(65536, 24), B), cb) == L.EINVAL
    assert mix(L, t, o, cb, x=E + 8) == mix(L, t, o, cb, dense=D + 2) == L.EALIGN
    assert mix(L, t, o, cb, coef=D + 2) == L.EALIGN
    assert mix(L, t, o, cb, x=o.sf) == mix(L, t, o, cb, x=o.scratch) == L.EALIAS
    assert mix(L, t, o, cb, dense=E + 16) == L.EALIAS                # half over x
    assert mix(L, t, o, cb, dense=t.sf) == mix(L, t, o, cb, dense=o.pay) == L.EALIAS
    assert mix(L, t, o, cb, coef=o.status) == L.EALIAS
    assert mix(L, t, o, cb, coef=D + 4, dense=D) == L.EALIAS
    # in place: the fixed side, and nothing but it
    same = _fake_tensor(L, n, lay, B, sf=t.sf, pay=t.pay, cnt=t.cnt, obase=t.obase)
    assert mix(L, t, same, cb) in ok
    assert mix(L, t, _fake_tensor(L, n, lay, B, sf=t.pay), cb) == L.EALIAS
    assert mix(L, t, _fake_tensor(L, n, lay, B, ovf=t.ovf), cb) == L.EALIAS
    assert mix(L, _fake_tensor(L, 0, lay, A), _fake_tensor(L, 0, lay, B), cb, x=None) == L.OK


# ------------------------------------------------------------------ rows and their gradient

def rows_scratch(L, count, cols):
    out = C.c_uint64(0)
    assert L.lib.lct_rows_scratch(count, cols, C.byref(out)) == L.OK
    return out.value


def test_rows_scratch(L):
    assert rows_scratch(L, 1000, 0) < rows_scratch(L, 1000, 64) < rows_scratch(L, 2000, 64)
    assert rows_scratch(L, 0, 0) <= 4096
    for bad in ((1 << 31, 1), (1, (1 << 24) + 1)):
        assert L.lib.lct_rows_scratch(*bad, C.byref(C.c_uint64())) == L.EINVAL
    assert L.lib.lct_rows_scratch(1, 1, None) == L.EINVAL


def test_rows_scratch_for_many_tokens_does_for_fewer(L):
    counts = sorted({c for k in range(0, 23) for c in ((1 << k) - 1, 1 << k, (1 << k) + 1, 3 << k, (3 << k) + 1)})
    for cols in (0, 1, 64, 2560):
        sizes = [rows_scratch(L, c, cols) for c in counts]
        assert sizes == sorted(sizes), cols


def test_lookup_refusals(L):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a device")
    lay, n = L.layout(65536, 25), 96_000
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None)
    t = _fake_tensor(L, n, lay, A)

    def call(cb=cb, t=t, cols=96, index=B, wide=1, count=10, y=D, ty=L.BF16, scr=None):
        return L.lib.lct_tensor_rows(cb and C.byref(cb), t and C.byref(t), cols, ptr(index), wide, count, 1.0, ptr(y), ty,
                                     ptr(scr), None)

    assert call() in (L.EARCH, L.EHIP) and call(scr=SCR) in (L.EARCH, L.EHIP)
    assert call(cb=None) == call(t=None) == call(index=None) == call(y=None) == L.EINVAL
    assert call(cols=0) == call(cols=97) == call(ty=3) == call(ty=-1) == L.EINVAL
    assert call(cols=1 << 25) == call(count=1 << 31) == L.EINVAL
    assert call(index=B + 4) == call(index=B + 2, wide=0) == call(y=D + 1) == call(y=D + 2, ty=L.FP32) == L.EALIGN
    assert call(scr=SCR + 16) == L.EALIGN
    assert call(y=B) == call(y=t.sf) == call(y=t.pay) == call(scr=B) == call(scr=D, y=D) == L.EALIAS
    assert call(count=0, index=None, y=None) == L.OK


def test_grad_refusals(L):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a device")

    def call(index=A, wide=1, count=100, dy=B, ty=L.BF16, rows=1000, cols=64, g=D, tg=L.BF16, scr=SCR):
        return L.lib.lct_rows_grad(ptr(index), wide, count, ptr(dy), ty, rows, cols, 1.0, 0, ptr(g), tg, ptr(scr), None)

    assert call() in (L.EARCH, L.EHIP)
    assert call(index=None) == call(dy=None) == call(g=None) == call(scr=None) == L.EINVAL
    assert call(ty=5) == call(tg=5) == call(count=1 << 31) == call(rows=(1 << 29) + 1) == call(cols=1 << 25) == L.EINVAL
    assert call(index=A + 4) == call(dy=B + 1) == call(g=D + 2, tg=L.FP32) == call(scr=SCR + 8) == L.EALIGN
    assert call(g=B) == call(g=A) == call(scr=A) == call(scr=B) == call(g=SCR) == L.EALIAS
    assert call(rows=0, g=None, scr=None) == call(cols=0, g=None, scr=None) == L.OK


def test_lookup_and_grad_check_their_tensors(L):
    """CPU tensors, wrong types and shapes never reach the library."""
    lay = L.layout(65536, 25)
    index, y = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8)
    t = L.LctTensor.wrap(64, lay, 0, L.lct_sizes(64, lay), *[torch.zeros(256, dtype=torch.uint8)] * 7)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None)
    with pytest.raises(TypeError, match="int64 or int32"):
        L.lct_tensor_rows(cb, t, index.float(), y)
    with pytest.raises(ValueError, match="contiguous"):
        L.lct_tensor_rows(cb, t, torch.zeros(6, dtype=torch.int64)[::2], y)
    with pytest.raises(ValueError, match="GPU"):
        L.lct_tensor_rows(cb, t, index, y)
    with pytest.raises(ValueError, match="GPU"):
        L.lct_rows_grad(index, y, y, L.RowsWork(torch.zeros(1 << 16, dtype=torch.uint8)))


# ------------------------------------------------------------------ orthogonalisation

def ortho(L, x, rows, y, steps=5, coef=(3.4445, -4.7750, 2.0315), scr=SCR):
    r = None if rows is None else (C.c_uint64 * len(rows))(*rows)
    c = None if coef is None else (C.c_float * 3)(*coef)
    return L.lib.lct_list_orthogonalize(x.ref, r, y.ref, steps, c, None, ptr(scr), None)


def test_orthogonalize_refusals(L):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a device")
    ok = L.EARCH, L.EHIP
    x = FakeList(L, [600, 0, 35], [A, 0, B], [L.FP32, L.BF16, L.FP16])
    y = FakeList(L, [600, 0, 35], [D, 0, E], [L.BF16] * 3)
    rows = [20, 0, 5]
    assert ortho(L, x, rows, y) in ok
    assert ortho(L, x, None, y) == ortho(L, x, rows, y, coef=None) == ortho(L, x, rows, y, scr=None) == L.EINVAL
    assert ortho(L, x, [20, 0, 0], y) == ortho(L, x, [7, 0, 5], y) == L.EINVAL          # no rows, or not whole ones
    assert ortho(L, x, rows, y, steps=0) == ortho(L, x, rows, y, steps=33) == L.EINVAL
    assert ortho(L, x, rows, FakeList(L, [600, 0, 35], [D, 0, E], [L.BF16, L.BF16, L.FP32])) == L.EINVAL
    assert ortho(L, x, rows, FakeList(L, [600, 1, 35], [D, A, E], [L.BF16] * 3)) == L.EINVAL
    long = FakeList(L, [1 << 23], [A], [L.BF16])
    assert ortho(L, long, [1], FakeList(L, [1 << 23], [D], [L.BF16])) == L.EINVAL       # a side past 2^22
    assert ortho(L, x, rows, y, scr=SCR + 128) == L.EALIGN
    assert ortho(L, x, rows, FakeList(L, [600, 0, 35], [D, 0, D + 100], [L.BF16] * 3)) == L.EALIAS
    assert ortho(L, x, rows, FakeList(L, [600, 0, 35], [A, 0, E], [L.BF16] * 3)) == L.EALIAS   # FP32 memory as BF16
    assert ortho(L, x, rows, y, scr=D) == ortho(L, x, rows, y, scr=A) == L.EALIAS
    b = FakeList(L, [600], [A], [L.BF16])
    assert ortho(L, b, [20], b) in ok                                                   # in place


def test_orthogonalize_coefficients(L):
    """Those whose iterates leave the range that the kernels hold are refused."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses stay off a device")
    x, y = FakeList(L, [600], [A], [L.BF16]), FakeList(L, [600], [D], [L.BF16])
    for coef in ((3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (0.0, 0.0, 0.0)):
        assert ortho(L, x, [20], y, coef=coef, steps=32) in (L.EARCH, L.EHIP), coef
    for coef in ((NAN, 0, 0), (1, INF, 0), (2.5, 0, 0), (-3, 0, 0), (1, 0, 2), (1, -9, 8), (5, -4, 0)):
        assert ortho(L, x, [20], y, coef=coef) == L.EINVAL, coef
    # the last result is not held in FP16: one step may go further
    assert ortho(L, x, [20], y, coef=(2.5, 0, 0), steps=1) in (L.EARCH, L.EHIP)


def test_orthogonal_scratch(L):
    def need(ns, rows):
        x = FakeList(L, ns, [A + (k << 40) for k in range(len(ns))], [L.BF16] * len(ns))
        out = C.c_uint64(0)
        assert L.lib.lct_orthogonal_scratch(x.ref, (C.c_uint64 * len(ns))(*rows), C.byref(out)) == L.OK
        return out.value

    one = need([2560 * 9728], [2560])
    assert 8 * 2560 * 9728 <= one <= 12 * 2560 * 9728 + (1 << 20)
    assert need([2560 * 9728], [9728]) == one
    # a long list is done in batches: its memory stops growing
    assert need([2560 * 9728] * 40, [2560] * 40) < 7 * one
    assert need([], []) >= 256


def test_matrices_check_their_tensors(L):
    with pytest.raises(ValueError, match="dimensions"):
        L.LctMatrices([torch.zeros(5)])
    with pytest.raises(ValueError, match="GPU"):
        L.LctMatrices([torch.zeros(5, 4)])
    with pytest.raises(ValueError, match="contiguous"):
        L.LctMatrices([torch.zeros(2, 5, 4).transpose(1, 2)])
