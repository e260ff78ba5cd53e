"""Host-side checks of the norms, the clip and the clipped steps (no GPU): the
structs match the header, scratch sizes, every refusal of the C calls before
anything reaches a device (addresses are made up), and the Python lists'
checks of their tensors."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import synth
from test_boundary_host import HEADER, _fake_tensor

INF = float("inf")
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    import lossless_bf16_tensor_split_amd as L
    return L


def test_struct_layouts_match_header(L, tmp_path):
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "lct.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu %zu %zu\\n", sizeof(lct_list), offsetof(lct_list, n),'
                   'offsetof(lct_list, d_x), offsetof(lct_list, type), sizeof(lct_norm_t),'
                   'offsetof(lct_norm_t, norm), offsetof(lct_norm_t, coef));return 0;}\n')
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I" + os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [C.sizeof(L._List), L._List.n.offset, L._List.d_x.offset, L._List.type.offset, 16, 8, 12]


def scratch(L, count, nblk):
    out = C.c_uint64(0)
    assert L.lib.lct_norm_scratch(count, nblk, C.byref(out)) == L.OK
    return out.value


def test_scratch_grows_with_tensors_and_blocks(L):
    sizes = [scratch(L, c, 0) for c in (0, 1, 192, 193, 400, 20000)]
    assert sizes == sorted(sizes) and sizes[3] > sizes[2]
    assert scratch(L, 1, 0) <= 1 << 16
    assert scratch(L, 0, 100000) >= 8 * 100000
    assert scratch(L, 400, 100000) >= max(scratch(L, 400, 0), scratch(L, 0, 100000))
    assert scratch(L, 0, 0xFFFFFFFF) >= 8 * 0xFFFFFFFF
    assert L.lib.lct_norm_scratch(1, 1 << 32, C.byref(C.c_uint64())) == L.EINVAL
    assert L.lib.lct_norm_scratch(1, 1, None) == L.EINVAL
    assert L.lib.lct_norm_scratch((1 << 24) + 1, 0, C.byref(C.c_uint64())) == L.EINVAL


class FakeList:
    """A C list over made-up device addresses."""

    def __init__(self, L, ns, ptrs, types):
        self.a = (C.c_uint64 * len(ns))(*ns)
        self.b = (C.c_void_p * len(ns))(*ptrs)
        self.c = (C.c_int32 * len(ns))(*types)
        self.s = L._List(len(ns), C.cast(self.a, C.c_void_p), C.cast(self.b, C.c_void_p), C.cast(self.c, C.c_void_p))

    @property
    def ref(self):
        return C.byref(self.s)


A, B, D = 0x1000_0000_0000, 0x2000_0000_0000, 0x3000_0000_0000
SCR, EACH, OUT = 0x6000_0000_0000, 0x7000_0000_0000, 0x7100_0000_0000


def test_list_norm_refusals(L):
    good = FakeList(L, [100, 0, 5], [A, 0, B + 2], [L.BF16, L.FP32, L.FP16])

    def call(x=None, kind=0, mx=1.0, sc=1.0, scr=SCR, each=EACH, out=OUT):
        x = good if x is None else x
        return L.lib.lct_list_norm(x.ref, kind, mx, sc, C.c_void_p(scr), C.c_void_p(each), C.c_void_p(out), None)

    assert L.lib.lct_list_norm(None, 0, 1.0, 1.0, C.c_void_p(SCR), None, C.c_void_p(OUT), None) == L.EINVAL
    bad = L._List(2, None, None, None)
    assert L.lib.lct_list_norm(C.byref(bad), 0, 1.0, 1.0, C.c_void_p(SCR), None, C.c_void_p(OUT), None) == L.EINVAL
    for kw in ({"kind": 2}, {"kind": -1}, {"mx": -1.0}, {"mx": NAN}, {"sc": NAN}, {"sc": INF}, {"sc": -INF},
               {"scr": 0}, {"out": 0}):
        assert call(**kw) == L.EINVAL, kw
    for kw in ({"scr": SCR + 128}, {"each": EACH + 2}, {"out": OUT + 4}):
        assert call(**kw) == L.EALIGN, kw
    # element types, null pointers, sizes, alignment of the elements
    assert call(FakeList(L, [4], [A], [3])) == L.EINVAL
    assert call(FakeList(L, [4], [A], [-1])) == L.EINVAL
    assert call(FakeList(L, [4], [0], [0])) == L.EINVAL
    assert call(FakeList(L, [(1 << 44) + 1], [A], [0])) == L.EINVAL
    assert call(FakeList(L, [1 << 43, 1 << 43, 1], [A, A, A], [0, 0, 0])) == L.EINVAL
    assert call(FakeList(L, [(1 << 64) - 1, 1], [A, A], [0, 0])) == L.EINVAL
    many = FakeList(L, [4], [A], [0])
    for count in ((1 << 24) + 1, 0xFFFFFFFF):
        many.s.count = count                 # refused before its arrays are read
        assert call(many) == L.EINVAL
    assert call(FakeList(L, [4], [A + 1], [L.BF16])) == L.EALIGN
    assert call(FakeList(L, [4], [A + 2], [L.FP32])) == L.EALIGN
    # outputs and scratch on an input or each other
    for kw in ({"scr": A}, {"each": A + 196}, {"out": A + 192}, {"out": SCR + 8}, {"each": SCR + 64},
               {"each": OUT + 8}):
        assert call(**kw) == L.EALIAS, kw
    x = FakeList(L, [4], [SCR + scratch(L, 1, 0) - 2], [L.BF16])
    assert call(x) == L.EALIAS


def test_code_norm_refusals(L):
    lay = L.layout(65536, 25)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None)
    n = 100000
    t = _fake_tensor(L, n, lay, A)

    def call(cb_=cb, t_=t, kind=0, mx=1.0, sc=1.0, scr=SCR, out=OUT):
        return L.lib.lct_tensor_norm(C.byref(cb_), C.byref(t_), kind, mx, sc, C.c_void_p(scr), C.c_void_p(out), None)

    assert call(cb_=L.Codebook()) == L.EINVAL
    for kw in ({"kind": 5}, {"mx": -0.5}, {"mx": NAN}, {"sc": INF}, {"scr": 0}, {"out": 0}):
        assert call(**kw) == L.EINVAL, kw
    for kw in ({"scr": SCR + 8}, {"out": OUT + 4}):
        assert call(**kw) == L.EALIGN, kw
    for kw in ({"scr": t.pay & ~255}, {"out": t.sf}, {"out": t.obase}, {"out": SCR}):
        assert call(**kw) == L.EALIAS, kw
    bad = _fake_tensor(L, n, lay, A, sf=A + 8)
    assert call(t_=bad) == L.EALIGN
    bad = _fake_tensor(L, n, lay, A)
    bad.layout = L.layout(4096, 0)
    assert call(t_=bad) == L.EINVAL
    bad = _fake_tensor(L, n, lay, A)
    bad.n = 1 << 52
    assert call(t_=bad) == L.EINVAL
    # groups: never bound, and storage of other sizes
    g = L.Group()
    assert L.lib.lct_group_norm(C.byref(g), C.byref(t), 0, 1.0, 1.0, C.c_void_p(SCR), None, C.c_void_p(OUT),
                                None) == L.EINVAL
    assert L.lib.lct_group_norm(None, C.byref(t), 0, 1.0, 1.0, C.c_void_p(SCR), None, C.c_void_p(OUT),
                                None) == L.EINVAL


def test_norm_join_refusals(L):
    def call(parts=A, count=2, kind=0, mx=1.0, sc=1.0, out=OUT):
        return L.lib.lct_norm_join(C.c_void_p(parts), count, kind, mx, sc, C.c_void_p(out), None)

    for kw in ({"parts": 0}, {"kind": 2}, {"mx": NAN}, {"mx": -1.0}, {"sc": NAN}, {"out": 0}):
        assert call(**kw) == L.EINVAL, kw
    for kw in ({"parts": A + 4}, {"out": OUT + 4}):
        assert call(**kw) == L.EALIGN, kw


def test_clip_refusals(L):
    ns = [100, 0, 8]
    x = FakeList(L, ns, [A, 0, B], [L.FP32, L.BF16, L.BF16])
    y = FakeList(L, ns, [D, 0, D + 4096], [L.BF16, L.BF16, L.BF16])

    def call(x_=x, y_=y, coef=OUT):
        return L.lib.lct_list_clip(x_.ref, C.c_void_p(coef), y_.ref, None)

    assert call(coef=0) == L.EINVAL
    assert call(coef=OUT + 2) == L.EALIGN
    assert L.lib.lct_list_clip(x.ref, C.c_void_p(OUT), None, None) == L.EINVAL
    assert L.lib.lct_list_clip(None, C.c_void_p(OUT), y.ref, None) == L.EINVAL
    # sizes that differ
    assert call(y_=FakeList(L, [100, 0], [D, 0], [0, 0])) == L.EINVAL
    assert call(y_=FakeList(L, [100, 0, 9], [D, 0, D + 4096], [0, 0, 0])) == L.EINVAL
    # outputs on each other, on another input, shifted on their own input, in
    # place with another type, on the coefficient
    assert call(y_=FakeList(L, ns, [D, 0, D + 196], [0, 0, 0])) == L.EALIAS
    assert call(y_=FakeList(L, ns, [D, 0, A + 40], [0, 0, 0])) == L.EALIAS
    assert call(y_=FakeList(L, ns, [D, 0, B + 2], [0, 0, 0])) == L.EALIAS
    assert call(y_=FakeList(L, ns, [A, 0, D], [0, 0, 0])) == L.EALIAS
    assert call(coef=D + 16) == L.EALIAS
    # one tensor twice in place (it would be scaled twice, in no order)
    twice = FakeList(L, [8, 8], [A, A], [0, 0])
    assert call(twice, twice) == L.EALIAS
    # an input within another one's output span
    assert call(FakeList(L, [1000, 4], [A, D + 100], [0, 0]), FakeList(L, [1000, 4], [D, B], [0, 0])) == L.EALIAS


def test_clipped_steps_refusals(L):
    lay = L.layout(65536, 25)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None)
    n = 100000
    w, m = _fake_tensor(L, n, lay, A), _fake_tensor(L, n, lay, B)
    ow, om = _fake_tensor(L, n, lay, D), _fake_tensor(L, n, lay, 0x4000_0000_0000)
    g = C.c_void_p(0x5000_0000_0000)
    eta, mu = C.c_float(1e-3), C.c_float(0.9)

    def sgd(coef, m_=m, ow_=ow):
        return L.lib.lct_sgd_step_clip(C.byref(cb), C.byref(w), C.byref(cb), C.byref(m_), eta, C.c_void_p(coef),
                                       C.byref(ow_), None)

    def mom(coef, g_=g, ow_=ow, om_=om):
        return L.lib.lct_momentum_step_clip(C.byref(cb), C.byref(w), C.byref(cb), C.byref(m), g_, C.c_void_p(coef),
                                            mu, eta, C.byref(ow_), C.byref(om_), None)

    assert sgd(0) == L.EINVAL and mom(0) == L.EINVAL
    assert sgd(OUT + 2) == L.EALIGN and mom(OUT + 1) == L.EALIGN
    for p in (ow.sf + 16, ow.status, ow.scratch + 8, ow.obase):
        assert sgd(p) == L.EALIAS and mom(p) == L.EALIAS
    for p in (om.pay, om.status, om.ovf):
        assert mom(p) == L.EALIAS
    # the rules of the calls they clip still hold
    bad = _fake_tensor(L, n, lay, D, ovf=w.ovf)
    assert sgd(OUT, ow_=bad) == L.EALIAS and mom(OUT, ow_=bad) == L.EALIAS
    assert mom(OUT, g_=C.c_void_p(om.pay)) == L.EALIAS
    m2 = _fake_tensor(L, n + 1, lay, B)
    assert sgd(OUT, m_=m2) == L.EINVAL
    # groups
    z = L.Group()
    assert L.lib.lct_sgd_step_clip_group(C.byref(z), C.byref(w), C.byref(z), C.byref(m), eta, None, C.byref(ow),
                                         None) == L.EINVAL
    assert L.lib.lct_momentum_step_clip_group(C.byref(z), C.byref(w), C.byref(z), C.byref(m), C.byref(z), None, mu,
                                              eta, C.byref(ow), C.byref(om), None) == L.EINVAL


def test_python_lists_check_their_tensors(L):
    with pytest.raises(TypeError, match="tensor 0"):
        L.LctList([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(TypeError, match="tensor 1"):
        L.LctList([_cuda_like(torch.float32), torch.zeros(4, dtype=torch.int16)])
    with pytest.raises(ValueError, match="on the GPU"):
        L.LctList([torch.zeros(4)])
    with pytest.raises(ValueError, match="contiguous"):
        L.LctList([torch.zeros(4, 4).t()])
    assert len(L.LctList([])) == 0
    with pytest.raises(TypeError):
        L._coef(1.0)
    with pytest.raises(TypeError):
        L._coef(torch.zeros(2))
    with pytest.raises(TypeError):
        L._coef(torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError, match="on the GPU"):
        L._coef(torch.zeros(1))
    with pytest.raises(ValueError, match="on the GPU"):
        L._current(torch.device("cpu"), "x")


class _cuda_like:
    """As much of a tensor as a list's checks look at before the next one."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, dtype):
        self.dtype = dtype

    def is_contiguous(self):
        return True


def test_lists_of_two_devices_are_refused(L):
    a, b = _cuda_like(torch.float32), _cuda_like(torch.bfloat16)
    b.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="tensor 1 is on cuda:1"):
        L.LctList([a, b])


def test_another_device_than_the_current_one_is_refused(L, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        L._current(torch.device("cuda", 0), "x")
    L._current(torch.device("cuda", 1), "x")


def test_oracle_clipped_momentum(orc):
    """With c = 1 the clipped step is the plain one; with another c it is the
    definition, evaluated with more bits: mu * m and c * g are exact in 64
    bits' 53 (16 and 32 significant bits), their sum in the 64 of a long
    double where the exponents are near."""
    g = np.random.default_rng(3)
    n = 4000
    w, m, gr = (synth.to_bf16_bits(g.normal(0, s, n)) for s in (0.02, 1e-3, 1e-3))
    sp = [0x7FC0, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x7F7F]
    w[:6], m[20:26], gr[40:46] = sp, sp, sp
    a = orc.momentum_clip_dense(w, m, gr, 1.0, 0.9, 0.1)
    b = orc.momentum_dense(w, m, gr, 0.9, 0.1)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    c, mu, eta = np.float32(0.37), np.float32(0.9), np.float32(0.1)
    wo, mo = orc.momentum_clip_dense(w, m, gr, float(c), float(mu), float(eta))

    def f(x):
        return (x.astype(np.uint32) << 16).view(np.float32)

    keep = slice(50, n)
    cg = c * f(gr[keep])
    want = (np.longdouble(mu) * f(m[keep]).astype(np.longdouble) + cg.astype(np.longdouble)).astype(np.float32)
    assert np.array_equal(synth.to_bf16_bits(want), mo[keep])
    want = (np.longdouble(-eta) * f(mo[keep]).astype(np.longdouble) + f(w[keep]).astype(np.longdouble))
    assert np.array_equal(synth.to_bf16_bits(want.astype(np.float32)), wo[keep])
