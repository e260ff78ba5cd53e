"""The mix of a compressed tensor with a dense one on the GPU: every byte of the
codes against the oracle's encoding of the mixed values, and the dense results
bit for bit.  The reference is the oracle's clipped momentum, y' = rne(fmaf(a, y,
c * x)) in C's fmaf, with c = b * coef rounded to fp32; looked ahead, the same
formula applied to y'."""
import numpy as np
import pytest
import torch

import synth
from test_gpu_parity import assert_same, check_codebook, dev, host_parts

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def values(n, seed, specials=True):
    g = np.random.default_rng(seed)
    y = synth.to_bf16_bits(g.normal(0, 1e-2, n))
    x = synth.to_bf16_bits(g.normal(0, 0.1, n))
    if specials and n > 400:
        sp = [0x7FC0, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x8001, 0x7F7F, 0xFF7F]
        y[:64] = sp * 8
        x[100:164] = sp * 8
        x[8:16] = sp[::-1]
    return y, x


def mixed(orc, y, x, a, b, c):
    """(y', looked ahead) as BF16 bits."""
    bc = float(np.float32(b) * np.float32(c))
    zero = np.zeros_like(y)
    _, v = orc.momentum_clip_dense(zero, y, x, bc, a, 0.0)
    _, u = orc.momentum_clip_dense(zero, v, x, bc, a, 0.0)
    return v, u


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def take_over(o, t):
    o.sf, o.pay, o.cnt, o.obase = t.sf, t.pay, t.cnt, t.obase


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 1), (8192, 3), (32768, 12), (32768, 11)])
def test_mix_equals_the_oracle(L, orc, B, cw, inplace):
    """Full and partial blocks, with spills where the capacity is small."""
    n = 2 * B + 531
    y, x = values(n, B + cw)
    lay = L.layout(B, cw)
    cb, ocb = check_codebook(L, orc, synth.Model(0, 1e-2), y)
    for a, b, c, kind in ((0.9, 1.0, 0.3701, "value"), (0.95, 1.0, None, "ahead"), (0.999, -0.02, 1.0, None),
                          (1.0, 0.0, None, "value"), (0.0, 1.0, NAN, None), (INF, -1.0, 1.0, "ahead")):
        t, o = L.encode(cb, dev(y), lay), L.alloc_tensor(n, lay)
        if inplace:
            take_over(o, t)
        xd = dev(x)
        d = torch.full((n,), 0x5555, dtype=torch.int16, device="cuda") if kind else None
        coef = None if c is None else torch.tensor(c, device="cuda")
        L.lct_mix_step(cb, t, a, xd, b, o, coef, d, kind == "ahead")
        v, u = mixed(orc, y, x, a, b, 1.0 if c is None else c)
        assert_same(host_parts(o), orc.encode(ocb, v, B, cw), "y' a=%s b=%s c=%s" % (a, b, c))
        if kind:
            assert np.array_equal(bits(d), u if kind == "ahead" else v)
        assert np.array_equal(bits(xd), x)


@pytest.mark.parametrize("n", [1, 2, 255, 256, 257, 4095, 4096, 4097, 65535, 65536, 65537, 200_000])
def test_mix_sizes(L, orc, n):
    """Blocks of every kind of length; the dense result over x itself."""
    y, x = values(n, n)
    lay = L.lct_layout_init(L.CLEAN)
    cb, ocb = check_codebook(L, orc, synth.Model(0, 1e-2), y)
    t, o = L.encode(cb, dev(y), lay), L.alloc_tensor(n, lay)
    xd = dev(x)
    L.lct_mix_step(cb, t, 0.95, xd, 1.0, o, dense=xd, ahead=True)
    v, u = mixed(orc, y, x, 0.95, 1.0, 1.0)
    assert_same(host_parts(o), orc.encode(ocb, v, lay.block_elems, lay.cap_words))
    assert np.array_equal(bits(xd), u)
    assert np.array_equal(bits(L.decode(cb, o)), v)


def test_mix_moves_to_another_codebook(L, orc):
    """A tensor that has grown by 2^6 goes onto a shifted codebook."""
    n = 70_000
    y, x = values(n, 5, specials=False)
    lay = L.lct_layout_init(L.CLEAN)
    cb, ocb = check_codebook(L, orc, synth.Model(0, 1e-2), y)
    v, _ = mixed(orc, y, x, 64.0, 0.5, 1.0)
    new = L.lct_codebook_reshift_dense(cb, dev(v))
    assert new.shift == cb.shift + 6
    onew = orc.codebook_from_base(np.frombuffer(bytes(cb.len_base), np.uint8), cb.esc_len, new.shift)
    t, o = L.encode(cb, dev(y), lay), L.alloc_tensor(n, lay)
    L.lct_mix_step(cb, t, 64.0, dev(x), 0.5, o, cb_out=new)
    assert_same(host_parts(o), orc.encode(onew, v, lay.block_elems, lay.cap_words))


def test_mix_overflow_is_reported(L, orc):
    """A region too small for the spill: the status word, the size needed and
    the dense result, which does not depend on it."""
    n, B, cw = 3 * 4096 + 7, 4096, 1
    y, x = values(n, 3)
    lay = L.layout(B, cw)
    cb, ocb = check_codebook(L, orc, synth.Model(0, 1e-2), y)
    t, o = L.encode(cb, dev(y), lay), L.alloc_tensor(n, lay, 100)
    o.ovf = torch.full((4096,), 0x77, dtype=torch.uint8, device="cuda")
    d = torch.zeros(n, dtype=torch.int16, device="cuda")
    L.lct_mix_step(cb, t, 0.9, dev(x), 1.0, o, dense=d)
    v, _ = mixed(orc, y, x, 0.9, 1.0, 1.0)
    ref = orc.encode(ocb, v, B, cw)
    assert o.status_word() == L.ST_OVF_FULL
    assert int(o.obase[-1]) == ref.spilled > 100
    assert bool((o.ovf[100:] == 0x77).all())
    assert np.array_equal(bits(d), v)


GROUP_NS = [2 * 65536, 65536 + 17, 5, 0, 70_001, 256]


@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 2), (32768, 12)])
def test_group_mix_equals_single_ones(L, orc, B, cw):
    lay = L.layout(B, cw)
    src = [values(n, 40 + k, specials=k == 0) for k, n in enumerate(GROUP_NS)]
    ys, xs = [dev(y) if y.size else dev(np.zeros(1, np.uint16))[:0] for y, _ in src], None
    xs = [dev(x) if x.size else dev(np.zeros(1, np.uint16))[:0] for _, x in src]
    models = [L.Model(0, 1e-2 * 2.0 ** (k % 2), 0.0) for k in range(len(src))]
    cbs = [L.lct_codebook_build(m, y if y.numel() else None) for m, y in zip(models, ys)]
    ds = [torch.zeros(max(n, 8), dtype=torch.int16, device="cuda") for n in GROUP_NS]
    ys = [y if y.numel() else torch.zeros(8, dtype=torch.int16, device="cuda") for y in ys]
    xs = [x if x.numel() else torch.zeros(8, dtype=torch.int16, device="cuda") for x in xs]
    g, gx, gd = (L.LctGroup(GROUP_NS, lay, cbs, d) for d in (ys, xs, ds))
    cap = sum(GROUP_NS) + len(GROUP_NS) * B
    coef = torch.tensor(0.61, device="cuda")
    for dense, ahead in ((None, False), (gd, False), (gd, True), (gx, True)):
        xs_before = [x.clone() for x in xs]
        for inplace in (False, True):
            for x, was in zip(xs, xs_before):
                x.copy_(was)
            st = g.alloc_storage(cap)
            L.lct_encode_group(g, st)
            out = g.alloc_storage(cap)
            if inplace:
                take_over(out, st)
            L.lct_mix_step_group(g, st, 0.9, gx, 1.0, out, coef, dense, ahead)
            for k, (y, x) in enumerate(src):
                if not y.size:
                    continue
                v, u = mixed(orc, y, x, 0.9, 1.0, 0.61)
                assert np.array_equal(bits(L.decode(cbs[k], g.tensor(out, k))), v), (k, inplace)
                if dense is not None:
                    got = bits((xs if dense is gx else ds)[k])[:y.size]
                    assert np.array_equal(got, u if ahead else v), (k, inplace, ahead)
        for x, was in zip(xs, xs_before):
            x.copy_(was)


def test_mix_on_a_side_stream_and_from_a_graph(L):
    """The same bytes on another stream and from every replay of a graph whose
    inputs change, with other work between the replays."""
    lay = L.lct_layout_init(L.CLEAN)
    n = 3 * 65536 + 999
    y = (torch.randn(n, device="cuda") * 1e-2).bfloat16()
    cb = L.lct_codebook_build(L.Model(0, 1e-2, 0.0), y)
    t, o = L.encode(cb, y, lay), L.alloc_tensor(n, lay)
    x, d, coef = torch.empty_like(y), torch.empty_like(y), torch.empty((), device="cuda")

    def fill(seed):
        torch.manual_seed(seed)
        x.copy_(torch.randn(n, device="cuda") * 0.1)
        coef.fill_(0.1 * seed)

    def run(stream=None):
        L.lct_mix_step(cb, t, 0.9, x, 1.0, o, coef, d, True, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [b.clone() for b in (o.sf, o.pay, o.cnt, o.obase, o.status, d)]

    fill(1)
    run()
    want = results()
    d.zero_()
    o.pay.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(4):
        fill(2 + rep)
        run()
        want = results()
        d.zero_()
        o.pay.zero_()
        o.sf.zero_()
        L.decode(cb, t)
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, results())), rep
