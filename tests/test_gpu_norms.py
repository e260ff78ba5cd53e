"""Norms of dense lists and of compressed tensors, the clip and the clipped
steps on the GPU, against plain forms in 64 bits and the oracle's bytes.

Tolerances.  S is summed in 64 bits: a path of additions is at most n long, so
it is off by at most (n + 64) * 2^-53 of itself (all terms are positive).  The
square root halves that; the few operations after it add 2^-51 at most; norm
and coef are rounded to fp32 once (2^-24, or half of fp32's smallest step).
Of compressed tensors, 16 squares are summed in fp32 before the sum goes on in
64 bits: the first square is exact (16 significant bits), each of the 15 fused
multiply-adds after it is off by half a step (2^-24) of a partial sum that is
at most the whole, all terms being positive, so S is off by 15 * 2^-24 more and
the norm and the coefficient by half of that.
Largest magnitudes are exact up to that one rounding.  Scaled values are
compared bit for bit with fp32 products rounded to the output's type."""
import numpy as np
import pytest
import torch

import synth
from test_gpu_parity import assert_same, check_codebook, dev, host_parts

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def f64(x):
    """A tensor's values in float64 on the host."""
    return x.detach().cpu().double().numpy().reshape(-1)


def want(values, kind, max_norm, scale):
    """(S, norm, coef) in 64 bits of the concatenated values, S summed in the
    long double's 64-bit significand."""
    v = np.concatenate([np.zeros(1)] + list(values))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if kind == "l2":
            S = float(np.sum(v.astype(np.longdouble) ** 2))
            N = abs(scale) * np.sqrt(np.float64(S))
        else:
            S = float(np.max(np.abs(v)))
            N = np.float64(abs(scale) * S)
        q = np.float64(max_norm) / (N + 1e-6)
        c = scale * (1.0 if q >= 1.0 else q)
    return S, float(N), float(c)


CODES = 15 * 2.0 ** -24      # what fp32 sums of 16 squares add to S's relative error


def close32(got, ref, n, what="", more=0.0):
    """got (a float32 value) is ref to one fp32 rounding and S's error (more:
    beyond that of its sum in 64 bits)."""
    got = float(got)
    if np.isnan(ref):
        assert np.isnan(got), what
        return
    with np.errstate(over="ignore"):
        r32 = float(np.float32(ref))
    if np.isinf(r32):
        assert got == r32, what
        return
    tol = abs(ref) * (2.0 ** -24 + (n + 64) * 2.0 ** -54 + 2.0 ** -51 + more / 2) + 2.0 ** -150
    assert abs(got - ref) <= tol, "%s: %r for %r" % (what, got, ref)


def check_norm(out, values, kind, max_norm, scale, what="", more=0.0):
    torch.cuda.synchronize()
    n = sum(len(v) for v in values)
    S, N, c = want(values, kind, max_norm, scale)
    s = float(out.sum)
    if np.isnan(S):
        assert np.isnan(s), what
    elif kind == "max" or np.isinf(S) or S == 0:
        assert s == S, what
    else:
        assert abs(s - S) <= S * ((n + 64) * 2.0 ** -53 + more), what
    close32(out.norm, N, n, what + " norm", more)
    close32(out.coef, c, n, what + " coef", more)
    if out.each is not None:
        got = out.each.cpu().numpy()
        assert len(got) == len(values)
        for k, v in enumerate(values):
            close32(got[k], want([v], kind, max_norm, scale)[1], len(v), "%s each[%d]" % (what, k), more)


def kind_of(L, kind):
    return L.NORM_L2 if kind == "l2" else L.NORM_MAX


def list_norm(L, xs, kind="l2", max_norm=1.0, scale=1.0, each=True, what=""):
    lst = L.LctList(xs)
    out = L.alloc_norm(len(xs), each)
    out.scratch.fill_(0xFF)          # NaN where nothing was written
    L.lct_list_norm(lst, out, max_norm, scale, kind_of(L, kind))
    check_norm(out, [f64(x) for x in xs], kind, max_norm, scale, what)
    return out


EDGES = [0, 1, 2, 3, 7, 8, 9, 15, 17, 255, 257, 2047, 2048, 2049, 16383, 16384, 16385, 3 * 16384 + 5, 100003]


def views(ns, dtype, seed, shift=0, sigma=1e-3, device="cuda"):
    """Tensors of ns elements back to back in one buffer that starts `shift`
    elements in, with guard values around."""
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(sum(ns) + shift + 8, generator=g) * sigma).to(dtype).to(device)
    out, at = [], shift
    for n in ns:
        out.append(flat[at:at + n])
        at += n
    return flat, out


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_list_norm_sizes_and_alignments(L, dtype, kind):
    """Every edge of the vector, the chunk and the workgroup, tensors back to
    back at every alignment of an element; all together and one by one."""
    sigma = 0.5 if dtype == HF else 1e-3
    for shift in (0, 1, 3):
        _, xs = views(EDGES, dtype, 11 + shift, shift, sigma)
        list_norm(L, xs, kind, 0.25, 0.5, True, "all shift %d" % shift)
        list_norm(L, xs, kind, 0.25, 0.5, False, "no each, shift %d" % shift)
    for n in EDGES:
        _, xs = views([n], dtype, n, 1, sigma)
        list_norm(L, xs, kind, 10.0, 1.0, n % 2 == 0, "one of %d" % n)


def test_list_norm_mixed_types_and_many_tensors(L):
    """More tensors than a launch takes, of three types, empty ones among
    them; more chunks than workgroups."""
    r = np.random.default_rng(5)
    xs = []
    for k in range(451):
        n = int(r.choice([0, 1, 128, 1000, 2560, 20011]))
        dt = [BF, HF, SF][k % 3]
        xs.append((torch.randn(n, generator=torch.Generator().manual_seed(k)) * 0.1).to(dt).cuda())
    list_norm(L, xs, "l2", 1.0, 0.125, True, "451 tensors")
    list_norm(L, xs, "max", 1.0, -0.125, True, "451 tensors, negative scale")
    # 2048 workgroups take runs of several chunks; tensor ends inside runs
    ns = [30_000_001, 5, 16384 * 100, 40_000_000 - 3]
    big = [(torch.randn(n, device="cuda") * 1e-2).to(BF) for n in ns]
    list_norm(L, big, "l2", 1.0, 1.0, True, "71M elements")
    list_norm(L, big, "max", 1.0, 1.0, False, "71M elements")


def test_list_norm_values_out_of_the_ordinary(L):
    """Zeros, infinities, NaNs, the largest and the subnormal values: squares
    that 32 bits cannot hold keep their sum, and the norm and coefficient
    follow their formulas."""
    fmax, tiny = 3.4028234663852886e38, 1e-45
    cases = [([0.0, -0.0], SF), ([fmax] * 100, SF), ([fmax] * 100, BF), ([tiny] * 77, SF), ([1e-40, 1e-30], SF),
             ([6e-8] * 9, HF), ([65504.0] * 33, HF), ([1e-40] * 50, BF), ([1e20, 1e-20], BF),
             ([INF, 1.0], BF), ([-INF, 1.0], HF), ([INF, NAN], SF), ([NAN], BF), ([NAN, 5.0], HF)]
    for i, (v, dt) in enumerate(cases):
        x = torch.tensor(v, dtype=torch.float64).to(dt).cuda()
        y = torch.ones(20000, dtype=SF, device="cuda")
        for kind in ("l2", "max"):
            for mx in (1.0, 0.0, INF):
                list_norm(L, [x], kind, mx, 1.0, True, "case %d max_norm %s" % (i, mx))
            list_norm(L, [y, x, y], kind, 1.0, 1.0, True, "case %d between others" % i)
    # a negative NaN with a payload is not lost by the maximum
    x = torch.tensor([0xFFC1 - 65536, 0x3F80], dtype=torch.int16, device="cuda").view(BF)
    list_norm(L, [x], "max", 1.0, 1.0, True, "negative NaN")


def test_list_norm_empty_sets_and_repeated_tensors(L):
    for xs in ([], [torch.empty(0, device="cuda")], [torch.empty(0, dtype=BF, device="cuda")] * 200):
        for kind in ("l2", "max"):
            out = list_norm(L, xs, kind, 2.0, 0.5, True, "%d empty tensors" % len(xs))
            assert float(out.norm) == 0.0 and float(out.coef) == 0.5
    x = torch.randn(5000, device="cuda")
    list_norm(L, [x, x, x[:100]], "l2", 1.0, 1.0, True, "a tensor listed twice")


def test_list_norm_repeats_bit_for_bit(L):
    xs = [(torch.randn(n, device="cuda") * 1e-3).to(BF) for n in (5_000_003, 77, 1_000_000)]
    lst = L.LctList(xs)
    a, b, c = L.alloc_norm(3, True), L.alloc_norm(3, True), L.alloc_norm(3, False)
    L.lct_list_norm(lst, a)
    for _ in range(3):
        b.buf.fill_(7)
        L.lct_list_norm(lst, b)
        torch.cuda.synchronize()
        assert torch.equal(a.buf, b.buf) and torch.equal(a.each, b.each)
    # with and without the tensors' own norms: the same sum but for its order
    L.lct_list_norm(lst, c)
    check_norm(c, [f64(x) for x in xs], "l2", INF, 1.0)


def test_norm_result_is_checked_for_size_and_place(L):
    xs = L.LctList([torch.randn(100, device="cuda")] * 3)
    out = L.alloc_norm(3, True)
    with pytest.raises(ValueError, match="each"):
        L.lct_list_norm(xs, L.alloc_norm(2, True))
    out.scratch = out.scratch[:64]
    with pytest.raises(ValueError, match="scratch"):
        L.lct_list_norm(xs, out)
    out = L.alloc_norm(3)
    with pytest.raises(ValueError, match="on the GPU"):
        out.scratch = out.scratch.cpu()
    with pytest.raises(ValueError, match="contiguous"):
        out.scratch = out.scratch[::2]
    out = L.alloc_norm(3)
    for kw in ({"max_norm": -1.0}, {"max_norm": NAN}, {"scale": INF}, {"kind": 3}):
        with pytest.raises(L.LctError):
            L.lct_list_norm(xs, out, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        L.LctList([torch.randn(8, 8, device="cuda").t()])


# ------------------------------------------------------------------ join

@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm_join(L, kind):
    """Results of several sets joined, as ranks do after gathering them."""
    sets = [[torch.randn(n, device="cuda") * s for n in ns]
            for ns, s in (((1000, 3), 1.0), ((0,), 1.0), ((70000,), 1e-3), ((5, 5, 5), 30.0))]
    parts = [list_norm(L, xs, kind, 1.0, 1.0, False) for xs in sets]
    out = L.alloc_norm()
    L.lct_norm_join(parts, out, 2.0, 0.25, kind_of(L, kind))
    every = [f64(x) for xs in sets for x in xs]
    check_norm(out, every, kind, 2.0, 0.25, "joined")
    gathered = torch.stack([p.buf for p in parts])
    L.lct_norm_join(gathered, parts[0], 2.0, 0.25, kind_of(L, kind))
    torch.cuda.synchronize()
    assert torch.equal(parts[0].buf, out.buf)
    # in place of a part, and of one part alone
    L.lct_norm_join([out], out, 0.125, 1.0, kind_of(L, kind))
    check_norm(out, every, kind, 0.125, 1.0, "again")
    L.lct_norm_join([], out, 1.0, 1.0, kind_of(L, kind))
    torch.cuda.synchronize()
    assert float(out.norm) == 0.0 and float(out.coef) == 1.0
    parts[1].sum.fill_(NAN)
    L.lct_norm_join(parts, out, 1.0, 1.0, kind_of(L, kind))
    torch.cuda.synchronize()
    assert np.isnan(float(out.norm)) and np.isnan(float(out.coef))
    with pytest.raises(ValueError, match="uint8"):
        L.lct_norm_join(torch.zeros(2, 4, device="cuda"), out)


# ------------------------------------------------------------------ clip

def scaled(x, c, dtype):
    """fp32 products rounded to dtype, on the host."""
    return (x.detach().cpu().float() * torch.tensor(c, dtype=SF)).to(dtype)


def same_bits(a, b, what=""):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    nan = torch.isnan(a)
    assert torch.equal(nan, torch.isnan(b)), what + " NaNs"
    it = torch.int32 if a.dtype == SF else torch.int16
    assert torch.equal(a.view(it)[~nan], b.view(it)[~nan]), what


@pytest.mark.parametrize("to", [BF, HF, SF])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_clip_sizes_types_and_alignments(L, dtype, to):
    """Every edge size at several alignments of source and target; what lies
    around the targets stays as it was."""
    c = torch.tensor(0.3337, device="cuda")
    for sx, sy in ((0, 0), (1, 1), (3, 0), (0, 5)):
        _, xs = views(EDGES, dtype, 100 + sx, sx, 1.0)
        flat, ys = views(EDGES, to, 200 + sy, sy, 1.0)
        before = flat.clone()
        L.lct_list_clip(L.LctList(xs), c, L.LctList(ys))
        torch.cuda.synchronize()
        for n, x, y in zip(EDGES, xs, ys):
            same_bits(y, scaled(x, 0.3337, to), "%d elements, shifts %d %d" % (n, sx, sy))
        at = sy + sum(EDGES)
        same_bits(flat[:sy], before[:sy])
        same_bits(flat[at:], before[at:])


@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_clip_in_place(L, dtype):
    """In place, with the coefficients 1 (memory stays untouched, NaN payloads
    too), 0, NaN and infinity."""
    ns = EDGES + [300_000]
    for c in (0.5, 1.0, 0.0, NAN, INF, -2.0, 1e-30):
        flat, xs = views(ns, dtype, 7, 1, 1.0)
        xs[-1][:8] = torch.tensor([INF, -INF, NAN, 0.0, -0.0, 1e-7, 65504.0, -65504.0], dtype=SF).to(dtype).cuda()
        if dtype == BF:
            flat.view(torch.int16)[1 + sum(EDGES) + 9] = 0x7F81    # a signalling NaN
        before = flat.clone()
        L.lct_list_clip(L.LctList(xs), torch.tensor(c, device="cuda"))
        torch.cuda.synchronize()
        lo, hi = 1, 1 + sum(ns)
        if c == 1.0:
            it = torch.int32 if dtype == SF else torch.int16
            assert torch.equal(flat.view(it), before.view(it))
        same_bits(flat[lo:hi], scaled(before[lo:hi], c, dtype), "c = %s" % c)
        same_bits(flat[:lo], before[:lo])
        same_bits(flat[hi:], before[hi:])


def test_clip_rounds_and_overflows(L):
    """Every finite BF16 value times a coefficient to BF16 and FP16 (overflow
    to infinity, subnormal results), and every FP16 value."""
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16)
    for src in (every.view(BF), every.view(HF)):
        for c in (0.77, 1e-6, 300.0):
            for to in (BF, HF, SF):
                y = torch.empty(65536, dtype=to, device="cuda")
                L.lct_list_clip(L.LctList([src.cuda()]), torch.tensor(c, device="cuda"), L.LctList([y]))
                torch.cuda.synchronize()
                same_bits(y, scaled(src, c, to), "%s to %s, c = %s" % (src.dtype, to, c))


def test_clip_many_tensors_and_refusals(L):
    r = np.random.default_rng(9)
    ns = [int(v) for v in r.choice([0, 1, 130, 2560, 33000], size=301)]
    types = [[BF, HF, SF][int(k)] for k in r.integers(0, 3, 301)]
    xs = [(torch.randn(n, device="cuda")).to(t) for n, t in zip(ns, types)]
    ys = [torch.empty(n, dtype=t, device="cuda") for n, t in zip(ns, types[::-1])]
    c = torch.tensor([0.9], device="cuda")
    L.lct_list_clip(L.LctList(xs), c, L.LctList(ys))
    torch.cuda.synchronize()
    for k, (x, y) in enumerate(zip(xs, ys)):
        same_bits(y, scaled(x, 0.9, y.dtype), "tensor %d" % k)
    L.lct_list_clip(L.LctList([]), c)
    with pytest.raises(L.LctError, match="overlap"):
        L.lct_list_clip(L.LctList([xs[2], xs[2]]) if ns[2] else L.LctList([c, c]), torch.tensor(1.0, device="cuda"))
    x = torch.randn(100, device="cuda")
    with pytest.raises(L.LctError, match="overlap"):
        L.lct_list_clip(L.LctList([x[:50]]), c, L.LctList([x[10:60]]))
    with pytest.raises(L.LctError, match="overlap"):
        L.lct_list_clip(L.LctList([x]), x[3:4])
    with pytest.raises(L.LctError):
        L.lct_list_clip(L.LctList([x]), c, L.LctList([x[:50].clone()]))


def test_clip_grad_norm_of_a_module(L):
    """Gradients of a small module clipped in place: the formula, and the norm
    afterwards."""
    torch.manual_seed(3)
    net = torch.nn.Sequential(torch.nn.Linear(96, 130), torch.nn.GELU(), torch.nn.Linear(130, 7)).cuda().to(BF)
    net(torch.randn(33, 96, device="cuda", dtype=BF)).float().square().sum().backward()
    grads = [p.grad for p in net.parameters()]
    before = [g.clone() for g in grads]
    out = L.clip_grad_norm(grads, 0.5)
    check_norm(out, [f64(g) for g in before], "l2", 0.5, 1.0, "module")
    assert float(out.norm) > 0.5
    for g, b in zip(grads, before):
        same_bits(g, scaled(b, float(out.coef), BF))
    # each value is off by half a step at most, so the norm is too
    after = L.grad_norm(grads, each=True)
    torch.cuda.synchronize()
    assert abs(float(after.norm) - 0.5) <= 0.5 * (2.0 ** -8 + 2.0 ** -22 + 1e-6 / float(out.norm))


# ------------------------------------------------------------------ compressed norms

def coded(L, x16, model, B, cw):
    cb = L.lct_codebook_build(L.Model(model.family, model.scale, model.shape), dev(x16))
    return cb, L.encode(cb, dev(x16), L.layout(B, cw))


def bits64(x16):
    return (np.asarray(x16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 1), (8192, 3), (32768, 12), (32768, 11)])
def test_tensor_norm(L, B, cw, kind):
    """Full and partial blocks, with and without spilled fields, from one
    element up."""
    g = np.random.default_rng(B + cw)
    for n in (1, 255, 256, 4097, B, B + 1, 5 * B + 531):
        x = synth.to_bf16_bits(g.laplace(0, 0.02, n))
        cb, t = coded(L, x, synth.Model(1, 0.02), B, cw)
        out = L.alloc_norm(nblk=t.sizes.nblk)
        out.scratch.fill_(0xFF)
        L.lct_tensor_norm(cb, t, out, 0.5, 0.25, kind_of(L, kind))
        check_norm(out, [bits64(x)], kind, 0.5, 0.25, "n=%d B=%d cw=%d" % (n, B, cw), more=CODES)
    if cw == 1:
        assert t.spilled() > 0


def test_tensor_norm_values_out_of_the_ordinary(L):
    """Runs of escapes that overrun a window, values whose squares 32 bits
    cannot hold, infinities and NaNs, on full blocks and partial ones."""
    g = np.random.default_rng(17)
    for n in (2 * 65536, 65536 + 4000):
        base = synth.to_bf16_bits(g.normal(0, 0.02, n))
        tiny = synth.to_bf16_bits(np.array([1e-30, -3e-33, 2e-35, -1e-36]))
        for j in range(4):
            base[(40 + j) * 256 + 5] = tiny[j]
        for special in (None, 0x7F7F, 0x0001, 0x7F80, 0xFF80, 0x7FC0, 0xFFC1):
            x = base.copy()
            if special is not None:
                x[n - 77] = special
            cb, t = coded(L, x, synth.Model(0, 0.02), 65536, 25)
            for kind in ("l2", "max"):
                out = L.alloc_norm(nblk=t.sizes.nblk)
                L.lct_tensor_norm(cb, t, out, 1.0, 1.0, kind_of(L, kind))
                check_norm(out, [bits64(x)], kind, 1.0, 1.0, "special %s" % special, more=CODES)
    x = np.zeros(70000, np.uint16)
    cb, t = coded(L, x, synth.Model(0, 0.02), 65536, 25)
    out = L.alloc_norm(nblk=t.sizes.nblk)
    L.lct_tensor_norm(cb, t, out, 1.0, 1.0)
    check_norm(out, [bits64(x)], "l2", 1.0, 1.0, "zeros", more=CODES)
    # an empty tensor
    t = L.alloc_tensor(0, L.layout(65536, 25))
    L.lct_tensor_norm(cb, t, out, 1.0, 1.0)
    torch.cuda.synchronize()
    assert float(out.norm) == 0.0 and float(out.coef) == 1.0


def group_of(L, xs, B, cw, sigma):
    """A group over the given BF16 bit arrays, a codebook for each, encoded."""
    lay = L.layout(B, cw)
    dense = [dev(x).view(BF) if len(x) else torch.empty(8, dtype=BF, device="cuda") for x in xs]
    cbs = [L.lct_codebook_build(L.Model(0, sigma * (k % 3 + 1), 0.0), dense[k][:len(x)]) for k, x in enumerate(xs)]
    g = L.LctGroup([len(x) for x in xs], lay, cbs, dense)
    st = g.alloc_storage(L.full_ovf_cap(sum(len(x) for x in xs) + 65536 * len(xs), lay))
    L.lct_encode_group(g, st)
    return g, st, cbs, dense


GROUP_NS = [3 * 65536 + 5, 0, 1, 255, 4097, 65536, 2 * 65536 + 300, 70000, 256, 9000, 0]


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 2), (32768, 12), (32768, 11)])
def test_group_norm(L, B, cw, kind):
    g = np.random.default_rng(50 + cw)
    xs = [synth.to_bf16_bits(g.normal(0, 0.02 * (k % 3 + 1), n)) for k, n in enumerate(GROUP_NS)]
    grp, st, _, _ = group_of(L, xs, B, cw, 0.02)
    for each in (True, False):
        out = L.alloc_norm(len(xs), each, st.sizes.nblk)
        out.scratch.fill_(0xFF)
        L.lct_group_norm(grp, st, out, 1.0, 2.0, kind_of(L, kind))
        check_norm(out, [bits64(x) for x in xs], kind, 1.0, 2.0, "group B=%d cw=%d" % (B, cw), more=CODES)
    # a group with no blocks
    e = L.LctGroup([0, 0], L.layout(B, cw), list(grp.codebooks)[:2])
    es = e.alloc_storage(16)
    out = L.alloc_norm(2, True)
    L.lct_group_norm(e, es, out, 1.0, 1.0, kind_of(L, kind))
    torch.cuda.synchronize()
    assert float(out.norm) == 0.0 and float(out.each.abs().sum()) == 0.0


def test_tensor_norm_of_many_blocks(L):
    """More blocks than are joined at once, flat and as a group of two."""
    n = 4096 * 5000 + 9
    x = (torch.randn(n, device="cuda") * 0.02).to(BF)
    lay = L.layout(4096, 4)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), x)
    t = L.encode(cb, x, lay)
    v = f64(x)
    for kind in ("l2", "max"):
        out = L.alloc_norm(nblk=t.sizes.nblk)
        out.scratch.fill_(0xFF)
        L.lct_tensor_norm(cb, t, out, 1.0, 1.0, kind_of(L, kind))
        check_norm(out, [v], kind, 1.0, 1.0, "5001 blocks", more=CODES)
    k = 4096 * 4500
    grp = L.LctGroup([k, n - k], lay, [cb, cb], [x[:k], x[k:].clone()])
    st = grp.alloc_storage(L.full_ovf_cap(n + 4096, lay))
    L.lct_encode_group(grp, st)
    out = L.alloc_norm(2, True, st.sizes.nblk)
    L.lct_group_norm(grp, st, out, 1.0, 1.0)
    check_norm(out, [v[:k], v[k:]], "l2", 1.0, 1.0, "group of 5001 blocks", more=CODES)


# ------------------------------------------------------------------ clipped steps

def step_inputs(n, seed, specials=True):
    g = np.random.default_rng(seed)
    w = synth.to_bf16_bits(g.laplace(0, 0.02, n))
    m = synth.to_bf16_bits(g.normal(0, 1e-2, n))
    gr = synth.to_bf16_bits(g.normal(0, 0.1, n))
    if specials and n > 400:
        sp = [0x7FC0, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x8001, 0x7F7F, 0xFF7F]
        m[:64] = sp * 8
        w[100:164] = sp * 8
        gr[300:364] = sp * 8
    return w, m, gr


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 1), (8192, 3), (32768, 12), (32768, 11)])
def test_clipped_steps_equal_the_oracle(L, orc, B, cw, inplace):
    """Full and partial blocks, with spills where the capacity is small: every
    byte of the outputs."""
    n = 3 * B + 531
    w, m, gr = step_inputs(n, B + cw)
    lay = L.layout(B, cw)
    cbw, ocw = check_codebook(L, orc, synth.Model(1, 0.02), w)
    cbm, ocm = check_codebook(L, orc, synth.Model(0, 1e-2), m)
    rw, rm = orc.encode(ocw, w, B, cw), orc.encode(ocm, m, B, cw)
    for c in (0.3701, 1.0, 0.0, NAN):
        coef = torch.tensor([c], device="cuda")
        tw, tm = L.encode(cbw, dev(w), lay), L.encode(cbm, dev(m), lay)
        ow, om = L.alloc_tensor(n, lay), L.alloc_tensor(n, lay)
        if inplace:
            ow.sf, ow.pay, ow.cnt, ow.obase = tw.sf, tw.pay, tw.cnt, tw.obase
            om.sf, om.pay, om.cnt, om.obase = tm.sf, tm.pay, tm.cnt, tm.obase
        L.lct_momentum_step_clip(cbw, tw, cbm, tm, dev(gr), coef, 0.9, 0.05, ow, om)
        wo, mo = orc.momentum_clip_dense(w, m, gr, c, 0.9, 0.05)
        assert_same(host_parts(ow), orc.encode(ocw, wo, B, cw), "W' c=%s" % c)
        assert_same(host_parts(om), orc.encode(ocm, mo, B, cw), "M' c=%s" % c)
        # the update: eta * c is one fp32 product
        tw, tm = L.encode(cbw, dev(w), lay), L.encode(cbm, dev(m), lay)
        ow = L.alloc_tensor(n, lay)
        if inplace:
            ow.sf, ow.pay, ow.cnt, ow.obase = tw.sf, tw.pay, tw.cnt, tw.obase
        L.lct_sgd_step_clip(cbw, tw, cbm, tm, 0.05, coef, ow)
        ref = orc.sgd(ocw, rw, ocm, rm, float(np.float32(0.05) * np.float32(c)))
        assert_same(host_parts(ow), ref, "sgd c=%s" % c)


def test_clipped_full_blocks_take_the_full_path(L, orc):
    """Full blocks without spills: every unit runs on the full-block path, NaNs
    and escape runs included, at each mode's capacity."""
    for B, cw in ((65536, 25), (32768, 12), (32768, 11)):
        g = np.random.default_rng(cw)
        n = 3 * B
        w, m, gr = (synth.to_bf16_bits(g.normal(0, s, n)) for s in (0.01, 5e-4, 1e-4))
        if cw == 25:
            gr[17 * 256 + 129] = 0x7F81
            tiny = synth.to_bf16_bits(np.array([1e-30, -3e-33, 2e-35, -1e-36]))
            for j in range(4):
                m[(40 + j) * 256 + 70] = tiny[j]
        ocw, ocm = orc.codebook_build(0, 0.01, 0.0, w), orc.codebook_build(0, 5e-4, 0.0, m)
        cbw, cbm = L.lct_codebook_build(L.Model(0, 0.01, 0.0), dev(w)), L.lct_codebook_build(L.Model(0, 5e-4, 0.0), dev(m))
        lay = L.layout(B, cw)
        rw, rm = orc.encode(ocw, w, B, cw), orc.encode(ocm, m, B, cw)
        coef = torch.tensor(0.61, device="cuda")
        tw, tm = L.encode(cbw, dev(w), lay), L.encode(cbm, dev(m), lay)
        ow, om = L.alloc_tensor(n, lay), L.alloc_tensor(n, lay)
        L.lct_momentum_step_clip(cbw, tw, cbm, tm, dev(gr), coef, 0.9, 1e-3, ow, om)
        wo, mo = orc.momentum_clip_dense(w, m, gr, 0.61, 0.9, 1e-3)
        assert_same(host_parts(ow), orc.encode(ocw, wo, B, cw), "W' cw=%d" % cw)
        assert_same(host_parts(om), orc.encode(ocm, mo, B, cw), "M' cw=%d" % cw)
        if cw == 25:
            assert rw.spilled == 0 and rm.spilled == 0
            assert ow.full_path_units() == 12 and om.full_path_units() == 12
        L.lct_sgd_step_clip(cbw, tw, cbm, tm, 0.5, coef, ow)
        assert_same(host_parts(ow), orc.sgd(ocw, rw, ocm, rm, float(np.float32(0.5) * np.float32(0.61))),
                    "sgd cw=%d" % cw)


@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 2), (32768, 12)])
def test_clipped_group_steps_equal_single_ones(L, B, cw):
    """The group forms write each member's values as the single calls do, and
    with a coefficient of 1 the unclipped group calls' bytes."""
    ns = [2 * 65536, 65536 + 17, 5, 0, 3 * 65536, 40000]
    ins = [step_inputs(n, 70 + k, specials=k == 1) for k, n in enumerate(ns)]
    gw, ws, cbw, _ = group_of(L, [i[0] for i in ins], B, cw, 0.02)
    gm, ms, cbm, _ = group_of(L, [i[1] for i in ins], B, cw, 1e-2)
    gdense = [dev(i[2]).view(BF) if n else torch.empty(8, dtype=BF, device="cuda") for i, n in zip(ins, ns)]
    gg = L.LctGroup(ns, L.layout(B, cw), cbm, gdense)
    cap = ws.ovf_cap

    def stores():
        return gw.alloc_storage(cap), gm.alloc_storage(cap)

    def buffers(t):
        torch.cuda.synchronize()
        sp = int(t.obase[-1])
        return [t.sf, t.pay[:t.sizes.pay // 4], t.cnt[:t.sizes.cnt // 2], t.obase, t.ovf[:sp], t.status[:1]]

    def equal(a, b, what):
        for k, (u, v) in enumerate(zip(buffers(a), buffers(b))):
            assert torch.equal(u, v), "%s buffer %d" % (what, k)

    one, c = torch.tensor(1.0, device="cuda"), torch.tensor(0.25, device="cuda")
    (w1, m1), (w2, m2) = stores(), stores()
    L.lct_momentum_step_group(gw, ws, gm, ms, gg, 0.9, 0.05, w1, m1)
    L.lct_momentum_step_clip_group(gw, ws, gm, ms, gg, one, 0.9, 0.05, w2, m2)
    equal(w1, w2, "momentum W'")
    equal(m1, m2, "momentum M'")
    L.lct_sgd_step_group(gw, ws, gm, ms, 0.05, w1)
    L.lct_sgd_step_clip_group(gw, ws, gm, ms, 0.05, one, w2)
    equal(w1, w2, "sgd W'")
    # another coefficient, against the single-tensor calls
    L.lct_momentum_step_clip_group(gw, ws, gm, ms, gg, c, 0.9, 0.05, w1, m1)
    L.lct_sgd_step_clip_group(gw, ws, gm, ms, 0.05, c, w2)
    lay = L.layout(B, cw)
    for k, n in enumerate(ns):
        if n == 0:
            continue
        tw, tm = L.encode(cbw[k], dev(ins[k][0]), lay), L.encode(cbm[k], dev(ins[k][1]), lay)
        ow, om = L.alloc_tensor(n, lay), L.alloc_tensor(n, lay)
        L.lct_momentum_step_clip(cbw[k], tw, cbm[k], tm, dev(ins[k][2]), c, 0.9, 0.05, ow, om)
        for group, store, single, cb in ((gw, w1, ow, cbw[k]), (gm, m1, om, cbm[k])):
            a, b = L.decode(cb, group.tensor(store, k)), L.decode(cb, single)
            torch.cuda.synchronize()
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), k
        L.lct_sgd_step_clip(cbw[k], tw, cbm[k], tm, 0.05, c, ow)
        a, b = L.decode(cbw[k], gw.tensor(w2, k)), L.decode(cbw[k], ow)
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), k


# ------------------------------------------------------------------ a step as a whole

class Step:
    """A training step's tail on a group: fp32 accumulators, their norm, the
    clip into the BF16 gradients, the momentum step; and the fused form, with
    the BF16 gradients' norm and the clipped momentum step."""

    def __init__(self, L, ns, seed):
        self.L, self.ns = L, ns
        lay = L.layout(65536, 25)
        ins = [step_inputs(n, seed + k, specials=False) for k, n in enumerate(ns)]
        self.w, self.m = [i[0] for i in ins], [i[1] for i in ins]
        self.gw, self.ws, self.cbw, _ = group_of(L, self.w, 65536, 25, 0.02)
        self.gm, self.ms, self.cbm, _ = group_of(L, self.m, 65536, 25, 1e-2)
        self.acc = [torch.zeros(n, device="cuda") for n in ns]
        self.g16 = [torch.zeros(n, dtype=BF, device="cuda") for n in ns]
        self.gg = L.LctGroup(ns, lay, self.cbm, self.g16)
        self.xs, self.ys = L.LctList(self.acc), L.LctList(self.g16)
        cap = self.ws.ovf_cap
        self.wo, self.mo = self.gw.alloc_storage(cap), self.gm.alloc_storage(cap)
        self.norm, self.norm16 = L.alloc_norm(len(ns), True), L.alloc_norm(len(ns))
        self.mnorm = L.alloc_norm(len(ns), True, self.ms.sizes.nblk)
        self.wf, self.mf, self.ws2 = (g.alloc_storage(cap) for g in (self.gw, self.gm, self.gw))

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        for a in self.acc:
            a.copy_(torch.randn(a.numel(), generator=g) * 0.3)

    def run(self):
        L = self.L
        L.lct_list_norm(self.xs, self.norm, 1.0, 1.0 / 8)
        L.lct_list_clip(self.xs, self.norm, self.ys)
        L.lct_momentum_step_group(self.gw, self.ws, self.gm, self.ms, self.gg, 0.9, 0.05, self.wo, self.mo)
        L.lct_list_norm(self.ys, self.norm16, 0.5)
        L.lct_momentum_step_clip_group(self.gw, self.ws, self.gm, self.ms, self.gg, self.norm16, 0.9, 0.05,
                                       self.wf, self.mf)
        L.lct_group_norm(self.gm, self.ms, self.mnorm, 0.25)
        L.lct_sgd_step_clip_group(self.gw, self.ws, self.gm, self.ms, 0.05, self.mnorm, self.ws2)

    def results(self):
        torch.cuda.synchronize()
        out = [self.norm.buf, self.norm.each, self.norm16.buf, self.mnorm.buf, self.mnorm.each] + self.g16
        for t in (self.wo, self.mo, self.wf, self.mf, self.ws2):
            out += [t.sf, t.pay[:t.sizes.pay // 4], t.cnt[:t.sizes.cnt // 2], t.obase, t.ovf[:int(t.obase[-1])]]
        return [x.clone() for x in out]

    def wipe(self):
        for t in (self.wo, self.mo, self.wf, self.mf, self.ws2):
            t.pay.fill_(-1)
            t.cnt.fill_(-1)
            t.obase.fill_(-1)
        for n in (self.norm, self.norm16, self.mnorm):
            n.buf.fill_(0xFF)
        for g in self.g16:
            g.fill_(7.0)


STEP_NS = [2 * 65536 + 100, 1, 300, 70001, 128]


def test_step_as_a_whole(L, orc):
    s = Step(L, STEP_NS, 500)
    s.fill(1)
    s.run()
    s.results()
    check_norm(s.norm, [f64(a) for a in s.acc], "l2", 1.0, 1.0 / 8, "accumulators")
    c = float(s.norm.coef)
    for a, g in zip(s.acc, s.g16):
        same_bits(g, scaled(a, c, BF))
    check_norm(s.norm16, [f64(g) for g in s.g16], "l2", 0.5, 1.0, "gradients")
    check_norm(s.mnorm, [bits64(m) for m in s.m], "l2", 0.25, 1.0, "momentum", CODES)
    c16, cm = float(s.norm16.coef), float(s.mnorm.coef)
    assert c < 0.125 and c16 < 1 and cm < 1
    for k, n in enumerate(STEP_NS):
        gr = s.g16[k].view(torch.int16).cpu().numpy().view(np.uint16)
        for (wt, mt), cc in (((s.wo, s.mo), 1.0), ((s.wf, s.mf), c16)):
            wr, mr = orc.momentum_clip_dense(s.w[k], s.m[k], gr, cc, 0.9, 0.05)
            for grp, st, cb, ref in ((s.gw, wt, s.cbw[k], wr), (s.gm, mt, s.cbm[k], mr)):
                y = L.decode(cb, grp.tensor(st, k))
                torch.cuda.synchronize()
                assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), ref), k


def test_step_on_a_side_stream(L):
    s = Step(L, STEP_NS, 600)
    s.fill(2)
    s.run()
    ref = s.results()
    s.wipe()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    side.synchronize()
    for k, (a, b) in enumerate(zip(ref, s.results())):
        assert torch.equal(a, b), k


def test_step_replayed_from_a_graph(L):
    """The whole tail captured once and replayed with other gradients; between
    the replays the outputs are overwritten and another step runs eagerly."""
    s, other = Step(L, STEP_NS, 700), Step(L, [5000, 65536], 800)
    other.fill(9)
    s.fill(3)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for rep in range(4):
        s.fill(20 + rep)
        s.wipe()
        s.run()
        ref = s.results()
        s.wipe()
        if rep % 2:
            other.run()
        torch.cuda.synchronize()
        graph.replay()
        for k, (a, b) in enumerate(zip(ref, s.results())):
            assert torch.equal(a, b), "replay %d, result %d" % (rep, k)


def test_norms_on_two_streams_at_once(L):
    """Two calls that overlap in time, each with its own result and scratch."""
    xs = [[(torch.randn(n, device="cuda") * (i + 1)).to(BF) for n in (3_000_000, 17)] for i in range(2)]
    lists = [L.LctList(x) for x in xs]
    outs = [L.alloc_norm(2, True) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, li, o in zip(streams, lists, outs):
            L.lct_list_norm(li, o, 1.0, stream=st)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        check_norm(o, [f64(t) for t in x], "l2", 1.0, 1.0)


def test_another_current_device_is_refused(L, monkeypatch):
    """Buffers on a device that is not the current one never reach a kernel."""
    x = torch.randn(100, device="cuda")
    lst, out = L.LctList([x]), L.alloc_norm(1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        L.lct_list_norm(lst, out)
    with pytest.raises(ValueError, match="current device"):
        L.lct_list_clip(lst, torch.ones(1, device=x.device))


# ------------------------------------------------------------------ where the updates' kernels meet

def update_case(L, orc, w, m, gr, B, cw, c, eta, inplace, what):
    """The clipped and the plain update and momentum step of one tensor against
    the oracle's bytes; (W', M', update's W') as device tensors."""
    n = w.size
    lay = L.layout(B, cw)
    cbw, ocw = check_codebook(L, orc, synth.Model(0, 0.02), w)
    cbm, ocm = check_codebook(L, orc, synth.Model(0, 1e-3), m)
    rw, rm = orc.encode(ocw, w, B, cw), orc.encode(ocm, m, B, cw)
    outs = []
    for clip in (True, False):
        coef = torch.tensor([c if clip else 1.0], device="cuda")
        cc = float(np.float32(c)) if clip else 1.0

        def fresh():
            tw, tm = L.encode(cbw, dev(w), lay), L.encode(cbm, dev(m), lay)
            ow, om = L.alloc_tensor(n, lay), L.alloc_tensor(n, lay)
            if inplace:
                ow.sf, ow.pay, ow.cnt, ow.obase = tw.sf, tw.pay, tw.cnt, tw.obase
            return tw, tm, ow, om

        tw, tm, ow, om = fresh()
        if inplace:
            om.sf, om.pay, om.cnt, om.obase = tm.sf, tm.pay, tm.cnt, tm.obase
        if clip:
            L.lct_momentum_step_clip(cbw, tw, cbm, tm, dev(gr), coef, 0.9, eta, ow, om)
        else:
            L.lct_momentum_step(cbw, tw, cbm, tm, dev(gr), 0.9, eta, ow, om)
        wo, mo = orc.momentum_clip_dense(w, m, gr, cc, 0.9, eta)
        ref_w, ref_m = orc.encode(ocw, wo, B, cw), orc.encode(ocm, mo, B, cw)
        assert_same(host_parts(ow), ref_w, what + " W'")
        assert_same(host_parts(om), ref_m, what + " M'")
        tw, tm, os_, _ = fresh()
        if clip:
            L.lct_sgd_step_clip(cbw, tw, cbm, tm, eta, coef, os_)
        else:
            L.lct_sgd_step(cbw, tw, cbm, tm, eta, os_)
        assert_same(host_parts(os_), orc.sgd(ocw, rw, ocm, rm, float(np.float32(eta) * np.float32(cc))), what + " sgd")
        outs.append((ow, om, os_, ref_w, ref_m))
        for cb, t, x in ((cbw, os_, None), (cbw, ow, wo), (cbm, om, mo)):
            y = L.decode(cb, t)
            torch.cuda.synchronize()
            if x is not None:
                assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), x), what
    return outs


def three(n, seed, sg=1e-3):
    g = np.random.default_rng(seed)
    return [synth.to_bf16_bits(g.normal(0, s, n)) for s in (0.02, 1e-3, sg)]


LAST = [1, 255, 256, 257, 4095, 4096, 4097, 5 * 4096 + 300, 8192, 30000, 32767]


@pytest.mark.parametrize("B,cw", [(65536, 25), (32768, 12), (32768, 11)])
def test_partial_blocks_of_every_kind(L, orc, B, cw):
    """A whole block and a last one of many lengths: shorter than a step, whole
    steps, whole steps and a rest, one element short of a block."""
    for last in LAST + ([B - 256, B - 1] if B == 65536 else []):
        n = B + last
        w, m, gr = three(n, last)
        update_case(L, orc, w, m, gr, B, cw, 0.37, 0.1, last % 2 == 0, "last=%d cw=%d" % (last, cw))


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,cw,last", [(65536, 25, 40000), (65536, 25, 65535), (32768, 11, 20001), (32768, 12, 4097)])
def test_partial_blocks_whose_outputs_spill(L, orc, B, cw, last, inplace):
    """No input field spilled, so a partial block takes the full-block path,
    whose outputs run out of room midway and go on spilling in its rest."""
    g = np.random.default_rng(last + cw)
    n = B + last
    # inputs from a narrow band of exponents (short codes), a gradient far
    # outside M's codes and a rate that carries W outside its own
    w = synth.to_bf16_bits(np.sign(g.normal(size=n)) * g.uniform(0.016, 0.031, n))
    m = synth.to_bf16_bits(np.sign(g.normal(size=n)) * g.uniform(0.8e-3, 1.5e-3, n))
    gr = synth.to_bf16_bits(g.normal(0, 0.5, n))
    outs = update_case(L, orc, w, m, gr, B, cw, 0.9, 40.0, inplace, "spills last=%d cw=%d" % (last, cw))
    assert all(o[4].spilled > n // 8 for o in outs)


@pytest.mark.parametrize("B,cw", [(4096, 25), (8192, 25), (4096, 12), (4096, 11), (4096, 7)])
def test_more_blocks_than_workgroups(L, orc, B, cw):
    """More blocks than the general kernels have workgroups: full blocks run in
    the kernels of their own (the ring kernel at 25 words), the last, partial
    one and those with spilled inputs in the general ones."""
    n = 700 * B + 1234
    w, m, gr = three(n, B + cw)
    if cw >= 11:
        w[5 * B:5 * B + 3000] = synth.to_bf16_bits(np.full(3000, 1e-25))    # spills one block's inputs
    outs = update_case(L, orc, w, m, gr, B, cw, 0.37, 0.1, False, "700 blocks of %d, cw=%d" % (B, cw))
    full = outs[0][2].full_path_units()
    assert full == outs[1][2].full_path_units() and full <= 4 * 700
    if cw == 25:
        assert full >= 4 * 690
    update_case(L, orc, w, m, gr, B, cw, 0.37, 0.1, True, "in place, 700 blocks of %d, cw=%d" % (B, cw))


def test_around_one_workgroup_per_block(L, orc):
    """Numbers of blocks about the size from which one scan, and from which one
    kernel, no longer does all of them."""
    for nblk in (255, 256, 257, 511, 512, 513):
        n = (nblk - 1) * 4096 + 77
        w, m, gr = three(n, nblk)
        update_case(L, orc, w, m, gr, 4096, 25, 0.5, 0.1, nblk % 2 == 0, "%d blocks" % nblk)


def test_norm_scratch_is_not_passed(L):
    """Guards after the scratch and around the results stay, for every form of
    the norms."""
    def guarded(need):
        buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[:need]

    r = np.random.default_rng(2)
    for ns in ([3], [100, 0, 5000], [3_000_000], [int(v) for v in r.integers(1, 70000, 401)], [50] * 193):
        xs = [torch.randn(n, device="cuda").to(BF) for n in ns]
        lst = L.LctList(xs)
        for each in (True, False):
            buf, scr = guarded(lst.need)
            out = L.alloc_norm(len(ns), each, scratch=scr)
            L.lct_list_norm(lst, out, 1.0)
            check_norm(out, [f64(x) for x in xs], "l2", 1.0, 1.0, "%d tensors" % len(ns))
            assert (buf[lst.need:] == 0xA5).all()
    for n in (100, 4096 * 4200 + 5):
        x = (torch.randn(n, device="cuda") * 0.02).to(BF)
        cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), x)
        t = L.encode(cb, x, L.layout(4096, 4))
        need = L._norm_scratch(0, t.sizes.nblk)
        buf, scr = guarded(need)
        out = L.alloc_norm(scratch=scr, nblk=t.sizes.nblk)
        L.lct_tensor_norm(cb, t, out, 1.0)
        check_norm(out, [f64(x)], "l2", 1.0, 1.0, "codes", CODES)
        assert (buf[need:] == 0xA5).all()


def test_short_norm_and_clip_replayed_from_a_graph(L):
    """The one-launch norm and the clip in place captured together: each replay
    scales what the one before left."""
    xs = [torch.empty(n, device="cuda") for n in (1000, 1, 20000)]
    ref = [torch.empty_like(x) for x in xs]
    lst, rl = L.LctList(xs), L.LctList(ref)
    out, ro = L.alloc_norm(3, True), L.alloc_norm(3, True)

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        for x, y in zip(xs, ref):
            v = torch.randn(x.numel(), generator=g)
            x.copy_(v)
            y.copy_(v)

    fill(0)
    L.lct_list_norm(lst, out, 5.0)
    L.lct_list_clip(lst, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lct_list_norm(lst, out, 5.0)
        L.lct_list_clip(lst, out)
    for rep in range(4):
        fill(rep)
        L.lct_list_norm(rl, ro, 5.0)
        L.lct_list_clip(rl, ro)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.buf, ro.buf) and torch.equal(out.each, ro.each), rep
        assert all(torch.equal(a, b) for a, b in zip(xs, ref)), rep
        assert abs(float(L.grad_norm(xs).norm) - 5.0) < 5.0 * 2.0 ** -20


def test_a_kept_descriptor_follows_its_buffers(L):
    """A tensor's descriptor is kept from call to call: a buffer that is
    replaced (by a right one, a short one, none) is seen, and not held."""
    import weakref
    n = 70000
    x = (torch.randn(n, device="cuda") * 0.02).to(BF)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), x)
    t = L.encode(cb, x, L.layout(65536, 25))
    a = t.c()
    assert t.c() is a and t.c(need_scratch=False) is a
    t.status.set_(torch.zeros(4, dtype=torch.int32, device="cuda"))      # the same tensor over other memory
    assert t.c() is not a and t.c().status == t.status.data_ptr()
    a = t.c()
    old = weakref.ref(t.scratch)
    t.scratch = torch.empty_like(t.scratch)
    assert old() is None
    b = t.c()
    assert b is not a and b.scratch == t.scratch.data_ptr()
    t.scratch = None
    assert t.c().scratch is None
    t.scratch = torch.empty(16, dtype=torch.uint8, device="cuda")
    assert t.c(need_scratch=False).scratch == t.scratch.data_ptr()
    with pytest.raises(ValueError, match="scratch"):
        t.c()
    t.sf = t.sf[:n - 1]
    with pytest.raises(ValueError, match="sf"):
        t.c(need_scratch=False)
    t = L.encode(cb, x, L.layout(65536, 25))
    t.c()
    t.ovf_cap = t.ovf_cap * 2
    with pytest.raises(ValueError, match="ovf"):
        t.c()


def test_offsets_past_32_bits(L):
    """A tensor of more than 2^32 elements: the norm finds what lies at its far
    end, the clip scales it there and nothing else."""
    n = (1 << 32) + 70001
    x = torch.zeros(n, dtype=BF, device="cuda")
    at = torch.tensor([7, (1 << 32) + 5, n - 1], device="cuda")
    x[at] = torch.tensor([12.0, 4.0, -3.0], dtype=BF, device="cuda")
    lst = L.LctList([x[1:], x[:1]])
    out = L.alloc_norm(2, True)
    L.lct_list_norm(lst, out, 6.5)
    torch.cuda.synchronize()
    assert float(out.norm) == 13.0 and float(out.sum) == 169.0 and float(out.each[1]) == 0.0
    L.lct_list_norm(lst, out, kind=L.NORM_MAX)
    L.lct_list_clip(lst, torch.tensor(0.25, device="cuda"))
    torch.cuda.synchronize()
    assert float(out.norm) == 12.0
    assert x[at].tolist() == [3.0, 1.0, -0.75]
    L.lct_list_norm(lst, out)
    torch.cuda.synchronize()
    assert float(out.sum) == 9.0 + 1.0 + 0.5625
    # FP32 to FP16 over the same border
    del x, lst
    y = torch.zeros((1 << 32) + 3, device="cuda")
    y[-1] = 1.5
    z = torch.empty(y.numel(), dtype=HF, device="cuda")
    L.lct_list_clip(L.LctList([y]), torch.tensor(2.0, device="cuda"), L.LctList([z]))
    torch.cuda.synchronize()
    assert float(z[-1]) == 3.0 and float(z[-2]) == 0.0
    assert float(L.grad_norm([z]).norm) == 3.0


def test_a_list_holds_the_memory_it_was_made_for(L):
    """A tensor that is given other memory after the list was made: the calls
    reach neither that nor what is allocated next."""
    x = torch.ones(1 << 20, device="cuda")
    lst, old = L.LctList([x]), x.data_ptr()
    x.data = torch.ones(1 << 20, device="cuda")
    z = [torch.ones(1 << 20, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != old for t in z + [x])
    L.lct_list_clip(lst, torch.tensor(0.5, device="cuda"))
    out = L.alloc_norm(1)
    L.lct_list_norm(lst, out)
    assert out.sum.item() == (1 << 18)
    assert all(bool((t == 1).all()) for t in z + [x])
    L.lct_list_norm(L.LctList([x]), out)
    assert out.sum.item() == (1 << 20)


def test_clipped_steps_refuse_buffers_elsewhere(L):
    """Every buffer that stands for a step's operand, on the CPU or absent from
    the current device, is refused before a kernel could read it."""
    lay = L.layout(4096, 12)
    x = (0.02 * torch.randn(5000, device="cuda")).to(torch.bfloat16)
    cb = L.lct_codebook_build(L.Model(L.GAUSSIAN, 0.02, 0.0), x)
    t = [L.encode(cb, x, lay) for _ in range(4)]
    c = torch.ones(1, device="cuda")
    for k in range(4):
        sf = t[k].sf
        t[k].sf = sf.cpu()
        with pytest.raises(ValueError):
            L.lct_momentum_step_clip(cb, t[0], cb, t[1], x, c, 0.9, 0.1, t[2], t[3])
        if k < 3:
            with pytest.raises(ValueError):
                L.lct_sgd_step_clip(cb, t[0], cb, t[1], 0.1, c, t[2])
        t[k].sf = sf
    with pytest.raises((ValueError, TypeError)):
        L.lct_momentum_step_clip(cb, t[0], cb, t[1], x.cpu(), c, 0.9, 0.1, t[2], t[3])
    with pytest.raises(ValueError):
        L.lct_sgd_step_clip(cb, t[0], cb, t[1], 0.1, c.cpu(), t[2])
    g = L.LctGroup([5000], lay, [cb], [x])
    a, b, o = (g.alloc_storage(5000) for _ in range(3))
    L.lct_encode_group(g, a)
    L.lct_encode_group(g, b)
    table = g.table
    g.table = table.cpu()
    with pytest.raises(ValueError, match="current device"):
        L.lct_sgd_step_clip_group(g, a, g, b, 0.1, c, o)
    with pytest.raises(ValueError, match="the group's table"):
        L.lct_group_norm(g, a, L.alloc_norm(1, nblk=a.sizes.nblk))
    g.table = table
    L.lct_sgd_step_clip_group(g, a, g, b, 0.1, c, o)
    torch.cuda.synchronize()
    assert o.status_word() == 0
