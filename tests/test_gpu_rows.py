"""Rows of a compressed table, and a table's gradient by its tokens, on the GPU,
against plain forms.

Tolerances.  A lookup is one fp32 product of exact values (a BF16 value and the
scale), rounded to fp32 once and to a 16-bit type once more: it is compared bit
for bit with torch's product and conversion.  A gradient's element is a sum of k
terms in fp32: every partial sum is off by at most 2^-24 of its magnitude, which
is at most S, the sum of the magnitudes, so the sum is off by at most k * 2^-24 *
S; the scale's product and (with add) the fused addition add 2^-24 of the scaled
magnitudes each, and rounding to the result's type half a step of the value,
finfo.eps / 2 (or half of its smallest step)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def table(L, rows, cols, lay, seed=0, sigma=0.02, model_sigma=None, ovf_cap=None):
    torch.manual_seed(seed)
    w = (torch.randn(rows, cols, device="cuda") * sigma).bfloat16()
    cb = L.lct_codebook_build(L.Model(0, model_sigma or sigma, 0.0), w.view(-1))
    return w, cb, L.encode(cb, w.view(-1), lay, ovf_cap)


def looked_up(w, index, scale, dtype):
    inside = (index >= 0) & (index < w.shape[0])
    at = torch.where(inside, index, torch.zeros_like(index)).long()
    y = w[at].float() * scale
    y[~inside] = 0
    return y.to(dtype)


def same(a, b, what=""):
    it = torch.int32 if a.dtype == SF else torch.int16
    fa, fb = a.reshape(-1), b.reshape(-1)
    nan = torch.isnan(fb)
    assert torch.equal(torch.isnan(fa), nan), what
    assert torch.equal(fa.view(it)[~nan], fb.view(it)[~nan]), what


@pytest.mark.parametrize("cols", [1, 7, 255, 256, 257, 768, 2560, 65536, 70_001])
def test_lookup_widths(L, cols):
    """Rows shorter than a stream's step, rows that cross blocks, rows longer
    than a block; the first and the last row, repeats, indices outside."""
    rows = max(3, 300_000 // cols)
    w, cb, t = table(L, rows, cols, L.lct_layout_init(L.CLEAN), cols)
    torch.manual_seed(1)
    index = torch.cat([torch.tensor([0, rows - 1, -1, rows, 0, 2 ** 40, -(2 ** 40)]), torch.randint(0, rows, (40,))])
    index = index.cuda()
    for dtype, scale in ((BF, 1.0), (BF, 50.5964), (HF, 3.0), (SF, 0.1)):
        y = torch.full((index.numel(), cols), 7.0, dtype=dtype, device="cuda")
        L.lct_tensor_rows(cb, t, index, y, scale=scale)
        same(y, looked_up(w, index, scale, dtype), "%s %s" % (dtype, scale))


@pytest.mark.parametrize("B,cw", [(4096, 1), (8192, 3), (32768, 12), (32768, 11), (65536, 25), (4096, 64)])
def test_lookup_layouts_and_spills(L, B, cw):
    """Small capacities spill most fields; a model that does not fit spills
    more, and values out of the ordinary come back as they are."""
    rows, cols = 301, 531
    lay = L.layout(B, cw)
    for model_sigma in (0.02, 4.0):
        w, cb, t = table(L, rows, cols, lay, cw, model_sigma=model_sigma)
        w.view(-1)[1000:1008] = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-40, 3e38, -1e-38])
        L.lct_encode(cb, w.view(-1), t)
        index = torch.arange(-2, rows + 2, device="cuda", dtype=torch.int32)
        y = torch.empty(index.numel(), cols, dtype=BF, device="cuda")
        L.lct_tensor_rows(cb, t, index, y, scale=1.0)
        same(y, looked_up(w, index, 1.0, BF))


@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 1000, 1024, 4096, 4097, 5000, 40_000, 100_000])
def test_lookup_counts(L, count):
    """Few and many tokens (more than the table has rows), frequent ones often,
    in a batch of two dimensions; an unaligned output."""
    rows, cols = 4001, 321
    w, cb, t = table(L, rows, cols, L.lct_layout_init(L.CLEAN), 3)
    u = torch.rand(count, device="cuda", dtype=torch.float64)
    index = (torch.exp(u * np.log(rows + 1.0)) - 1).long().clamp(0, rows - 1)
    if count > 60:
        index[::50] = -1
    for work in (L.alloc_rows(count), None):
        flat = torch.full((count * cols + 9,), 7.0, dtype=BF, device="cuda")
        y = flat[1:1 + count * cols].view(count, cols)
        L.lct_tensor_rows(cb, t, index, y, work, scale=2.5)
        same(y, looked_up(w, index, 2.5, BF))
        assert bool((flat[0] == 7.0) & (flat[1 + count * cols:] == 7.0).all())


@pytest.mark.parametrize("cols", [1, 100, 256, 300, 4096, 20_000])
def test_sorted_lookups_of_rows_that_share_blocks_and_positions(L, cols):
    """Every row several times, in no order: rows that end within the position
    of a stream where the next begins, rows over several blocks, spills."""
    rows = max(2, 200_000 // cols)
    count = max(2048, 3 * min(rows, 5000))
    for lay in (L.lct_layout_init(L.CLEAN), L.layout(4096, 2)):
        w, cb, t = table(L, rows, cols, lay, cols)
        torch.manual_seed(2)
        index = torch.randint(-1, rows + 1, (count,), device="cuda", dtype=torch.int32)
        y = torch.full((count, cols), 7.0, dtype=SF, device="cuda")
        L.lct_tensor_rows(cb, t, index, y, L.alloc_rows(count), scale=0.5)
        same(y, looked_up(w, index, 0.5, SF))


def test_lookup_in_a_groups_member(L):
    """A member's rows, its spills in the group's shared region."""
    ns, lay = [5000, 301 * 64, 70_001], L.layout(4096, 2)
    xs = [(torch.randn(n, device="cuda") * 0.02).bfloat16() for n in ns]
    cbs = [L.lct_codebook_build(L.Model(0, 0.02, 0.0), x) for x in xs]
    g = L.LctGroup(ns, lay, cbs, xs)
    st = g.alloc_storage(sum(ns) + 3 * 4096)
    L.lct_encode_group(g, st)
    index = torch.randint(0, 301, (100,), device="cuda")
    y = torch.empty(4, 25, 64, dtype=SF, device="cuda")
    L.lct_tensor_rows(cbs[1], g.tensor(st, 1), index.view(4, 25), y)
    same(y.view(100, 64), looked_up(xs[1].view(301, 64), index, 1.0, SF))


def test_empty_lookups(L):
    w, cb, t = table(L, 10, 16, L.lct_layout_init(L.CLEAN))
    y = torch.empty(0, 16, dtype=BF, device="cuda")
    L.lct_tensor_rows(cb, t, torch.empty(0, dtype=torch.int64, device="cuda"), y)
    none = L.alloc_tensor(0, L.lct_layout_init(L.CLEAN))
    y = torch.full((3, 16), 7.0, device="cuda")
    L.lct_tensor_rows(cb, none, torch.tensor([0, -1, 5], device="cuda"), y)
    assert bool((y == 0).all())


# ------------------------------------------------------------------ gradient

def check_grad(g, index, dy, scale, before=None, what=""):
    rows, cols = g.shape
    inside = (index >= 0) & (index < rows)
    at = index[inside].long()
    d = dy.double().view(-1, cols)[inside]
    ref = torch.zeros(rows, cols, dtype=torch.float64, device="cuda").index_add_(0, at, d)
    mag = torch.zeros_like(ref).index_add_(0, at, d.abs()) * abs(scale)
    k = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones(at.numel(), dtype=torch.float64, device="cuda"))
    ref = ref * scale
    if before is not None:
        ref = ref + before.double()
        mag = mag + before.double().abs()
        untouched = k == 0
        assert torch.equal(g[untouched], before[untouched]), what
    fi = torch.finfo(g.dtype)
    off = (g.double() - ref).abs()
    tol = (k[:, None] + 2) * 2.0 ** -24 * mag
    tol = tol + (ref.abs() + tol) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2
    assert bool((off <= tol).all()), "%s: %g past the tolerance" % (what, float((off - tol).max()))


def zipf(count, rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(count, device="cuda", dtype=torch.float64, generator=g)
    return (torch.exp(u * np.log(rows + 1.0)) - 1).long().clamp(0, rows - 1)


@pytest.mark.parametrize("dtype,to", [(BF, BF), (SF, SF), (BF, SF), (SF, BF), (HF, HF), (HF, SF)])
@pytest.mark.parametrize("add", [False, True])
def test_grad_types_and_shapes(L, dtype, to, add):
    for rows, cols, count in ((1, 1, 1), (7, 3, 100), (1001, 131, 777), (513, 512, 64), (300, 513, 65), (5, 2560, 3000),
                              (70_000, 33, 2049)):
        index = zipf(count, rows, rows)
        if count > 10:
            index[::9] = -1
            index[4::17] = rows
        dy = (torch.randn(count, cols, device="cuda") * 0.1).to(dtype)
        before = torch.randn(rows, cols, device="cuda").to(to)
        g = before.clone()
        L.lct_rows_grad(index.int() if count % 2 else index, dy, g, L.alloc_rows(count, cols), scale=1.7, add=add)
        check_grad(g, index, dy, 1.7, before if add else None, "%d x %d, %d tokens" % (rows, cols, count))


@pytest.mark.parametrize("count", [1, 15, 16, 17, 255, 1023, 1024, 1025, 16_384, 16_385, 100_000])
def test_grad_counts(L, count):
    """Runs that lie in a tile of the sorted tokens, end at its border, and
    cross many; one token for all; every token another's row."""
    rows, cols = 211, 40
    for index in (zipf(count, rows, count), torch.full((count,), 17, device="cuda"),
                  torch.arange(count, device="cuda") % rows, torch.full((count,), rows - 1, device="cuda"),
                  torch.full((count,), -1, device="cuda"), torch.arange(count, device="cuda") // 16 % rows):
        dy = torch.randn(count, cols, device="cuda")
        g = torch.full((rows, cols), float("nan"), device="cuda")
        L.lct_rows_grad(index, dy, g, L.alloc_rows(count, cols))
        check_grad(g, index, dy, 1.0)


def test_grad_leaves_what_lies_beside_it(L):
    """Rows at odd places of one buffer, and scratch with a guard behind it."""
    rows, cols, count = 101, 37, 500
    for to in (BF, SF):
        flat = torch.full((rows * cols + 40,), 7.0, dtype=to, device="cuda")
        g = flat[3:3 + rows * cols].view(rows, cols)
        dyf = torch.randn(count * cols + 5, device="cuda").to(to)
        dy = dyf[5:].view(count, cols)
        index = zipf(count, rows, 1)
        work = L.alloc_rows(count, cols)
        need = work.scratch.numel()
        work.scratch = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        L.lct_rows_grad(index, dy, g, work)
        check_grad(g, index, dy, 1.0)
        assert bool((flat[:3] == 7.0).all() and (flat[3 + rows * cols:] == 7.0).all())
        assert bool((work.scratch[need:] == 0x5A).all())


def test_grad_of_infinite_and_nan_values(L):
    """They reach the rows of their tokens and no other."""
    rows, cols = 50, 24
    index = torch.tensor([3, 3, 9, -1, 20], device="cuda")
    dy = torch.ones(5, cols, device="cuda")
    dy[0, 0], dy[1, 1], dy[2, 2], dy[3, 3] = float("nan"), float("inf"), -float("inf"), float("nan")
    g = torch.empty(rows, cols, device="cuda")
    L.lct_rows_grad(index, dy, g, L.alloc_rows(5, cols))
    ref = torch.zeros(rows, cols, device="cuda").index_add_(0, index[[0, 1, 2, 4]], dy[[0, 1, 2, 4]])
    assert torch.equal(torch.nan_to_num(g, 5.0, 6.0, 7.0), torch.nan_to_num(ref, 5.0, 6.0, 7.0))


def test_grad_of_nothing(L):
    g = torch.full((5, 8), 3.0, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    L.lct_rows_grad(none, torch.empty(0, 8, device="cuda"), g, L.alloc_rows(0, 8), add=True)
    assert bool((g == 3.0).all())
    L.lct_rows_grad(none, torch.empty(0, 8, device="cuda"), g, L.alloc_rows(0, 8))
    assert bool((g == 0.0).all())


def test_grad_repeats_bit_for_bit_and_beside_another(L):
    """Two calls that overlap in time on two streams, twenty times."""
    rows, cols, count = 3001, 520, 9000
    cases = []
    for s in range(2):
        index, dy = zipf(count, rows, s), torch.randn(count, cols, device="cuda").bfloat16()
        g, work = torch.empty(rows, cols, dtype=BF, device="cuda"), L.alloc_rows(count, cols)
        L.lct_rows_grad(index, dy, g, work)
        cases.append((index, dy, g, work, g.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for index, dy, g, work, _, st in cases:
            with torch.cuda.stream(st):
                g.fill_(5.0)
            L.lct_rows_grad(index, dy, g, work, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[2], c[4])


def test_table_gradient_by_differences(L):
    """The loss sum(y * dy) is linear in W: its change over a change of one
    element is the gradient's element, times the change."""
    rows, cols, count = 40, 48, 200
    lay = L.lct_layout_init(L.CLEAN)
    w, cb, t = table(L, rows, cols, lay, 8)
    index = zipf(count, rows, 2)
    dy = torch.randn(count, cols, device="cuda")
    g = torch.empty(rows, cols, device="cuda")
    L.lct_rows_grad(index, dy, g, L.alloc_rows(count, cols), scale=3.0)

    def loss(values):
        y = torch.empty(count, cols, device="cuda")
        L.lct_tensor_rows(cb, L.encode(cb, values.view(-1), lay), index, y, scale=3.0)
        return float((y.double() * dy.double()).sum())

    for v, c in ((0, 0), (1, 47), (5, 13), (39, 2)):
        up = w.clone()
        up[v, c] += 0.25
        h = float(up[v, c].double() - w[v, c].double())
        # (the products y are rounded to fp32: 2^-24 of each of the row's terms)
        k = int((index == v).sum())
        tol = (2 * k + 4) * 2.0 ** -24 * 3.0 * float(dy[index == v, c].abs().sum() + 1e-9) * (1 + 0.3 / abs(h))
        assert abs((loss(up) - loss(w)) / h - float(g[v, c])) <= tol + 1e-9


def test_rows_and_grad_from_a_graph(L):
    """Replays with other tokens and gradients equal the eager calls, with eager
    work on the same buffers between them."""
    rows, cols, count = 2003, 384, 3000
    w, cb, t = table(L, rows, cols, L.lct_layout_init(L.CLEAN), 4)
    index, dy = zipf(count, rows, 0), torch.randn(count, cols, device="cuda").bfloat16()
    y, g = torch.empty(count, cols, dtype=BF, device="cuda"), torch.empty(rows, cols, dtype=BF, device="cuda")
    work = L.alloc_rows(count, cols)

    def run():
        L.lct_tensor_rows(cb, t, index, y, work, scale=2.0)
        L.lct_rows_grad(index, dy, g, work, scale=2.0)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(4):
        index.copy_(zipf(count, rows, 10 + rep))
        dy.copy_(torch.randn(count, cols, device="cuda"))
        run()
        want = y.clone(), g.clone()
        y.zero_()
        g.fill_(9.0)
        work.scratch.fill_(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(g, want[1]), rep
