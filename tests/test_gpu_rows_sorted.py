"""Lookups that take the sorted kernel, seen by what they leave in the working
memory (the kernel in the indices' order leaves it alone): workgroups of every
number of tokens, rows longer than a workgroup's room, every type; tables of
more rows than two passes of the sort can tell apart; offsets past 32 bits.
Tolerances are those of the tests of the same calls: lookups bit for bit."""
import pytest
import torch

from test_gpu_rows import check_grad, looked_up, same, table, zipf

pytestmark = pytest.mark.gpu
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


def sorted_lookup(L, cb, t, index, y, scale):
    """A lookup, once it is seen that it took the sorted kernel."""
    work = L.alloc_rows(index.numel())
    work.scratch.fill_(0xA5)
    L.lct_tensor_rows(cb, t, index, y, work, scale=scale)
    assert not bool((work.scratch[:4 * index.numel()] == 0xA5).all()), "took the kernel in the indices' order"


# (the room is 12288 exponents: 16, 8, 4, 2 and 1 tokens to a workgroup, then pieces)
@pytest.mark.parametrize("cols", [1, 331, 768, 769, 1500, 2560, 6000, 9001, 12_288, 12_289, 20_000, 70_001])
@pytest.mark.parametrize("B,cw", [(65536, 25), (4096, 2)])
def test_widths(L, cols, B, cw):
    """Every row several times, in no order, with padding: neighbours that share
    a block, rows that end within the position where the next begins, rows over
    several blocks, spills."""
    rows = max(3, 250_000 // cols)
    w, cb, t = table(L, rows, cols, L.layout(B, cw), cols)
    count = max(4097, 2 * (-(-rows * cols // B)) + 1)
    g = torch.Generator(device="cuda").manual_seed(cols)
    index = torch.randint(-1, rows + 1, (count,), device="cuda", generator=g)
    index[:3] = torch.tensor([0, rows - 1, 2 ** 40])
    for dtype, scale in ((BF, 50.5964), (HF, 3.0), (SF, 0.1)):
        y = torch.full((count, cols), 7.0, dtype=dtype, device="cuda")
        sorted_lookup(L, cb, t, index if dtype != HF else index.clamp(-1, rows).int(), y, scale)
        same(y, looked_up(w, index, scale, dtype), "%s" % dtype)


@pytest.mark.parametrize("count", [4096, 4097, 65_536, 65_537, 200_000])
def test_counts_and_odd_places(L, count):
    """A frequent row fills whole workgroups; few rows in all; an output at an
    odd place leaves what lies beside it."""
    rows, cols = 501, 37
    w, cb, t = table(L, rows, cols, L.lct_layout_init(L.CLEAN), 3)
    for index in (zipf(count, rows, count), torch.full((count,), 17, device="cuda"),
                  torch.full((count,), -1, device="cuda"), torch.arange(count, device="cuda") % rows):
        flat = torch.full((count * cols + 9,), 7.0, dtype=BF, device="cuda")
        y = flat[3:3 + count * cols].view(count, cols)
        sorted_lookup(L, cb, t, index, y, 2.5)
        same(y, looked_up(w, index, 2.5, BF))
        assert bool((flat[:3] == 7.0).all() and (flat[3 + count * cols:] == 7.0).all())


def test_empty_table(L):
    """Every index is outside it."""
    lay = L.lct_layout_init(L.CLEAN)
    cb, none = L.lct_codebook_build(L.Model(0, 0.02, 0.0), None), L.alloc_tensor(0, lay)
    for count in (4096, 5000):
        y = torch.full((count, 16), 7.0, device="cuda")
        sorted_lookup(L, cb, none, torch.arange(count, device="cuda") % 7 - 3, y, 1.0)
        assert bool((y == 0).all())


def test_a_groups_member(L):
    """Spills in the group's shared region."""
    ns, lay = [5000, 301 * 640, 70_001], L.layout(4096, 2)
    xs = [(torch.randn(n, device="cuda") * 0.02).bfloat16() for n in ns]
    cbs = [L.lct_codebook_build(L.Model(0, 0.02, 0.0), x) for x in xs]
    g = L.LctGroup(ns, lay, cbs, xs)
    st = g.alloc_storage(sum(ns) + 3 * 4096)
    L.lct_encode_group(g, st)
    index = zipf(5000, 301, 4)
    y = torch.empty(5000, 640, dtype=SF, device="cuda")
    sorted_lookup(L, cbs[1], g.tensor(st, 1), index, y, 1.0)
    same(y, looked_up(xs[1].view(301, 640), index, 1.0, SF))


@pytest.mark.parametrize("count", [5000, 70_000])
def test_from_a_graph(L, count):
    """The sort and the lookup replayed with other tokens, with eager work on
    the same memory between the replays."""
    rows, cols = 2003, 384
    w, cb, t = table(L, rows, cols, L.lct_layout_init(L.CLEAN), 4)
    index, y = zipf(count, rows, 0), torch.empty(count, cols, dtype=BF, device="cuda")
    work = L.alloc_rows(count)
    L.lct_tensor_rows(cb, t, index, y, work, scale=2.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lct_tensor_rows(cb, t, index, y, work, scale=2.0)
    for rep in range(4):
        index.copy_(zipf(count, rows, 10 + rep))
        y.zero_()
        work.scratch.fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not bool((work.scratch[:4 * count] == 0xA5).all())
        same(y, looked_up(w, index, 2.0, BF), "replay %d" % rep)
        L.lct_tensor_rows(cb, t, index.flip(0).contiguous(), y, work, scale=1.0)


# rows whose numbers take three and four passes of nine bits, and the border of two
@pytest.mark.parametrize("rows", [(1 << 18) - 1, 1 << 18, (1 << 18) + 7, (1 << 27) + 5])
@pytest.mark.parametrize("count", [4096, 5001, 140_000])
def test_sorts_of_many_rows(L, rows, count):
    """Numbers over the whole range, neighbours, and repeats, in no order: the
    gradient of each row, and (where there are tokens enough for it) its lookup."""
    g = torch.Generator(device="cuda").manual_seed(count)
    index = torch.randint(0, rows, (count,), device="cuda", generator=g)
    index[::3] = (index[::3] >> 9 << 9) % rows
    index[1::5] = torch.randint(0, 1500, (index[1::5].numel(),), device="cuda", generator=g)
    index[::11], index[7::500], index[8::500] = -1, rows, rows - 1
    dy = torch.randn(count, 1, device="cuda", generator=g)
    out = torch.full((rows, 1), float("nan"), device="cuda")
    L.lct_rows_grad(index, dy, out, L.alloc_rows(count, 1))
    check_grad(out, index, dy, 1.0)
    del out
    lay = L.lct_layout_init(L.CLEAN)
    if count >= 2 * -(-rows // lay.block_elems):
        w, cb, t = table(L, rows, 1, lay, 1)
        y = torch.full((count, 1), 7.0, dtype=BF, device="cuda")
        sorted_lookup(L, cb, t, index, y, 1.0)
        same(y, looked_up(w, index, 1.0, BF))


def test_offsets_past_32_bits(L):
    """A table of more than 2^32 elements: rows from its end, sorted and in
    order, its gradient, and a mix of it."""
    rows, cols, lay = 2_100_001, 2049, L.lct_layout_init(L.CLEAN)
    n = rows * cols
    assert n > 1 << 32
    w = torch.empty(n, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in range(0, n, 1 << 28):
        m = min(1 << 28, n - at)
        w[at:at + m] = torch.randn(m, device="cuda", generator=g).mul_(0.02)
    cb = L.lct_codebook_build(L.Model(0, 0.02, 0.0), w)
    t = L.encode(cb, w, lay, n // 8)
    assert t.status_word() == 0
    last = torch.arange(rows - 40, rows, device="cuda")
    some = torch.randint(0, rows, (2 * (n // 65536) + 5000,), device="cuda", generator=g)
    for index, call in ((torch.cat([last, last[:3], some[:20]]), L.lct_tensor_rows), (torch.cat([some, last]), None)):
        y = torch.empty(index.numel(), cols, dtype=BF, device="cuda")
        if call:
            call(cb, t, index, y)
        else:
            sorted_lookup(L, cb, t, index, y, 1.0)
        for k in range(0, index.numel(), 20_000):
            i = index[k:k + 20_000]
            same(y[k:k + 20_000], w.view(rows, cols).index_select(0, i), "rows")
    # the mix: 0.5 w + (0.25 * 0.5) x, every product exact, so the sum is rounded once to fp32 and once to BF16
    x, o = w.flip(0).contiguous(), L.alloc_tensor(n, lay, n // 8)
    L.lct_mix_step(cb, t, 0.5, x, 0.25, o, torch.tensor(0.5, device="cuda"), x, False)
    assert o.status_word() == 0
    v = L.decode(cb, o)
    for at in (0, (1 << 31) - 5, (1 << 32) - 70_000, n - 300_000):
        s = slice(at, min(n, at + 300_000))
        want = (0.5 * w[s].float() + 0.125 * w[n - s.stop:n - s.start].flip(0).float()).to(BF)
        assert torch.equal(v[s].view(torch.int16), want.view(torch.int16)), at
        assert torch.equal(x[s].view(torch.int16), want.view(torch.int16)), at
    del v, o, x, t
    # the gradient over the table's values: rows with tokens, and others cleared
    index = torch.cat([last, last, some[:3000]])
    dy = torch.randn(index.numel(), cols, device="cuda", generator=g).to(BF)
    L.lct_rows_grad(index, dy, w.view(rows, cols), L.alloc_rows(index.numel(), cols))
    have = torch.unique(index)
    small = torch.searchsorted(have, index)
    check_grad(w.view(rows, cols).index_select(0, have), small, dy, 1.0)
    none = torch.ones(rows, dtype=torch.bool, device="cuda")
    none[have] = False
    for k in range(0, rows, 200_000):
        assert not bool(w.view(rows, cols)[k:k + 200_000][none[k:k + 200_000]].any()), k
