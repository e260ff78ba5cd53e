"""A training step over parameters that stay compressed, as a program makes it:
matrices by momentum (mix), orthogonalisation and weight step (mix), a token
table by lookup, loss, gradient and momentum step.  Every stage against its plain
form on the values that the stage before left."""
import numpy as np
import pytest
import torch

from test_gpu_mix import bits, mixed
from test_gpu_ortho import check
from test_gpu_parity import dev
from test_gpu_rows import check_grad, looked_up, same, zipf

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [(256, 700), (513, 130), (300, 300)]
MU, ETA, DECAY = 0.95, 0.02, 0.1


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_bf16_tensor_split_amd as L
    return L


class Matrices:
    """Weights and momentum as codes, one dense buffer per matrix that holds the
    gradient, then the momentum looked ahead, then the orthogonal update."""

    def __init__(self, L, seed):
        self.L, lay = L, L.lct_layout_init(L.CLEAN)
        ns = [m * n for m, n in SHAPES]
        torch.manual_seed(seed)
        self.w = [(torch.randn(n, device="cuda") * 0.02).to(BF) for n in ns]
        self.m = [(torch.randn(n, device="cuda") * 1e-3).to(BF) for n in ns]
        self.g = [torch.zeros(n, dtype=BF, device="cuda") for n in ns]
        cw = [L.lct_codebook_build(L.Model(0, 0.02, 0.0), w) for w in self.w]
        cm = [L.lct_codebook_build(L.Model(0, 1e-3, 0.0), m) for m in self.m]
        self.gw, self.gm = L.LctGroup(ns, lay, cw, self.w), L.LctGroup(ns, lay, cm, self.m)
        self.gg = L.LctGroup(ns, lay, cm, self.g)
        cap = sum(ns) // 4 + 65536
        self.wc, self.mc = self.gw.alloc_storage(cap), self.gm.alloc_storage(cap)
        self.wo, self.mo = self.gw.alloc_storage(cap), self.gm.alloc_storage(cap)
        L.lct_encode_group(self.gw, self.wc)
        L.lct_encode_group(self.gm, self.mc)
        self.mats = L.LctMatrices([g.view(s) for g, s in zip(self.g, SHAPES)])
        self.work = L.alloc_orthogonal(self.mats)
        self.norm = L.alloc_norm(len(ns))
        self.list = L.LctList(self.g)
        self.scale = [0.2 * max(s) ** 0.5 for s in SHAPES]

    def fill(self, seed):
        torch.manual_seed(seed)
        for g in self.g:
            g.copy_(torch.randn(g.numel(), device="cuda") * 1e-2)

    def ahead(self):
        self.L.lct_list_norm(self.list, self.norm, max_norm=1.0)
        self.L.lct_mix_step_group(self.gm, self.mc, MU, self.gg, 1.0, self.mo, self.norm, self.gg, True)

    def update(self):
        self.L.lct_list_orthogonalize(self.mats, self.mats, self.work, scale=self.scale)
        self.L.lct_mix_step_group(self.gw, self.wc, 1 - ETA * DECAY, self.gg, -ETA, self.wo)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.wo.sf, self.wo.pay, self.wo.cnt, self.mo.sf, self.mo.pay, self.mo.cnt, *self.g)]

    def wipe(self):
        for t in (self.wo.pay, self.wo.cnt, self.mo.pay, self.mo.cnt):
            t.zero_()


def test_matrices_stage_by_stage(L, orc):
    s = Matrices(L, 1)
    s.fill(2)
    g = [t.clone() for t in s.g]
    s.ahead()
    c = float(s.norm.coef)
    assert 0 < c < 1
    u = [t.clone() for t in s.g]
    for k in range(len(SHAPES)):
        v, a = mixed(orc, bits(s.m[k]), bits(g[k]), MU, 1.0, c)
        assert np.array_equal(bits(L.decode(s.gm.codebooks[k], s.gm.tensor(s.mo, k))), v), k
        assert np.array_equal(bits(u[k]), a), k
    s.update()
    for k, shape in enumerate(SHAPES):
        check(s.g[k].view(shape), u[k].view(shape), 5, L.NEWTON_SCHULZ, s.scale[k])
        v, _ = mixed(orc, bits(s.w[k]), bits(s.g[k]), 1 - ETA * DECAY, -ETA, 1.0)
        assert np.array_equal(bits(L.decode(s.gw.codebooks[k], s.gw.tensor(s.wo, k))), v), k


def test_matrices_replayed_from_a_graph(L):
    s, other = Matrices(L, 3), Matrices(L, 4)
    other.fill(1)
    s.fill(5)
    s.ahead()
    s.update()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.ahead()
        s.update()
    for rep in range(4):
        s.fill(10 + rep)
        s.wipe()
        s.ahead()
        s.update()
        want = s.results()
        s.fill(10 + rep)
        s.wipe()
        other.ahead()
        other.update()
        torch.cuda.synchronize()
        graph.replay()
        for k, (a, b) in enumerate(zip(want, s.results())):
            assert torch.equal(a, b), (rep, k)


def test_token_table_step(L, orc):
    """Lookup, a loss whose gradient autograd makes, the table's gradient, and
    the momentum step on it; tied weights add the head's gradient first."""
    rows, cols, count = 1501, 192, 3000
    lay = L.lct_layout_init(L.CLEAN)
    torch.manual_seed(7)
    w = (torch.randn(rows * cols, device="cuda") * 0.02).to(BF)
    m = (torch.randn(rows * cols, device="cuda") * 1e-3).to(BF)
    cw, cm = (L.lct_codebook_build(L.Model(0, s, 0.0), t) for s, t in ((0.02, w), (1e-3, m)))
    tw, tm = L.encode(cw, w, lay), L.encode(cm, m, lay)
    index = zipf(count, rows, 1)
    index[::31] = -1
    work = L.alloc_rows(count, cols)
    y = torch.empty(count, cols, dtype=BF, device="cuda")
    L.lct_tensor_rows(cw, tw, index, y, work, scale=cols ** 0.5)
    same(y, looked_up(w.view(rows, cols), index, cols ** 0.5, BF))
    y.requires_grad_(True)
    head = torch.randn(cols, 5, device="cuda")
    (torch.tanh(y.float() @ head) ** 2).mean().backward()
    g = torch.randn(rows, cols, device="cuda").mul_(1e-3).to(BF)     # the head's
    before = g.clone()
    L.lct_rows_grad(index, y.grad, g, work, scale=cols ** 0.5, add=True)
    check_grad(g, index, y.grad, cols ** 0.5, before)
    ow, om = L.momentum_step(cw, tw, cm, tm, g.view(-1), 0.9, 0.1)
    wo, mo = orc.momentum_dense(bits(w), bits(m), bits(g.view(-1)), 0.9, 0.1)
    assert np.array_equal(bits(L.decode(cw, ow)), wo) and np.array_equal(bits(L.decode(cm, om)), mo)
