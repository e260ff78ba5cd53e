"""Copies, pickles and replaced buffers of the binding's objects on the GPU:
calls on a copy leave the original alone, and nothing is written to memory that
a result no longer has."""
import copy
import pickle

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


def copies(v):
    return [copy.deepcopy(v), pickle.loads(pickle.dumps(v))]


def test_a_norm_on_a_copied_result(L):
    a = L.LctList([torch.full((300,), 2.0, device="cuda"), torch.full((100,), 1.0, device="cuda")])
    b = L.LctList([torch.full((1 << 20,), 0.5, dtype=BF, device="cuda"), torch.zeros(7, device="cuda")])
    out = L.alloc_norm(2, True)
    L.lct_list_norm(a, out, 1.0)
    torch.cuda.synchronize()
    before, each = out.buf.clone(), out.each.clone()
    for c in copies(out):
        assert torch.equal(c.buf, before) and torch.equal(c.each, each) and c.kind == L.NORM_L2
        L.lct_list_norm(b, c, 1.0)
        torch.cuda.synchronize()
        assert float(c.norm) == 512.0 and c.each.tolist() == [512.0, 0.0]
        assert torch.equal(out.buf, before) and torch.equal(out.each, each)
        L.lct_norm_join([out, c], c)
        torch.cuda.synchronize()
        assert float(c.sum) == 300 * 4.0 + 100.0 + 512.0 ** 2


def test_each_turned_off_and_replaced(L):
    """The memory that each had is another tensor's: it stays as it was."""
    xs = [torch.full((5,), float(k), device="cuda") for k in range(192)]
    guard = torch.full((4096,), -7.0, device="cuda")
    out = L.alloc_norm(3, True)
    out.each = guard[64:67]
    L.lct_list_norm(L.LctList(xs[:3]), out, kind=L.NORM_MAX)
    torch.cuda.synchronize()
    assert guard[64:67].tolist() == [0.0, 1.0, 2.0]
    guard.fill_(-7.0)
    out.each = None
    L.lct_list_norm(L.LctList(xs), out, kind=L.NORM_MAX)
    torch.cuda.synchronize()
    assert float(out.norm) == 191.0 and bool((guard == -7.0).all())
    out.each = guard[128:320]
    L.lct_list_norm(L.LctList(xs), out, kind=L.NORM_MAX)
    torch.cuda.synchronize()
    assert guard[128:320].tolist() == [float(k) for k in range(192)]
    assert bool((guard[:128] == -7.0).all()) and bool((guard[320:] == -7.0).all())


def test_steps_on_copied_tensors(L):
    """Tensors that took part in a step are copied and pickled; the copies
    decode to the same values and are updated apart from the originals."""
    n = 70001
    w = (torch.randn(n, device="cuda") * 0.02).to(BF)
    m = (torch.randn(n, device="cuda") * 1e-3).to(BF)
    lay = L.layout(4096, 25)
    cw, cm = (L.lct_codebook_build(L.Model(L.GAUSSIAN, s, 0.0), x) for s, x in ((0.02, w), (1e-3, m)))
    tw, tm, to = L.encode(cw, w, lay), L.encode(cm, m, lay), L.alloc_tensor(n, lay)
    L.lct_sgd_step(cw, tw, cm, tm, 0.5, to)
    want = L.decode(cw, to)
    for c in copies(tw):
        assert torch.equal(L.decode(cw, c), w)
        o = L.alloc_tensor(n, lay)
        L.lct_sgd_step(cw, c, cm, tm, 0.5, o)
        assert torch.equal(L.decode(cw, o), want)
        L.lct_encode(cw, torch.zeros_like(w), c)
        assert torch.equal(L.decode(cw, tw), w) and not bool(L.decode(cw, c).any())
