"""What the binding's objects keep between calls (no GPU): the addresses that
reach the library are those of the memory that a result or a tensor has when a
call is made, and copies and pickles have memory of their own.  Buffers are CPU
tensors that say they are on the GPU; the library's calls are recorded, not
made."""
import copy
import gc
import pickle

import pytest
import torch

U8, F32 = torch.uint8, torch.float32


class OnGpu(torch.Tensor):
    """A CPU tensor for the binding's checks of its place."""
    is_cuda = True

    def __deepcopy__(self, memo):
        return gpu(self.as_subclass(torch.Tensor).clone())

    def __reduce_ex__(self, proto):
        return gpu, (self.as_subclass(torch.Tensor).clone(),)


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def L(monkeypatch):
    import lossless_bf16_tensor_split_amd as L
    monkeypatch.setattr(L, "_current", lambda dev, what: None)
    monkeypatch.setattr(L, "_stream", lambda stream=None: None)
    return L


class Calls:
    """The (scratch, each, result) addresses of the norm calls made."""

    def __init__(self, L, monkeypatch):
        self.seen = []

        def norm(x, kind, mx, sc, scratch, each, res, stream):
            self.seen.append((scratch, each, res))
            return 0

        monkeypatch.setattr(L.lib, "lct_list_norm", norm)

    def last(self):
        return self.seen[-1]


@pytest.fixture
def calls(L, monkeypatch):
    return Calls(L, monkeypatch)


def result(L, members, each=True, scratch=None):
    need = L._norm_scratch(members, 0)
    out = L.LctNorm(members, 0, False, "cpu", gpu(torch.zeros(need if scratch is None else scratch, dtype=U8)))
    if each:
        out.each = gpu(torch.zeros(members))
    return out


def listed(L, count):
    """A list of so many (empty) tensors."""
    x = L.LctList([])
    x.count, x.need = count, L._norm_scratch(count, 0)
    return x


def addresses(out):
    return out.scratch.data_ptr(), None if out.each is None else out.each.data_ptr(), out.buf.data_ptr()


def test_a_call_gets_the_memory_that_the_result_has(L, calls):
    out = result(L, 3)
    L.lct_list_norm(listed(L, 3), out)
    first = addresses(out)
    assert calls.last() == first
    # each replaced, turned off, and put back
    out.each = gpu(torch.zeros(3))
    L.lct_list_norm(listed(L, 3), out)
    assert calls.last() == addresses(out) and out.each.data_ptr() != first[1]
    out.each = None
    L.lct_list_norm(listed(L, 3), out)
    assert calls.last() == (first[0], None, first[2])
    L.lct_list_norm(listed(L, 192), out)          # (the same scratch does for 192)
    assert calls.last()[1] is None
    out.each = gpu(torch.zeros(192))
    L.lct_list_norm(listed(L, 192), out)
    assert calls.last() == addresses(out)
    with pytest.raises(ValueError, match="each has room for 192"):
        L.lct_list_norm(listed(L, 3), out)
    # other memory behind the same tensors
    out.each.set_(gpu(torch.zeros(192)))
    out.scratch.set_(gpu(torch.zeros_like(out.scratch)))
    L.lct_list_norm(listed(L, 192), out)
    assert calls.last() == addresses(out) and out.scratch.data_ptr() != first[0]
    out.scratch.data = gpu(torch.zeros_like(out.scratch))
    L.lct_list_norm(listed(L, 192), out)
    assert calls.last() == addresses(out)


def test_memory_that_became_too_small_is_refused(L, calls):
    x = listed(L, 5)
    out = result(L, 5)
    out.each.set_(gpu(torch.zeros(4)))
    with pytest.raises(ValueError, match="each has room for 4"):
        L.lct_list_norm(x, out)
    out = result(L, 5)
    out.scratch.data = gpu(torch.zeros(64, dtype=U8))
    with pytest.raises(ValueError, match="scratch holds 64"):
        L.lct_list_norm(x, out)
    for what in ("each", "scratch"):
        out = result(L, 5)
        getattr(out, what).untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="memory of %s" % what):
            L.lct_list_norm(x, out)
    for other in (torch.zeros(16, dtype=U8), torch.zeros(4, dtype=U8)):
        out = result(L, 5)
        out.buf.set_(other)
        with pytest.raises(ValueError, match="buf"):
            L.lct_list_norm(x, out)
        with pytest.raises(ValueError, match="buf"):
            L.lct_norm_join(torch.zeros(2, 16, dtype=U8), out)
    assert not calls.seen


def test_memory_in_use_is_held(L, calls):
    """An address that did not change is the memory it was: what a tensor had
    at the last look cannot have been handed to another one meanwhile."""
    out = result(L, 5)
    at = addresses(out)
    out.scratch.data = gpu(torch.zeros(8, dtype=U8))
    out.each.data = gpu(torch.zeros(1))
    gc.collect()
    later = [gpu(torch.zeros(k, dtype=U8)) for k in (L._norm_scratch(5, 0), 20) for _ in range(50)]
    assert not {t.data_ptr() for t in later} & set(at)


def test_results_take_what_fits_only(L):
    out = result(L, 3)
    for bad in (torch.zeros(3, dtype=torch.float64), torch.zeros(1, 3)):
        with pytest.raises(TypeError, match="each"):
            out.each = gpu(bad)
    with pytest.raises(ValueError, match="on the GPU"):
        out.each = torch.zeros(3)
    with pytest.raises(ValueError, match="contiguous"):
        out.each = gpu(torch.zeros(6)[::2])
    with pytest.raises(AttributeError):
        out.buf = torch.zeros(16, dtype=U8)


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_copies_of_a_result(L, calls, how):
    """A deep copy or a pickle writes to its own memory, and its views show
    it; a shallow copy shares the tensors."""
    out = result(L, 3)
    out.buf.zero_()                              # (a result is unset until its first call)
    out.norm.fill_(2.5)
    if how == "copy":
        b = copy.copy(out)
    elif how == "deepcopy":
        b = copy.deepcopy(out)
    else:
        b = pickle.loads(pickle.dumps(out))
    assert float(b.norm) == 2.5 and b.members == 3
    L.lct_list_norm(listed(L, 3), b)
    assert calls.last() == addresses(b)
    own = how != "copy"
    assert all((p != q) == own for p, q in zip(addresses(b), addresses(out)))
    b.buf.view(F32)[3] = 0.125                   # what a call would leave in coef
    assert float(b.coef) == 0.125 and (float(out.coef) == 0.125) == (not own)


def test_results_of_another_kind_are_not_joined(L, calls, monkeypatch):
    """A sum of squares and a largest magnitude have no norm together."""
    joined = []
    monkeypatch.setattr(L.lib, "lct_norm_join", lambda parts, count, kind, *a: joined.append((count, kind)) or 0)
    a, b, c = result(L, 3), result(L, 3), result(L, 3)
    L.lct_list_norm(listed(L, 3), a, kind=L.NORM_L2)
    L.lct_list_norm(listed(L, 3), b, kind=L.NORM_MAX)
    assert (a.kind, b.kind, c.kind) == (L.NORM_L2, L.NORM_MAX, None)
    for parts, kind in (((a, b), L.NORM_L2), ((a, b), L.NORM_MAX), ((a,), L.NORM_MAX), ((c, b), L.NORM_L2)):
        with pytest.raises(ValueError, match="part"):
            L.lct_norm_join(parts, result(L, 0), kind=kind)
    assert not joined
    out = result(L, 0)
    L.lct_norm_join([a, copy.deepcopy(a), c], out)       # (c was filled by other means)
    L.lct_norm_join([b], out, kind=L.NORM_MAX)
    L.lct_norm_join(torch.zeros(2, 16, dtype=U8), out)
    assert joined == [(3, L.NORM_L2), (1, L.NORM_MAX), (2, L.NORM_L2)] and out.kind == L.NORM_L2


# ------------------------------------------------------------------ compressed tensors

def coded(L, n=70000):
    """A compressed tensor with made-up contents."""
    t = L.alloc_tensor(n, L.layout(65536, 25), device="cpu")
    for k, name in enumerate(("sf", "pay", "cnt", "obase", "ovf", "status", "scratch")):
        b = getattr(t, name)
        setattr(t, name, gpu(b.fill_(k)))
    return t


BUFFERS = ("sf", "pay", "cnt", "obase", "ovf", "status", "scratch")


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_copies_of_a_tensor_that_was_used(L, how):
    """A tensor is copied and saved after a call as before its first one, and
    the copy's descriptor is of the copy's buffers."""
    t = coded(L)
    a = t.c()
    b = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda v: pickle.loads(pickle.dumps(v))}[how](t)
    assert (b.n, b.ovf_cap) == (t.n, t.ovf_cap) and bytes(b.sizes) == bytes(t.sizes)
    assert bytes(b.layout) == bytes(t.layout)
    c = b.c()
    for name in BUFFERS:
        x, y = getattr(t, name), getattr(b, name)
        assert torch.equal(x, y) and getattr(c, name) == y.data_ptr() and getattr(a, name) == x.data_ptr()
        assert (x.data_ptr() == y.data_ptr()) == (how == "copy")
    assert t.c() is a                            # the original's is kept still


def test_a_kept_descriptor_follows_the_tensors_numbers(L):
    """Changed in place, they reach the next call, as they did before
    descriptors were kept; an edited descriptor is not given out again."""
    t = coded(L)
    a = t.c()
    assert t.c() is a
    t.layout.cap_words = 12
    assert t.c().layout.cap_words == 12 and t.c() is t.c()
    t.layout.block_elems = 32768
    assert t.c().layout.block_elems == 32768
    t.c().ovf_cap = 0
    t.c().pay = None
    assert t.c().ovf_cap == t.ovf_cap and t.c().pay == t.pay.data_ptr()


def test_a_kept_descriptor_follows_the_sizes_of_buffers(L):
    t = coded(L)
    t.c()
    t.sf.resize_(t.n - 1)                        # the same memory, shorter
    with pytest.raises(ValueError, match="sf"):
        t.c()
    t = coded(L)
    t.c()
    t.pay.set_(gpu(t.pay[:-4].clone()))
    with pytest.raises(ValueError, match="pay"):
        t.c()


def test_a_kept_descriptor_follows_replaced_and_missing_buffers(L):
    t = coded(L)
    for name in ("status", "scratch", "ovf"):
        old = getattr(t, name)
        assert getattr(t.c(), name) == old.data_ptr()
        setattr(t, name, gpu(old.clone()))
        assert getattr(t.c(), name) == getattr(t, name).data_ptr() != old.data_ptr()
        del old
        setattr(t, name, None)                   # (the last reference to it)
        assert getattr(t.c(), name) is None and t.c() is t.c()
        setattr(t, name, gpu(torch.zeros(t.sizes.scratch + t.ovf_cap, dtype=U8)))
        assert getattr(t.c(), name) == getattr(t, name).data_ptr()
