"""A GradList and tensors that change under it, on the host alone: a list holds
addresses, sizes and types, and a call on it must use those that its tensors
have now. The tensors are host tensors that pass for GPU ones: nothing here
launches a kernel."""

import pytest
import torch

from helpers import ensure_built


@pytest.fixture(scope="module")
def B():
    ensure_built()
    from precision_moe_numerics_nvfp4_amd import binding
    return binding


class _Posing(torch.Tensor):
    is_cuda = property(lambda self: True)


def _ts(*sizes):
    return [torch.zeros(n).as_subclass(_Posing) for n in sizes]


def _seen(h):
    h = h.current()
    return [(p, n, c) for p, n, c in zip(h.ptrs, h.numels, h.codes)]


def test_shorter_prefix_of_its_own_memory(B):
    """Same address, fewer elements: those behind are another's."""
    ts = _ts(100, 7)
    h = B.GradList(ts)
    at = ts[0].data_ptr()
    ts[0].data = ts[0].data[:40]
    assert ts[0].data_ptr() == at
    assert _seen(h) == [(at, 40, 0), (ts[1].data_ptr(), 7, 0)]
    assert h.sizes == [40, 7] and h.spans == sorted([(at, at + 160), (ts[1].data_ptr(), ts[1].data_ptr() + 28)])


def test_longer_again(B):
    whole = torch.zeros(100)
    t = whole[:40].as_subclass(_Posing)
    h = B.GradList([t])
    t.data = whole[:100]
    assert _seen(h) == [(whole.data_ptr(), 100, 0)]


def test_workspace_follows_the_sizes(B):
    whole = torch.zeros(1 << 20)
    t = whole[:4].as_subclass(_Posing)
    h = B.GradList([t])
    assert h.workspace_size == 0
    t.data = whole
    assert B.grad_workspace_size(h) == B.GradList([whole.as_subclass(_Posing)]).workspace_size > 0


def test_other_type_of_the_same_address(B):
    """As many elements of half the size, and the same bytes as twice as many."""
    for view in (lambda m: m.view(torch.bfloat16)[:100], lambda m: m.view(torch.bfloat16)):
        m = torch.zeros(100)
        t = m.as_subclass(_Posing)
        h = B.GradList([t])
        t.data = view(m)
        assert _seen(h) == [(m.data_ptr(), t.numel(), B.NVFP4MOE_BF16)]
    t.data = m.view(torch.int32)
    with pytest.raises(ValueError):
        h.current()
    with pytest.raises(ValueError):                       # and again: nothing half taken over
        h.current()


def test_other_strides_of_the_same_address(B):
    """As many elements of the type, but not one behind the other."""
    m = torch.zeros(200)
    t = m[:100].as_subclass(_Posing)
    h = B.GradList([t])
    t.data = m[::2]
    with pytest.raises(ValueError):
        h.current()
    t.data = m[:100]
    assert _seen(h) == [(m.data_ptr(), 100, 0)]


def test_resized_in_place(B):
    t = torch.zeros(100).as_subclass(_Posing)
    h = B.GradList([t])
    t.resize_(10)
    assert _seen(h) == [(t.data_ptr(), 10, 0)]
    t.untyped_storage().resize_(0)                        # memory given back: sizes stay, no address
    assert h.current().ptrs[0] is None


def test_overlap_made_later_is_refused(B):
    m = torch.zeros(100)
    a, b = m[:50].as_subclass(_Posing), m[50:].as_subclass(_Posing)
    h = B.GradList([a, b])
    a.data = m[:60]
    with pytest.raises(ValueError):
        h.current()


def test_list_of_tensors_changed(B):
    """Its own list of tensors, given more, fewer or other things."""
    ts = _ts(5, 6)
    h = B.GradList(ts)
    h.tensors.append(_ts(9)[0])
    assert [n for _, n, _ in _seen(h)] == [5, 6, 9]
    del h.tensors[1:]
    assert [n for _, n, _ in _seen(h)] == [5]
    h.tensors[0] = 3.0
    with pytest.raises(TypeError):
        h.current()


def test_unchanged_tensors_are_not_looked_at_again(B, monkeypatch):
    h = B.GradList(_ts(*range(1, 40)))
    monkeypatch.setattr(B.GradList, "_look", lambda self: pytest.fail("looked at again"))
    assert h.current() is h
    assert B.GradList.current(h) is h


def test_oracle_of_infinite_bounds_and_norms():
    """The definition the GPU is compared with: no bound is a factor of 1, an
    infinite norm under a bound one of 0, a NaN norm one of NaN."""
    import numpy as np
    from oracle import route as R
    g = [np.array([2.0, 1.0])]
    inf = float("inf")
    for total, bound, want in [(inf, inf, 1.0), (5.0, inf, 1.0), (inf, 3.0, 0.0), (0.0, inf, 1.0)]:
        assert np.array_equal(R.clip(g, total, bound)[1][0], want * g[0])
    for bound in (inf, 3.0):
        assert np.isnan(R.clip(g, float("nan"), bound)[1][0]).all()
