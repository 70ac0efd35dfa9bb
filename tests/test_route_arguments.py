"""Arguments of the routing and clipping calls that are refused on the host,
before anything is allocated or launched. The tensors are host tensors that
pass for GPU ones; a call that got past its checks would fail otherwise."""

import pytest
import torch

from helpers import ensure_built

EINVAL, EUNSUP = 1, 2


@pytest.fixture(scope="module")
def B():
    ensure_built()
    from precision_moe_numerics_nvfp4_amd import binding
    return binding


class _Posing(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


def _posing(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Posing)


@pytest.mark.parametrize("T,E,k,status", [
    (8, 16, 17, EUNSUP), (8, 16, 0, EINVAL), (8, 16, -1, EINVAL), (8, 16, 10 ** 12, EUNSUP),
    (8, 16, 1 << 70, EUNSUP), (8, 200, 65, EUNSUP), (8, 1025, 2, EUNSUP), (8, 0, 1, EINVAL),
])
def test_sizes_are_refused_before_outputs_are_made(B, monkeypatch, T, E, k, status):
    x = _posing(T, E)
    monkeypatch.setattr(torch, "empty", lambda *a, **b: pytest.fail("allocated"))
    with pytest.raises(B.Nvfp4moeError) as e:
        B.moe_route(x, k)
    assert e.value.status == status


def test_more_slots_than_32_bits(B, monkeypatch):
    x = torch.zeros(1, 64).expand(1 << 26, 64).as_subclass(_Posing)
    monkeypatch.setattr(_Posing, "is_contiguous", lambda self, **k: True, raising=False)
    monkeypatch.setattr(torch, "empty", lambda *a, **b: pytest.fail("allocated"))
    with pytest.raises(B.Nvfp4moeError) as e:
        B.moe_route(x, 32)
    assert e.value.status == EUNSUP


def test_backward_and_loss_sizes(B, monkeypatch):
    ids = _posing(8, 17, dtype=torch.int32)
    counts, probs = _posing(17, dtype=torch.int64), _posing(16)
    monkeypatch.setattr(torch, "empty", lambda *a, **b: pytest.fail("allocated"))
    for call in (lambda: B.moe_route_bwd(_posing(8, 16), ids),
                 lambda: B.moe_route_bwd(_posing(8, 1025), ids),
                 lambda: B.moe_balance_loss(counts, probs, 17, 0.1),
                 lambda: B.moe_balance_loss(counts, probs, (1 << 32) + 2, 0.1)):
        with pytest.raises(B.Nvfp4moeError) as e:
            call()
        assert e.value.status == EUNSUP
    for call in (lambda: B.moe_route_bwd(_posing(8, 16), ids[:, :0]),
                 lambda: B.moe_balance_loss(counts, probs, 0, 0.1)):
        with pytest.raises(B.Nvfp4moeError) as e:
            call()
        assert e.value.status == EINVAL


def test_numbers_on_the_device_are_refused(B, monkeypatch):
    """Reading one would make the call wait for the GPU."""
    x, one = _posing(8, 16), _posing()
    for get in ("__float__", "__int__", "item"):
        monkeypatch.setattr(_Posing, get, lambda self: pytest.fail("waited for the device"), raising=False)
    ids, f = _posing(8, 2, dtype=torch.int32), dict(dtype=torch.float64)
    h = B.GradList([])
    for call in (lambda: B.moe_route(x, one), lambda: B.moe_route(x, 2, scale=one, out=_out()),
                 lambda: B.moe_balance_loss(_posing(17, dtype=torch.int64), _posing(16), one, 0.1),
                 lambda: B.moe_balance_loss(_posing(17, dtype=torch.int64), _posing(16), 2, one, loss=_posing(1)),
                 lambda: B.moe_route_bwd(x, ids, scale=one, dlogits=_posing(8, 16)),
                 lambda: B.moe_route_bwd(x, ids, alpha=one, dlogits=_posing(8, 16)),
                 lambda: B.moe_grad_clip(h, _posing(1, **f), one, norm=_posing(1))):
        with pytest.raises(ValueError, match="host number"):
            call()


def _out():
    return {"topk_ids": _posing(8, 2, dtype=torch.int32), "gate": _posing(8, 2)}


def test_host_numbers_of_any_type(B):
    import numpy as np
    from fractions import Fraction
    for v in (2.5, 2, True, np.float32(2.5), np.int64(2), Fraction(5, 2), torch.tensor(2.5)):
        assert B._number(v, "scale") == float(v)
    assert B._number(np.int32(3), "k", int) == 3 and B._number(torch.tensor(3), "k", int) == 3
    with pytest.raises((TypeError, ValueError)):
        B._number("two", "scale")
