"""Refusals of the routing and gradient-clipping calls: on the host, before
any HIP call (CPU only)."""

import ctypes

import pytest

from helpers import ensure_built

EINVAL, EUNSUP, EWS = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: calls fail first
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from precision_moe_numerics_nvfp4_amd import binding
    return binding.lib()


def _route(L, logits=FAKE, dt=0, T=64, E=8, k=2, score=0, bias=None, mask=None, ids=FAKE,
           gate=FAKE, counts=None, prob=None, ws=None, wsb=0):
    return L.moe_route(logits, dt, T, E, k, score, 1, 1.0, bias, mask, ids, gate, counts, prob,
                       ws, wsb, None)


def test_route_refusals(L):
    assert _route(L, logits=None) == EINVAL
    assert _route(L, ids=None) == EINVAL
    assert _route(L, gate=None) == EINVAL
    assert _route(L, dt=2) == EINVAL
    assert _route(L, T=-1) == EINVAL
    assert _route(L, E=0) == EINVAL
    assert _route(L, k=0) == EINVAL
    assert _route(L, score=2) == EINVAL
    assert _route(L, counts=FAKE) == EINVAL                      # without prob_sum
    assert _route(L, prob=FAKE) == EINVAL                        # without counts
    assert _route(L, k=9) == EUNSUP                              # k > E
    assert _route(L, E=1025) == EUNSUP
    assert _route(L, E=100, k=65) == EUNSUP
    assert _route(L, T=1 << 30, k=2) == EUNSUP                   # T * k
    assert _route(L, T=1 << 62, k=4) == EUNSUP                   # T * k past 64 bits
    assert _route(L, bias=FAKE) == EUNSUP                        # softmax has no bias
    assert _route(L, logits=ODD) == EUNSUP
    assert _route(L, ids=ODD) == EUNSUP
    assert _route(L, T=5000, counts=FAKE, prob=FAKE) == EINVAL   # no workspace
    need = L.nvfp4moe_route_workspace_size(5000, 8)
    assert need > 0
    assert _route(L, T=5000, counts=FAKE, prob=FAKE, ws=FAKE, wsb=need - 1) == EWS
    assert L.nvfp4moe_route_workspace_size(1, 384) == 0          # few rows need none
    assert _route(L, logits=None, T=0, ids=None, gate=None) == 0  # nothing to do
    assert L.nvfp4moe_route_workspace_size(-1, 8) == 0
    assert L.nvfp4moe_route_workspace_size(8, 0) == 0
    assert L.nvfp4moe_route_workspace_size(1 << 40, 1024) < 1 << 24


def test_balance_loss_refusals(L):
    f = L.moe_balance_loss
    assert f(None, FAKE, 8, 2, 0.1, FAKE, None) == EINVAL
    assert f(FAKE, None, 8, 2, 0.1, FAKE, None) == EINVAL
    assert f(FAKE, FAKE, 8, 2, 0.1, None, None) == EINVAL
    assert f(FAKE, FAKE, 0, 2, 0.1, FAKE, None) == EINVAL
    assert f(FAKE, FAKE, 8, 9, 0.1, FAKE, None) == EUNSUP
    assert f(ctypes.c_void_p(0x10004), FAKE, 8, 2, 0.1, FAKE, None) == EUNSUP


def test_route_bwd_refusals(L):
    def f(logits=FAKE, dt=0, T=64, E=8, k=2, score=0, ids=FAKE, dg=FAKE, counts=FAKE, dl=FAKE, out=FAKE):
        return L.moe_route_bwd(logits, dt, T, E, k, score, 1, 1.0, ids, dg, counts, 0.1, dl, out, None)
    assert f(logits=None) == EINVAL
    assert f(ids=None) == EINVAL
    assert f(out=None) == EINVAL
    assert f(dt=5) == EINVAL
    assert f(score=-1) == EINVAL
    assert f(T=-1) == EINVAL
    assert f(k=9) == EUNSUP
    assert f(E=1025) == EUNSUP
    assert f(T=1 << 31, k=1) == EUNSUP
    assert f(T=1 << 62, k=4) == EUNSUP
    assert f(dl=ctypes.c_void_p(0x10002)) == EUNSUP
    assert f(out=ODD) == EUNSUP
    assert f(logits=None, T=0, ids=None, out=None) == 0


def _list(ptrs, types, sizes):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int * n)(*types), (ctypes.c_int64 * n)(*sizes), n)


def test_gradient_list_refusals(L):
    size = lambda sizes, n=None: L.nvfp4moe_grad_workspace_size(
        (ctypes.c_int64 * len(sizes))(*sizes), len(sizes) if n is None else n)
    need = size([1 << 20])
    assert need > 0 and size([4]) == 0                            # a short list needs none
    assert size([4], -1) == 0 and size([-4]) == 0
    assert L.nvfp4moe_grad_workspace_size(None, 1) == 0
    assert size([1 << 40] * 2) < 1 << 16 and size([1 << 62] * 4) == 0

    def s(ptrs, types, sizes, out=FAKE, ws=FAKE, wsb=1 << 30, n=None):
        p, t, m, k = _list(ptrs, types, sizes)
        return L.moe_grad_sumsq(p, t, m, k if n is None else n, out, ws, wsb, None)
    assert s([0x10000], [0], [4], out=None) == EINVAL
    assert s([0x10000], [0], [1 << 20], ws=None) == EINVAL
    assert s([0x10000], [0], [4], n=-1) == EINVAL
    assert s([0x10000], [2], [4]) == EINVAL
    assert s([0x10000], [0], [-4]) == EINVAL
    assert s([None], [0], [4]) == EINVAL
    assert s([0x10002], [0], [4]) == EUNSUP
    assert s([0x10001], [1], [4]) == EUNSUP
    assert s([0x10000], [0], [(1 << 44) + 1]) == EUNSUP
    assert s([0x10000, 0x10000], [0, 0], [1 << 43, (1 << 43) + 1]) == EUNSUP
    assert s([0x10000], [0], [1 << 20], wsb=need - 1) == EWS
    assert L.moe_grad_sumsq(None, None, None, 1, FAKE, FAKE, 1 << 30, None) == EINVAL

    def c(ptrs, outs, sizes, sumsq=FAKE, max_norm=1.0, norm=FAKE):
        p, t, m, k = _list(ptrs, [0] * len(ptrs), sizes)
        o = (ctypes.c_void_p * k)(*outs)
        return L.moe_grad_clip(p, o, t, m, k, sumsq, max_norm, norm, None)
    assert c([0x10000], [0x10000], [4], sumsq=None) == EINVAL
    assert c([0x10000], [0x10000], [4], max_norm=-1.0) == EINVAL
    assert c([0x10000], [0x10000], [4], max_norm=float("nan")) == EINVAL
    assert c([0x10000], [None], [4]) == EINVAL
    assert c([0x10000], [0x10004], [4]) == EINVAL                # overlaps its gradient
    assert c([0x10000], [0x10002], [4]) == EUNSUP
    assert c([0x10000], [0x10000], [4], norm=ODD) == EUNSUP


def test_binding_refusals():
    import torch
    from precision_moe_numerics_nvfp4_amd import binding as B
    with pytest.raises(ValueError):
        B.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        B.GradList([torch.zeros(4)])
    with pytest.raises(TypeError):
        B.GradList([[1.0]])
    with pytest.raises(ValueError):
        B.moe_balance_loss(torch.zeros(9, dtype=torch.int64), torch.zeros(8), 2, 0.1)
    assert B._overlap([(0, 4), (8, 12)], [(4, 8), (12, 16)]) is False
    assert B._overlap([(0, 4), (8, 12)], [(4, 8), (11, 16)]) is True
    assert B._overlap([(0, 100)], [(10, 20)]) is True
    assert B._overlap([], [(10, 20)]) is False
