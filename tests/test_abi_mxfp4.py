"""Refusals of the MXFP4 calls, the grouping without rows and the few-token
layer: on the host, before any HIP call (CPU only)."""

import ctypes

import pytest

from helpers import ensure_built

EINVAL, EUNSUP, EWS = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: calls fail first
ODD = ctypes.c_void_p(0x10001)
FOUR = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from precision_moe_numerics_nvfp4_amd import binding
    return binding.lib()


def test_quantize_refusals(L):
    def f(x=FAKE, dt=1, rows=4, cols=64, live=None, codes=FAKE, scales=FAKE):
        return L.mxfp4_quantize(x, dt, rows, cols, live, codes, scales, None)
    assert f(x=None) == f(codes=None) == f(scales=None) == EINVAL
    assert f(dt=2) == f(rows=-1) == f(cols=-32) == EINVAL
    assert f(cols=48) == f(cols=0) == EUNSUP
    assert f(rows=1 << 40) == f(rows=1 << 62, cols=1 << 40) == EUNSUP
    assert f(x=FOUR) == f(codes=FOUR) == f(scales=FOUR) == f(live=FOUR) == EUNSUP
    assert f(rows=0, x=None) == 0


@pytest.mark.parametrize("name", ["mxfp4_dequantize", "mxfp8_dequantize"])
def test_dequantize_refusals(L, name):
    def f(q=FAKE, e=FAKE, rows=4, cols=64, out=FAKE, dt=0):
        return getattr(L, name)(q, e, rows, cols, out, dt, None)
    assert f(q=None) == f(e=None) == f(out=None) == EINVAL
    assert f(dt=3) == f(rows=-1) == EINVAL
    assert f(cols=16) == f(rows=1 << 41) == f(q=FOUR) == f(out=FOUR) == f(e=ODD) == EUNSUP
    assert f(rows=0, q=None) == 0


def test_group_refusals(L):
    def f(ids=FAKE, T=64, k=2, n=8, off=FAKE, pad=FAKE, tok=FAKE, slot=FAKE, ws=FAKE, wsb=1 << 20):
        return L.moe_group(ids, T, k, 0, n, off, pad, tok, slot, None, ws, wsb, None)
    assert f(ids=None) == f(off=None) == f(pad=None) == f(tok=None) == f(slot=None) == f(ws=None) == EINVAL
    assert f(T=-1) == f(k=0) == f(n=0) == EINVAL
    assert f(k=65) == f(n=1025) == f(T=1 << 30) == f(T=1 << 62) == f(ws=FOUR) == EUNSUP
    assert f(wsb=L.nvfp4moe_permute_workspace_size(64, 2, 8) - 1) == EWS


def test_gemm_refusals(L):
    def f(ac=FAKE, as_=FAKE, rows=64, tok=None, bc=FAKE, bs=FAKE, off=FAKE, G=4, cap=64, N=128, K=256,
          y=FAKE, dt=0):
        return L.moe_fwd_grouped_gemm_mxfp4(ac, as_, rows, tok, bc, bs, off, G, cap, N, K, y, dt, None)
    assert f(ac=None) == f(as_=None) == f(bc=None) == f(bs=None) == f(off=None) == f(y=None) == EINVAL
    assert f(dt=7) == f(G=-1) == f(cap=-1) == f(N=-128) == f(K=-128) == f(rows=-1) == EINVAL
    assert f(rows=63) == EINVAL                                   # rows are read in place
    assert f(N=64) == f(K=64) == f(K=0) == f(K=1 << 23) == EUNSUP
    assert f(G=4001) == f(cap=1 << 31, rows=1 << 31) == f(N=1 << 40) == EUNSUP
    assert f(ac=FOUR) == f(bc=FOUR) == f(y=FOUR) == f(as_=ODD) == f(bs=ODD) == f(tok=ODD) == f(off=FOUR) == EUNSUP
    assert f(G=0) == f(cap=0) == f(N=0) == f(rows=0) == 0


def test_requant_refusals(L):
    def f(q=FAKE, e=FAKE, rows=64, cols=128, tok=None, rpg=0, off=FAKE, pad=FAKE, G=2, P=128, out=FAKE, oe=FAKE):
        return L.mxfp8_requant_sr_mxfp4(q, e, rows, cols, tok, rpg, off, pad, G, P, 1, 0, out, oe, None)
    assert f(q=None) == f(e=None) == f(off=None) == f(pad=None) == f(out=None) == f(oe=None) == EINVAL
    assert f(rows=-1) == f(cols=-1) == f(G=-1) == f(P=-32) == f(rpg=-1) == EINVAL
    assert f(tok=FAKE, rpg=32) == EINVAL                          # weights are not read through a map
    assert f(cols=64) == f(P=48) == f(q=FOUR) == f(out=FOUR) == f(e=ODD) == f(tok=ODD) == EUNSUP
    assert f(P=1 << 40) == EUNSUP
    assert f(G=0) == f(P=0) == f(cols=0) == 0


def test_ffn_tokens_refusals(L):
    def f(x=FAKE, lg=FAKE, dt=0, T=4, E=8, k=2, score=0, bias=None, mask=None, fmt=1, w1=FAKE, s1=FAKE,
          o1=None, w2=FAKE, s2=FAKE, o2=None, n=8, K=256, F=128, act=2, ids=FAKE, gate=FAKE, out=FAKE, odt=1,
          ws=FAKE, wsb=1 << 30):
        return L.moe_ffn_tokens(x, lg, dt, T, E, k, score, 1, 1.0, bias, mask, fmt, w1, s1, o1, w2, s2, o2, 0, n,
                                K, F, act, 0, ids, gate, out, odt, ws, wsb, None)
    for name in ("x", "lg", "w1", "s1", "w2", "s2", "ids", "gate", "out", "ws"):
        assert f(**{name: None}) == EINVAL, name
    assert f(dt=2) == f(odt=2) == f(score=2) == f(fmt=2) == f(act=3) == f(act=-1) == EINVAL
    assert f(T=-1) == f(E=0) == f(k=0) == f(n=0) == f(K=0) == f(F=0) == EINVAL
    assert f(fmt=0) == f(o1=FAKE) == f(fmt=0, o1=FAKE) == EINVAL  # outer scales go with NVFP4
    assert f(T=65) == f(k=9) == f(k=17, E=64) == f(T=64, k=9, E=64) == f(E=1025) == f(n=1025) == EUNSUP
    assert f(K=64) == f(F=192) == f(K=1 << 21) == f(F=1 << 21) == EUNSUP
    assert f(bias=FAKE) == EUNSUP                                 # softmax has no bias
    for name in ("x", "w1", "s1", "w2", "s2", "out", "ws"):
        assert f(**{name: FOUR}) == EUNSUP, name
    for name in ("lg", "ids", "gate"):
        assert f(**{name: ODD}) == EUNSUP, name
    need = L.nvfp4moe_ffn_tokens_workspace_size(4, 2, 128, 128)
    assert need > 0 and f(wsb=need - 1) == EWS
    assert f(T=0, x=None) == 0
    size = L.nvfp4moe_ffn_tokens_workspace_size
    assert size(65, 1, 128, 128) == size(64, 9, 128, 128) == size(-1, 2, 128, 128) == size(1 << 62, 2, 128, 128) == 0
    assert size(4, 2, 1 << 40, 128) == size(4, 2, 128, 1 << 40) == 0
