"""Rows whose shares are whole: one slot renormalised, or one open expert. A
number divided by itself is 1, so the gate is the scale itself and the
gradients of such a row are 0, not the rounding of gradients that cancel (which
would be all that dlogits holds where the balance loss's part is small)."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (50, 3), (200, 7), (4096, 8), (40, 60), (6000, 20), (70, 130), (300, 384), (60, 1000),
          (33000, 8), (66000, 60), (33000, 100)]


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


@pytest.mark.parametrize("T,E", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_slot_renormalised(nv, T, E, score, dtype):
    rng = np.random.default_rng(T + E)
    x = (3 * rng.normal(size=(T, E))).astype(np.float32)
    xd = to_dev(gen.to_bf16_bits(x) if dtype == "bf16" else x)
    dg = to_dev((100 * rng.normal(size=(T, 1))).astype(np.float32))
    o = nv.moe_route(xd, 1, score=score, scale=2.5)
    assert (from_dev(o["gate"]) == 2.5).all()
    d = nv.moe_route_bwd(xd, o["topk_ids"], dg, score=score, scale=2.5)
    assert (R._vals(from_dev(d)) == 0).all()


@pytest.mark.parametrize("T,E", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_one_open_expert(nv, T, E, score, renorm):
    """Its normalised score is 1: no gradient of the loss, nor of a softmax or
    renormalised gate; a plain sigmoid gate has its own."""
    rng = np.random.default_rng(T + E)
    x = np.full((T, E), -np.inf, np.float32)
    x[np.arange(T), rng.integers(0, E, size=T)] = 3 * rng.normal(size=T)
    k = min(E, 2)
    xd = to_dev(x)
    dg = (100 * rng.normal(size=(T, k))).astype(np.float32)
    o = nv.moe_route(xd, k, score=score, renorm=renorm, stats=True)
    r = R.route(x, k, score, renorm)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    whole = score == "softmax" or renorm
    if whole:
        assert np.array_equal(from_dev(o["gate"]), (r["topk_ids"] >= 0).astype(np.float32))
    assert np.allclose(from_dev(o["prob_sum"]), r["counts"][:E], rtol=2.0 ** -20)
    d = from_dev(nv.moe_route_bwd(xd, o["topk_ids"], to_dev(dg) if whole else None, score=score,
                                  renorm=renorm, counts=o["counts"], alpha=float(T)))
    assert (d == 0).all()


@pytest.mark.parametrize("T,E", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_loads_and_gate_gradients(nv, T, E, score):
    """Equal counts and equal gradients of every slot: what is subtracted is
    their mean, a quotient of two sums of up to E shares: off by 2 (E + 8) 2^-24
    of the value, then times a share."""
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, E)).astype(np.float32)
    k = min(E, 4)
    ids = R.select(R._vals(x), k)
    counts = np.full(E + 1, 10, np.int64)
    counts[E] = T
    d = from_dev(nv.moe_route_bwd(to_dev(x), to_dev(ids), to_dev(np.full((T, k), 64.0, np.float32)),
                                  score=score, counts=to_dev(counts), alpha=float(T) * T))
    a = T * T * E * 10 / (k * T * T)
    assert np.abs(d).max() <= 2 * (E + 8) * 2.0 ** -24 * (64.0 + a)
