"""Expert selection of the few-token layer where scores are equal as numbers but
not as bits: zeros of both signs. Ids are the oracle's (the lower index first),
whether the workgroups select by themselves (up to 16 tokens) or the router does."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import mxfp4 as M4
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["softmax", "softmax-sum", "sigmoid", "sigmoid-bias"])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (5, 9, 3), (16, 64, 8), (16, 65, 16), (17, 64, 8), (13, 500, 4), (40, 12, 4)])
def test_zeros_of_both_signs_are_equal(nv, T, E, k, form, dtype):
    rng = np.random.default_rng(T * E + k)
    lg = np.where(rng.random((T, E)) < 0.5, np.float32(0.0), np.float32(-0.0))
    lg[0, :4] = -0.0, 0.0, -1.0, 0.0
    lg[T // 2:, ::3] = -1.5                                 # some lower, some closed
    lg[T - 1, 1::4] = -np.inf
    score, renorm = form.split("-")[0], form == "softmax-sum"
    bias = np.where(rng.random(E) < 0.5, np.float32(0.0), np.float32(-0.0)) if form == "sigmoid-bias" else None
    x = gen.to_bf16_bits(rng.normal(size=(T, 128)).astype(np.float32))
    w1, w2 = (tuple(to_dev(a) for a in M4.quantize((rng.normal(size=(128, 128)) * 0.1).astype(np.float32))) for _ in "12")
    lg = gen.to_bf16_bits(lg) if dtype == "bf16" else lg
    o = nv.moe_ffn_tokens(to_dev(x), to_dev(lg), k, w1, w2, score=score, renorm=renorm,
                          bias=None if bias is None else to_dev(bias))
    r = R.route(lg, k, score, renorm, 1.0, bias)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    # logits of 0 and -1.5 only: moe_route's bound at a distance of 1.5
    rel = (6 * 1.5 + E + 16) * 2.0 ** -24
    assert (np.abs(from_dev(o["gate"]) - r["gate"]) <= rel * r["gate"] + 1e-37).all()


@pytest.mark.parametrize("form", ["softmax", "softmax-sum", "sigmoid", "sigmoid-bias"])
@pytest.mark.parametrize("T,E,k", [(16, 64, 8), (17, 64, 8), (1, 65, 16), (8, 65, 4), (9, 65, 4), (3, 128, 1), (8, 384, 16),
                                   (9, 384, 8), (8, 385, 8), (1, 1024, 16), (12, 1024, 4), (2, 65, 16),
                                   (2, 300, 8), (2, 1024, 16)])
def test_selection_by_size(nv, T, E, k, form):
    """Ties, closed and NaN logits and masked rows on both sides of where the workgroups select by themselves."""
    rng = np.random.default_rng(T + E + k)
    lg = np.round(rng.normal(size=(T, E)) * 4).astype(np.float32) / 2
    lg[rng.random((T, E)) < 0.3] = -np.inf
    lg[T // 3] = -np.inf
    lg[T // 2, 1::2] = np.nan                               # a row with NaN among others: never selected
    score, renorm = form.split("-")[0], form != "softmax"
    bias = (np.round(rng.normal(size=E)) / 4).astype(np.float32) if form == "sigmoid-bias" else None
    mask = rng.random(T) < 0.8
    x = to_dev(gen.to_bf16_bits(rng.normal(size=(T, 128)).astype(np.float32)))
    w1, w2 = (tuple(to_dev(a) for a in M4.quantize((rng.normal(size=(128, 128)) * 0.1).astype(np.float32))) for _ in "12")
    how = dict(score=score, renorm=renorm, scale=2.5)
    dev = dict(bias=None if bias is None else to_dev(bias), token_mask=to_dev(mask))
    o = nv.moe_ffn_tokens(x, to_dev(lg), k, w1, w2, **how, **dev)
    r = nv.moe_route(to_dev(lg), k, **how, **dev)
    assert np.array_equal(from_dev(o["topk_ids"]), from_dev(r["topk_ids"]))
    there = np.arange(T) != T // 2                          # gates of a row that holds NaN are not defined
    ref = R.route(np.where(np.isnan(lg), -np.inf, lg).astype(np.float32), k, score, renorm, 2.5, bias, mask)
    assert np.array_equal(from_dev(o["topk_ids"]), ref["topk_ids"])
    D = float(np.abs(lg[np.isfinite(lg)]).max(initial=0.0)) * 2
    rel = (6 * D + E + 16) * 2.0 ** -24
    assert (np.abs(from_dev(o["gate"]) - ref["gate"]) <= rel * ref["gate"] + 1e-37)[there].all()
