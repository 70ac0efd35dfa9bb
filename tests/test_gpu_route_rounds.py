"""Every form of the routing kernels past its first round of rows, against the
float64 oracle: rows and mask bytes loaded one round ahead are used there, with
padding that holds NaN and closed experts. Bounds as derived in test_gpu_route,
the probability sums' as in test_gpu_route_sums.

A forward launch takes 32 wavefronts a compute unit of 256, so 8192 rows a round
with a wavefront each, 32768 with 16 lanes each; a thread each 131072 with
statistics and 524288 without. The backward's rounds are 8192, 32768 and 524288.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUMS = 22 * U


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


def _inputs(T, E, dtype):
    rng = np.random.default_rng(T + E)
    x = rng.normal(size=(T, E)).astype(np.float32)
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[T // 2] = -np.inf
    mask = rng.random(T) < 0.8
    if dtype == "bf16":
        x = gen.to_bf16_bits(x)
    padded = x.copy()
    padded[~mask] = 0x7FC0 if dtype == "bf16" else np.nan
    return rng, x, padded, mask


def _rel(x, E, score):
    v = R._vals(x)
    f = np.isfinite(v)
    if score == "sigmoid":
        D = np.abs(np.where(f, v, 0)).max()
    else:
        top = v.max(axis=1, keepdims=True)
        D = np.where(f, np.where(f, top, 0) - np.where(f, v, 0), 0).max()
    return (6 * D + E + 16) * U


def _close(got, ref, bound, what):
    d = np.abs(np.asarray(got, np.float64) - ref)
    bad = ~(d <= bound + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} out of bound, worst {d.max():.3e} of {np.abs(ref).max():.3e}"


FORWARD = [
    # 16 lanes a row, of 4, 8 and 16 wavefronts a workgroup, then later rounds
    (3001, 60, 5, False, "f32"), (6001, 30, 4, False, "bf16"), (12001, 60, 16, False, "f32"),
    (45000, 60, 5, False, "f32"), (40001, 40, 6, False, "bf16"), (33001, 100, 3, False, "f32"),
    (70000, 128, 4, False, "bf16"), (40000, 40, 6, True, "f32"), (66000, 17, 5, True, "bf16"),
    (70001, 12, 3, True, "f32"), (33000, 64, 16, True, "f32"),
    # a wavefront a row: 1, 2, 4, 6, 8 and 16 experts a lane
    (20000, 50, 17, False, "f32"), (20001, 100, 8, False, "bf16"), (17000, 200, 8, False, "f32"),
    (17001, 384, 8, False, "bf16"), (9000, 500, 20, False, "f32"), (9001, 900, 8, False, "f32"),
    (20000, 60, 20, True, "f32"), (17000, 120, 8, True, "f32"), (20000, 200, 8, True, "bf16"),
    (17000, 384, 8, True, "f32"), (9000, 450, 8, True, "f32"), (9000, 1000, 33, True, "bf16"),
    # a thread a row
    (140001, 6, 2, False, "f32"), (140000, 16, 4, False, "bf16"), (140003, 30, 4, False, "f32"),
    (135000, 64, 6, False, "bf16"), (140000, 8, 2, True, "bf16"), (530000, 5, 3, False, "f32"),
    (530001, 7, 2, True, "f32"),
]


@pytest.mark.parametrize("T,E,k,biased,dtype", FORWARD)
def test_forward_rounds(nv, T, E, k, biased, dtype):
    rng, x, padded, mask = _inputs(T, E, dtype)
    score = "sigmoid" if biased or E % 3 == 0 else "softmax"
    bias = (0.2 * rng.normal(size=E)).astype(np.float32) if biased else None
    call = dict(score=score, scale=2.5, bias=to_dev(bias) if biased else None, token_mask=to_dev(mask))
    r = R.route(x, k, score, True, 2.5, bias, mask)
    rel = _rel(x, E, score)
    for stats in (True, False):
        o = nv.moe_route(to_dev(padded), k, stats=stats, **call)
        assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
        _close(from_dev(o["gate"]), r["gate"], rel * r["gate"], "gate")
        if stats:
            assert np.array_equal(from_dev(o["counts"]), r["counts"])
            _close(from_dev(o["prob_sum"]), r["prob_sum"], (rel + SUMS) * r["prob_sum"], "prob_sum")


BACKWARD = [
    (33000, 100, 4, "f32"), (70000, 128, 8, "bf16"), (70001, 12, 3, "f32"), (40000, 30, 5, "bf16"),
    (70000, 60, 6, "f32"), (20000, 50, 17, "f32"), (20001, 100, 20, "bf16"), (20000, 200, 8, "f32"),
    (17001, 384, 8, "bf16"), (9000, 500, 8, "f32"), (9001, 1000, 16, "bf16"), (530000, 8, 2, "bf16"),
    (530001, 5, 3, "f32"),
]


@pytest.mark.parametrize("T,E,k,dtype", BACKWARD)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_backward_rounds(nv, T, E, k, dtype, score, renorm):
    """Into new memory, and in place over the logits, whose later rounds are
    read ahead of the stores."""
    rng, x, padded, mask = _inputs(T, E, dtype)
    ids = R.select(R._vals(x), k, score, None, mask)
    dg = rng.normal(size=(T, k)).astype(np.float32)
    dg[ids < 0] = np.nan
    counts = R.route(x, k, score, token_mask=mask)["counts"]
    ref, mag = R.route_bwd(x, ids, dg, score, renorm, 2.5, counts, T * 0.5, 0.75)
    bound = 2 * _rel(x, E, score) * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
    call = dict(score=score, renorm=renorm, scale=2.5, counts=to_dev(counts), alpha=T * 0.5,
                dloss=to_dev(np.array([0.75], np.float32)))
    over = to_dev(padded)
    for logits, out in ((to_dev(padded), None), (over, over)):
        got = nv.moe_route_bwd(logits, to_dev(ids), to_dev(dg), dlogits=out, **call)
        _close(R._vals(from_dev(got)), ref, bound, "dlogits")


def test_probability_sums_past_32_bit_offsets(nv):
    """More than 2^32 logits: the equal rows' share in closed form, the others'
    from the oracle."""
    import torch
    T, E, k, tail = 4_300_000, 1000, 2, 70
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    ends = gen.to_bf16_bits(np.random.default_rng(12).normal(size=(2 * tail, E)).astype(np.float32))
    x[:tail], x[-tail:] = to_dev(ends[:tail]), to_dev(ends[tail:])
    o = nv.moe_route(x, k, stats=True)
    want = R.probabilities(R._vals(ends), "softmax").sum(axis=0) + (T - 2 * tail) / E
    # equal rows: a reciprocal's 2 u; the others, 3e-5 of them, _rel
    rel = 2 * U + _rel(ends, E, "softmax") * 2 * tail * E / T
    _close(from_dev(o["prob_sum"]), want, (rel + SUMS) * want, "prob_sum")
