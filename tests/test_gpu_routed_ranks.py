"""Statistics, routing-weight gradients and sums of squares added over ranks
between the calls, as the routed step allows: two ranks' steps on one GPU, the
additions in place of the collectives. Bounds as derived in test_gpu_route,
test_gpu_route_sums and test_gpu_gradclip; each addition of two float32 numbers
is one rounding more, u = 2^-24."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _data(seed, T, K, F, E, k, n):
    w = gen.ffn_case(seed, T, K, F, E, k, n_experts=n)
    logits = np.random.default_rng(seed).normal(size=(T, n)).astype(np.float32)
    return (to_dev(w["x"]), to_dev(w["w1"].reshape(E * F, K)), to_dev(w["w2"].reshape(E * K, F)),
            logits, to_dev(w["dout"]))


def _rel(x, n, score):
    D = np.abs(x).max() if score == "sigmoid" else (x.max(axis=1) - x.min(axis=1)).max()
    return (6 * D + n + 16) * U


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_data_parallel_statistics(score, renorm):
    """Each rank its own tokens: the loss and its gradient are the whole batch's."""
    ensure_built()
    from precision_moe_numerics_nvfp4_amd.layer import RoutedFFNStep
    K, F, E, k, n, alpha = 256, 256, 4, 3, 12, 40.0
    sizes = (300, 171)
    steps, data = [], []
    for i, T in enumerate(sizes):
        steps.append(RoutedFFNStep(T, K, F, E, k, n_experts=n, score=score, renorm=renorm, alpha=alpha))
        data.append(_data(50 + i, T, K, F, E, k, n))
        steps[i].ffn.quantize_weights(*data[i][1:3])
        steps[i].route(to_dev(data[i][3]))
    counts = steps[0].counts + steps[1].counts
    probs = steps[0].prob_sum + steps[1].prob_sum
    whole = np.concatenate([d[3] for d in data])
    r = R.route(whole, k, score, renorm)
    rel = _rel(whole, n, score)
    for s, (x, _, _, logits, dout) in zip(steps, data):
        s.counts.copy_(counts)
        s.prob_sum.copy_(probs)
        assert np.array_equal(from_dev(s.counts), r["counts"])
        ref = R.balance_loss(r["counts"], r["prob_sum"], k, alpha)
        assert abs(from_dev(s.loss())[0] - ref) <= (rel + 22 * U + 3 * U) * ref
        s.forward_ffn(x)
        s.backward_ffn(dout)
        got = from_dev(s.backward_route(to_dev(logits)))
        ids = from_dev(s.topk_ids)
        ref, mag = R.route_bwd(logits, ids, from_dev(s.ffn.dgate), score, renorm, 1.0, r["counts"], alpha)
        assert (np.abs(got - ref) <= 2 * rel * mag + 1e-37).all()
    # the batch's gradient rows are the two ranks', each normalised by all tokens
    alone, _ = R.route_bwd(whole, r["topk_ids"], None, score, renorm, 1.0, r["counts"], alpha)
    for s, d, lo in zip(steps, data, (0, sizes[0])):
        s.ffn.dgate.zero_()
        got = from_dev(s.backward_route(to_dev(d[3])))
        part = alone[lo:lo + len(got)]
        _, mag = R.route_bwd(d[3], from_dev(s.topk_ids), None, score, renorm, 1.0, r["counts"], alpha)
        assert (np.abs(got - part) <= 2 * rel * mag + 1e-37).all()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_expert_parallel_dgate_and_norm(score, renorm):
    """Each rank its own experts of the same tokens: dgate completed by the other
    rank's part before the gradient to the logits, sums of squares joined
    before the clip."""
    ensure_built()
    import torch
    from precision_moe_numerics_nvfp4_amd.layer import RoutedFFNStep
    T, K, F, n, k, alpha = 200, 256, 256, 8, 3, 0.5
    x, w1, w2, logits, dout = _data(60, T, K, F, n, k, n)
    steps = []
    for e0, E in ((0, 5), (5, 3)):
        s = RoutedFFNStep(T, K, F, E, k, n_experts=n, e0=e0, score=score, renorm=renorm, alpha=alpha)
        s.ffn.quantize_weights(w1[e0 * F:(e0 + E) * F], w2[e0 * K:(e0 + E) * K])
        s.route(to_dev(logits))
        s.loss()
        s.forward_ffn(x)
        s.backward_ffn(dout)
        s.grad_sumsq()
        steps.append(s)
    a, b = steps
    assert torch.equal(a.topk_ids, b.topk_ids) and torch.equal(a.counts, b.counts)
    ids, da, db = from_dev(a.topk_ids), from_dev(a.ffn.dgate), from_dev(b.ffn.dgate)
    assert (da[ids >= 5] == 0).all() and (db[ids < 5] == 0).all()       # each its own experts alone
    whole = a.ffn.dgate + b.ffn.dgate
    ref, mag = R.route_bwd(logits, ids, from_dev(whole), score, renorm, 1.0, from_dev(a.counts), alpha)
    total = a.sumsq + b.sumsq
    raw = [[from_dev(g.clone()) for g in (s.ffn.dw1, s.ffn.dw2)] for s in steps]
    want = R.sumsq(raw[0] + raw[1])
    elements = sum(g.size for r in raw for g in r)
    assert from_dev(total)[0] == pytest.approx(want, rel=2.0 ** -52 * (elements + 8))
    bound = float(np.float32(0.4 * np.sqrt(want)))
    for s, r in zip(steps, raw):
        s.ffn.dgate.copy_(whole)
        got = from_dev(s.backward_route(to_dev(logits)))
        assert (np.abs(got - ref) <= 2 * _rel(logits, n, score) * mag + 1e-37).all()
        s.sumsq.copy_(total)
        assert from_dev(s.clip(bound))[0] == pytest.approx(np.sqrt(want), rel=2.0 ** -23)
        for g, c in zip((s.ffn.dw1, s.ffn.dw2), R.clip(r, want, bound)[1]):
            assert (np.abs(from_dev(g) - c) <= 3 * U * np.abs(c) + 1e-37).all()
