"""The routing oracle pinned: selection by plain loops, gates and gradients by
differences of the forward, the balance loss by its closed form."""

import math

import numpy as np
import pytest

from oracle import formats as F
from oracle import route as R


def _logits(seed, T, E, closed=0.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E))
    if closed:
        x[rng.random((T, E)) < closed] = -np.inf
    return x


def _loop_select(x, k, bias, mask):
    out = np.full((x.shape[0], k), -1, np.int32)
    for t in range(x.shape[0]):
        if mask is not None and not mask[t]:
            continue
        left = [e for e in range(x.shape[1]) if x[t, e] > -math.inf]
        for j in range(k):
            best = None
            for e in left:
                v = x[t, e] if bias is None else 1 / (1 + math.exp(-x[t, e])) + bias[e]
                if best is None or v > best[0]:
                    best = (v, e)
            if best is None:
                break
            out[t, j] = best[1]
            left.remove(best[1])
    return out


@pytest.mark.parametrize("E,k,closed,biased,masked", [
    (1, 1, 0.0, False, False), (8, 2, 0.0, False, True), (9, 9, 0.4, False, False),
    (70, 5, 0.95, True, True), (130, 8, 0.0, True, False),
])
def test_selection_by_plain_loops(E, k, closed, biased, masked):
    rng = np.random.default_rng(E)
    x = np.round(_logits(E, 40, E, closed) * 4) / 4             # many ties
    bias = np.round(rng.normal(size=E) * 2) / 2 if biased else None
    mask = rng.random(40) < 0.5 if masked else None
    score = "sigmoid" if biased else "softmax"
    assert np.array_equal(R.select(x, k, score, bias, mask), _loop_select(x, k, bias, mask))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gates_sums_and_loss(score):
    T, E, k = 50, 12, 3
    x = _logits(1, T, E, 0.2)
    r = R.route(x, k, score, renorm=True, scale=2.5)
    assert np.allclose(r["gate"].sum(1), 2.5)
    for t in range(T):
        den = sum(math.exp(v) for v in x[t]) if score == "softmax" else 1.0
        for j, e in enumerate(R.route(x, k, score, renorm=False)["topk_ids"][t]):
            s = math.exp(x[t, e]) / den if score == "softmax" else 1 / (1 + math.exp(-x[t, e]))
            assert R.route(x, k, score, renorm=False)["gate"][t, j] == pytest.approx(s, rel=1e-12)
        break
    assert r["counts"][:E].sum() == T * k and r["counts"][E] == T
    assert r["prob_sum"].sum() == pytest.approx(T)
    # a uniform load costs alpha; all on one expert with all probability costs alpha * E
    assert R.balance_loss(np.array([5, 5, 5, 5, 10]), np.full(4, 2.5), 2, 0.1) == pytest.approx(0.1)
    assert R.balance_loss(np.array([7, 0, 0, 0, 7]), np.array([7.0, 0, 0, 0]), 1, 0.1) == pytest.approx(0.4)
    assert R.balance_loss(np.zeros(5), np.zeros(4), 1, 0.1) == 0.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("closed", [0.0, 0.5])
def test_gradient_by_differences(score, renorm, closed):
    """d/dx of sum(gate * dgate) + dloss * loss with the choice and the counts
    held: central differences in float64, step 1e-5 (truncation h^2/6 times a
    third derivative of order 1, rounding 1e-16 / h: both below 1e-9)."""
    T, E, k, alpha, dloss, scale = 6, 7, 3, 0.5, 1.7, 2.5
    x = _logits(3, T, E, closed)
    if closed:
        x[0] = -np.inf                                          # a row with nothing left
    ids = R.select(x, k, score)
    dg = np.random.default_rng(4).normal(size=(T, k))
    counts = R.route(x, k, score)["counts"]
    live = ids[:, :1] >= 0

    def f(y):
        g = R.gates(y, ids, score, renorm, scale)
        ps = (R.probabilities(y, score) * live).sum(0)
        return float((g * dg).sum() + dloss * R.balance_loss(counts, ps, k, alpha))

    d, mag = R.route_bwd(x, ids, dg, score, renorm, scale, counts, alpha, dloss)
    assert np.all(np.abs(d) <= mag + 1e-15)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if x[t, e] == -np.inf:
                assert d[t, e] == 0.0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert d[t, e] == pytest.approx((f(up) - f(dn)) / (2 * h), abs=2e-8)


def test_clip_closed_form():
    bits = F.f32_to_bf16_bits_rne(np.array([3.0, -4.0], np.float32))
    grads = [np.array([[12.0]], np.float32), bits]
    assert R.sumsq(grads) == 169.0
    norm, out = R.clip(grads, 169.0, 6.5)
    assert norm == 13.0
    assert np.allclose(np.concatenate([o.reshape(-1) for o in out]), [6.0, 1.5, -2.0], rtol=1e-6)
    assert R.clip(grads, 169.0, 20.0)[1][0] == 12.0
