"""The routed FFN step: router, balance loss, expert FFN, gradient to the logits
and clipped expert gradients in one run, each call checked on the GPU's own
inputs to it (bounds as derived in test_gpu_route and test_gpu_gradclip), and
the whole captured in a graph."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _case(seed, T, K, F, E, n, dtype):
    import torch
    w = gen.ffn_case(seed, T, K, F, E, 2, n_experts=n)
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(T, n)).astype(np.float32)
    if dtype == torch.bfloat16:
        logits = gen.to_bf16_bits(logits)
    mask = rng.random(T) < 0.8
    bias = (0.3 * rng.normal(size=n)).astype(np.float32)
    return (to_dev(w["x"]), to_dev(w["w1"].reshape(E * F, K)), to_dev(w["w2"].reshape(E * K, F)),
            to_dev(logits), to_dev(w["dout"])), to_dev(bias), to_dev(mask)


@pytest.mark.parametrize("score,renorm,n,e0,dtype", [
    ("softmax", True, 4, 0, "float32"), ("sigmoid", True, 12, 4, "bfloat16"),
    ("softmax", False, 70, 8, "float32"),
])
def test_routed_step(score, renorm, n, e0, dtype):
    ensure_built()
    import torch
    from precision_moe_numerics_nvfp4_amd.layer import ExpertFFNStep, RoutedFFNStep
    T, K, F, E, k, alpha, scale = 300, 256, 256, 4, 3, 0.2, 2.5
    dt = getattr(torch, dtype)
    args, bias, mask = _case(40, T, K, F, E, n, dt)
    x, w1, w2, logits, dout = args
    bias = bias if score == "sigmoid" else None
    S = RoutedFFNStep(T, K, F, E, k, n_experts=n, e0=e0, score=score, renorm=renorm, scale=scale,
                      alpha=alpha, logits_dtype=dt)
    S.ffn.dgate.fill_(5.0)                            # an earlier step's
    out, loss, dx, dlogits, norm = S.step(x, w1, w2, logits, dout, 1e30, bias, mask)
    torch.cuda.synchronize()
    h = lambda t: from_dev(t.clone())
    lg = from_dev(logits)
    D = float(np.abs(R._vals(lg)).max()) * 2
    rel = (6 * D + n + 16) * U
    r = R.route(lg, k, score, renorm, scale, None if bias is None else from_dev(bias), from_dev(mask))
    assert np.array_equal(h(S.topk_ids), r["topk_ids"]) and np.array_equal(h(S.counts), r["counts"])
    assert (np.abs(h(S.gate) - r["gate"]) <= rel * r["gate"] + 1e-37).all()
    ref = R.balance_loss(r["counts"], r["prob_sum"], k, alpha)
    assert abs(h(loss)[0] - ref) <= (rel + (T + 2) * U) * ref
    # the FFN is the existing one on these ids and gates, bit for bit
    G = ExpertFFNStep(T, K, F, E, k, e0=e0)
    G.quantize_weights(w1, w2)
    assert torch.equal(G.forward(x, S.topk_ids, S.gate), out)
    assert torch.equal(G.backward(dout, S.gate), dx)
    dg = h(S.ffn.dgate)
    local = (r["topk_ids"] >= e0) & (r["topk_ids"] < e0 + E)
    assert np.array_equal(dg[local], h(G.dgate)[local]) and (dg[~local] == 0).all()
    assert (h(out)[~from_dev(mask)] == 0).all() and (R._vals(h(dlogits))[~from_dev(mask)] == 0).all()
    ref, mag = R.route_bwd(lg, r["topk_ids"], dg, score, renorm, scale, r["counts"], alpha)
    bound = 2 * rel * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0.0) + 1e-37
    assert (np.abs(R._vals(h(dlogits)) - ref) <= bound).all()
    # 1e30: nothing clipped; then by half the norm, in place
    raw = [h(S.ffn.dw1), h(S.ffn.dw2)]
    assert np.array_equal(raw[0], h(G.dw1)) and np.array_equal(raw[1], h(G.dw2))
    total = R.sumsq(raw)
    assert h(norm)[0] == pytest.approx(np.sqrt(total), rel=2.0 ** -23)
    half = float(np.float32(0.5 * np.sqrt(total)))
    S.clip(half)
    for got, want in zip((S.ffn.dw1, S.ffn.dw2), R.clip(raw, total, half)[1]):
        assert (np.abs(h(got) - want) <= 2 * U * np.abs(want) + 1e-37).all()


def test_routed_step_graph():
    """Captured once, replayed with eager steps on other inputs in between."""
    ensure_built()
    import torch
    from precision_moe_numerics_nvfp4_amd.layer import RoutedFFNStep
    T, K, F, E, k = 300, 256, 256, 8, 2
    cases = [_case(41 + i, T, K, F, E, E, torch.float32) for i in range(2)]
    S = RoutedFFNStep(T, K, F, E, k, alpha=0.1)
    run = lambda c: S.step(*c[0], 1e-3, token_mask=c[2])
    outs = lambda: [S.topk_ids, S.gate, S.counts, S.balance, S.ffn.out, S.ffn.dx, S.dlogits,
                    S.norm, S.ffn.dw1, S.ffn.dw2]
    refs = []
    for c in cases:
        run(c)
        torch.cuda.synchronize()
        refs.append([t.clone() for t in outs()])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(cases[0])
    for _ in range(3):
        run(cases[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[1], outs()))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[0], outs()))
