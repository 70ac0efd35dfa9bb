"""GPU parity of the few-token expert layer against the float64 oracle.

Bit-exact: expert ids. Gates: within (6 D + E + 16) 2^-24 of the value, D the
logits' largest distance (as for moe_route). The output: the oracle carries a
bound through the layer, term by term: a sum of n terms loses n 2^-23 of its
terms' magnitudes (any order, the matrix unit may cut where it adds), the
activation's slope carries that on, h is held in two bfloat16 parts (2^-16 of
its value), gates to the bound above; and half a bfloat16 step, 2^-8 of the
value, where the output is stored so.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import mxfp4 as M4
from oracle import nvfp4 as Q
from oracle import route as R
from workloads import gen

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


def _case(seed, T, k, E, n, K, F, fmt, gated=False, logits="f32", bias=False, masked=False, closed=0.0):
    rng = np.random.default_rng(seed)
    m = 2 if gated else 1
    quantize = (lambda w, r: M4.quantize(w)) if fmt == "mxfp4" else Q.quantize
    lg = rng.normal(size=(T, E)).astype(np.float32)
    if closed:
        lg[rng.random((T, E)) < closed] = -np.inf
        lg[0] = -np.inf
    c = dict(x=gen.to_bf16_bits(rng.normal(size=(T, K)).astype(np.float32)),
             logits=gen.to_bf16_bits(lg) if logits == "bf16" else lg,
             w1=quantize((rng.normal(size=(n * m * F, K)) * 0.05).astype(np.float32), m * F),
             w2=quantize((rng.normal(size=(n * K, F)) * 0.05).astype(np.float32), K),
             bias=(0.3 * rng.normal(size=E)).astype(np.float32) if bias else None,
             token_mask=rng.random(T) < 0.7 if masked else None)
    return c


def _dev(c):
    up = lambda v: None if v is None else tuple(to_dev(a) for a in v) if isinstance(v, tuple) else to_dev(v)
    return {n: up(v) for n, v in c.items()}


def _spread(x):
    x = R._vals(x)
    f = np.isfinite(x)
    return float(np.abs(np.where(f, x, 0)).max()) * 2 if f.any() else 0.0


def _check(nv, c, k, n, out_dtype="bfloat16", **how):
    import torch
    d = _dev(c)
    o = nv.moe_ffn_tokens(d["x"], d["logits"], k, d["w1"], d["w2"], bias=d["bias"], token_mask=d["token_mask"],
                          out_dtype=getattr(torch, out_dtype), **how)
    rel = (6 * _spread(c["logits"]) + c["logits"].shape[1] + 16) * U
    r = M4.ffn_tokens(c["x"], c["logits"], k, c["w1"], c["w2"], bias=c["bias"], token_mask=c["token_mask"],
                      n_local=n, gate_rel=rel, **how)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    assert (np.abs(from_dev(o["gate"]) - r["gate"]) <= rel * r["gate"] + 1e-37).all()
    got = o["out"].double().cpu().numpy()
    bound = r["bound"] + (2.0 ** -8 * np.abs(r["out"]) if out_dtype == "bfloat16" else 0.0) + 1e-37
    e = np.abs(got - r["out"])
    assert (e <= bound).all(), f"worst {np.max(e / bound):.3f} of the bound, {np.max(e):.3e}"
    return o


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,k,E,n,e0,K,F", [
    (1, 1, 1, 1, 0, 128, 128), (1, 2, 8, 8, 0, 256, 384), (3, 2, 8, 3, 2, 640, 128), (16, 2, 4, 4, 0, 128, 256),
    (17, 3, 12, 6, 3, 256, 128), (33, 8, 130, 30, 60, 128, 256), (64, 8, 64, 16, 16, 384, 128),
    (64, 1, 2, 2, 0, 256, 256), (5, 16, 500, 40, 100, 128, 128), (2, 4, 1024, 1024, 0, 128, 128),
    (1, 8, 16, 16, 0, 2176, 640), (64, 2, 2, 2, 0, 1024, 1024), (47, 2, 5, 5, 0, 1152, 640), (30, 3, 40, 3, 20, 512, 640),
])
def test_sizes(nv, fmt, T, k, E, n, e0, K, F):
    c = _case(T + K, T, k, E, n, K, F, fmt)
    _check(nv, c, k, n, e0=e0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("act", ["none", "relu2", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_dtype", ["bfloat16", "float32"])
def test_activations(nv, fmt, act, gated, out_dtype):
    c = _case(3, 9, 2, 6, 4, 256, 128, fmt, gated=gated)
    _check(nv, c, 2, 4, out_dtype, act=act, gated=gated, e0=1)


@pytest.mark.parametrize("score,renorm,bias,logits,masked,closed", [
    ("softmax", False, False, "bf16", True, 0.0), ("softmax", True, False, "f32", False, 0.8),
    ("sigmoid", True, True, "f32", True, 0.0), ("sigmoid", False, True, "bf16", False, 0.6),
    ("sigmoid", False, False, "f32", True, 0.9),
])
@pytest.mark.parametrize("E,n,e0", [(10, 10, 0), (200, 20, 90), (700, 50, 300)])
def test_routing_options(nv, score, renorm, bias, logits, masked, closed, E, n, e0):
    c = _case(E, 21, 4, E, n, 128, 128, "mxfp4", logits=logits, bias=bias, masked=masked, closed=closed)
    o = _check(nv, c, 4, n, act="relu2", score=score, renorm=renorm, scale=2.5, e0=e0)
    r = nv.moe_route(to_dev(c["logits"]), 4, score=score, renorm=renorm, scale=2.5,
                     bias=None if c["bias"] is None else to_dev(c["bias"]),
                     token_mask=None if c["token_mask"] is None else to_dev(c["token_mask"]))
    assert np.array_equal(from_dev(o["topk_ids"]), from_dev(r["topk_ids"]))


def test_ties_take_the_lower_index(nv):
    c = _case(4, 12, 4, 70, 70, 128, 128, "mxfp4")
    c["logits"][:] = np.round(c["logits"])
    c["logits"][3] = 0.0
    c["logits"][4, ::2] = -0.0
    _check(nv, c, 4, 70)


def test_nan_and_closed_logits(nv):
    import torch
    c = _case(5, 4, 3, 40, 40, 128, 128, "mxfp4")
    c["logits"][1, 7] = np.nan
    c["logits"][2] = -np.inf
    c["logits"][3, 2:] = -np.inf
    d = _dev(c)
    o = nv.moe_ffn_tokens(d["x"], d["logits"], 3, d["w1"], d["w2"])
    ids = from_dev(o["topk_ids"])
    assert 7 not in ids[1] and (ids[1] >= 0).all() and (ids[2] == -1).all() and (ids[3, 2] == -1)
    assert (o["out"][2] == 0).all() and torch.isfinite(o["out"][[0, 3]].float()).all()
    clean = dict(c, logits=np.where(np.isnan(c["logits"]), -np.inf, c["logits"]).astype(np.float32))
    _check(nv, clean, 3, 40)


def test_nothing_local(nv):
    c = _case(6, 7, 2, 8, 4, 256, 128, "nvfp4")
    d = _dev(c)
    out = dict(out=to_dev(np.full((7, 256), 3, np.float32)))
    o = nv.moe_ffn_tokens(d["x"], d["logits"], 2, d["w1"], d["w2"], e0=8, out=out)
    assert (o["out"] == 0).all() and o["out"] is out["out"]
    assert nv.moe_ffn_tokens(d["x"][:0], d["logits"][:0], 2, d["w1"], d["w2"])["out"].shape == (0, 256)


def test_values_of_any_size(nv):
    """Outer scales, inputs and block scales far from one; silu at its ends."""
    c = _case(7, 6, 2, 5, 5, 256, 128, "nvfp4", gated=True)
    c["w1"] = (c["w1"][0], c["w1"][1], (c["w1"][2] * np.exp2([-40, 30, 0, 5, -3])).astype(np.float32))
    c["w2"] = (c["w2"][0], c["w2"][1], (c["w2"][2] * np.exp2([20, -50, 0, 1, 2])).astype(np.float32))
    _check(nv, c, 2, 5, act="silu", gated=True)
    c = _case(8, 6, 2, 5, 5, 256, 128, "mxfp4")
    rng = np.random.default_rng(1)
    c["w1"] = (c["w1"][0], rng.integers(100, 140, c["w1"][1].shape).astype(np.uint8))
    c["w2"] = (c["w2"][0], rng.integers(90, 130, c["w2"][1].shape).astype(np.uint8))
    _check(nv, c, 2, 5, act="none")


@pytest.mark.parametrize("lo,hi,mul", [(0, 4, 100), (250, 253, -100), (60, 190, 0)])
def test_scale_bytes_at_the_ends(nv, lo, hi, mul):
    """The smallest and the largest MXFP4 scales (252 is the last that holds all codes), inputs that make up for them."""
    c = _case(6, 3, 2, 4, 4, 256, 128, "mxfp4")
    rng = np.random.default_rng(2)
    c["x"] = gen.to_bf16_bits((rng.normal(size=(3, 256)) * 2.0 ** mul).astype(np.float32))
    c["w1"] = (rng.integers(0, 256, c["w1"][0].shape).astype(np.uint8),
               rng.integers(lo, hi, c["w1"][1].shape).astype(np.uint8))
    _check(nv, c, 2, 4, "float32", act="none")


def test_gates_of_rows_that_are_not_finite(nv):
    """Ids are moe_route's in rows with NaN or +inf too; where its gates are NaN, these are, up to 16 tokens and beyond."""
    import torch
    for T in (5, 20):
        lg = torch.randn(T, 24, device="cuda")
        lg[0, 3], lg[1, 2], lg[1, 7], lg[2, 5] = float("inf"), float("inf"), float("inf"), float("nan")
        c = _dev(_case(13, T, 4, 24, 24, 128, 128, "mxfp4"))
        for how in (dict(), dict(renorm=False), dict(score="sigmoid"), dict(score="sigmoid", renorm=False)):
            o = nv.moe_ffn_tokens(c["x"], lg, 4, c["w1"], c["w2"], **how)
            r = nv.moe_route(lg, 4, **how)
            assert torch.equal(o["topk_ids"], r["topk_ids"])
            assert torch.equal(o["gate"].isnan(), r["gate"].isnan()), how


def test_in_place(nv):
    """The result may take the place of x."""
    import torch
    c = _dev(_case(14, 20, 3, 16, 16, 256, 256, "mxfp4"))
    ref = nv.moe_ffn_tokens(c["x"], c["logits"], 3, c["w1"], c["w2"])["out"]
    x = c["x"].clone()
    out = nv.moe_ffn_tokens(x, c["logits"], 3, c["w1"], c["w2"], out=dict(out=x))["out"]
    assert out is x and torch.equal(x, ref)


def test_same_bits_and_two_streams(nv):
    """The same call gives the same bits, on two streams at once with a workspace each."""
    import torch
    c = _dev(_case(9, 40, 4, 16, 16, 512, 256, "mxfp4"))
    run = lambda **kw: nv.moe_ffn_tokens(c["x"], c["logits"], 4, c["w1"], c["w2"], **kw)["out"].clone()
    ref = run()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(nv.ffn_tokens_workspace_size(40, 4, 512, 256), dtype=torch.uint8, device="cuda") for _ in s]
    outs = []
    for i in range(6):
        with torch.cuda.stream(s[i % 2]):
            outs.append(run(workspace=ws[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs)


def test_graph(nv):
    """Captured once, replayed on new values in its inputs, eager calls in between."""
    import torch
    a, b = (_dev(_case(s, 20, 3, 24, 8, 256, 256, "nvfp4", masked=True)) for s in (10, 11))
    live = {n: (tuple(t.clone() for t in v) if isinstance(v, tuple) else None if v is None else v.clone())
            for n, v in a.items()}
    out = dict(out=torch.empty(20, 256, dtype=torch.bfloat16, device="cuda"),
               topk_ids=torch.empty(20, 3, dtype=torch.int32, device="cuda"),
               gate=torch.empty(20, 3, device="cuda"))
    ws = torch.empty(nv.ffn_tokens_workspace_size(20, 3, 256, 256), dtype=torch.uint8, device="cuda")
    run = lambda c, **kw: nv.moe_ffn_tokens(c["x"], c["logits"], 3, c["w1"], c["w2"], e0=8,
                                            token_mask=c["token_mask"], **kw)
    refs = [[t.clone() for t in run(c).values()] for c in (a, b)]
    run(live, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(live, out=out, workspace=ws)
    for i in (0, 1, 1, 0):
        for n, v in (a, b)[i].items():
            for dst, src in zip(live[n] if isinstance(v, tuple) else [live[n]], v if isinstance(v, tuple) else [v]):
                if src is not None:
                    dst.copy_(src)
        run((b, a)[i])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip((out["out"], out["topk_ids"], out["gate"]),
                             (refs[i][0], refs[i][1], refs[i][2])):
            assert torch.equal(got, want)


def test_against_the_capacity_sized_path(nv):
    """The same weights through moe_route, moe_group, the MXFP4 product and moe_combine, whose activations are
    quantized: the inputs are MXFP4 values already, so only h is rounded there."""
    import torch
    T, k, E, K, F = 24, 2, 8, 256, 128
    c = _case(12, T, k, E, E, K, F, "mxfp4")
    xq = M4.quantize(c["x"])
    c["x"] = gen.to_bf16_bits(M4.dequantize(*xq).astype(np.float32))
    d = _dev(c)
    o = _check(nv, c, k, E, act="none")
    r = nv.moe_route(d["logits"], k)
    p = nv.moe_group(r["topk_ids"], 0, E)
    q = tuple(to_dev(a) for a in xq)
    h = nv.moe_fwd_grouped_gemm_mxfp4(*q, *d["w1"], p["offsets"], row_token=p["row_token"], out_dtype=torch.bfloat16)
    hq = nv.mxfp4_quantize(h, offsets=p["offsets"])
    y = nv.moe_fwd_grouped_gemm_mxfp4(*hq, *d["w2"], p["offsets"], out_dtype=torch.bfloat16)
    out = nv.moe_combine(y, p["pair_row"], r["gate"])
    a, b = o["out"].double(), out.double()
    # a block of 32 normal values has its largest at 2.1 s, between 3 and 6 steps' units: s is 1.43 to 2.86 of them.
    # Errors are uniform in the grid's steps (1/2 below 2, 1 below 4, 2 above), rms 0.18 to 0.30: 0.105 to 0.125 of s.
    assert float((a - b).norm() / a.norm()) < 0.15


def test_refusals(nv):
    import torch
    c = _dev(_case(13, 4, 2, 8, 4, 256, 128, "mxfp4"))
    f = lambda x=c["x"], lg=c["logits"], k=2, w1=c["w1"], w2=c["w2"], **kw: nv.moe_ffn_tokens(x, lg, k, w1, w2, **kw)
    for bad in (dict(x=c["x"].float()), dict(x=c["x"].t()), dict(lg=c["logits"][:3]), dict(lg=c["logits"].half()),
                dict(w1=c["w1"][:1]), dict(w1=c["w2"]), dict(w1=c["w1"] + (torch.ones(4, device="cuda"),)),
                dict(gated=True), dict(act="gelu"), dict(score="max"), dict(e0=1 << 40),
                dict(out_dtype=torch.float16), dict(out=dict(out=torch.empty(4, 128, device="cuda"))),
                dict(out=dict(topk_ids=torch.empty(4, 2, dtype=torch.int64, device="cuda"))),
                dict(bias=torch.ones(7, device="cuda"), score="sigmoid"), dict(token_mask=torch.ones(3, device="cuda")),
                dict(scale=torch.ones(1, device="cuda")), dict(workspace=torch.empty(8, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f(**bad)
    for bad in (dict(k=0), dict(k=9), dict(bias=torch.ones(8, device="cuda")),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(nv.Nvfp4moeError):
            f(**bad)
    many = torch.zeros(65, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(nv.Nvfp4moeError):
        f(x=many, lg=torch.zeros(65, 8, device="cuda"))
