"""GPU parity of the router's selection, its statistics, the balance loss and
the gradient to the logits, against the float64 oracle.

Bit-exact: expert ids and counts. Rounded, with u = 2^-24:

* exp(x - top), |x - top| <= D: the difference, its product with log2(e) and
  that constant each cost a relative u of the exponent, D u of the value, and
  the hardware's 2^x one unit, 2 u: (3 D + 2) u. A sum of n such adds n u
  (any order), a quotient of two 2 (3 D + 2) u + (n + 2) u, a scale u.
* sigmoid from z = exp(-|x|): the same with D = max |x|, then 1 + z and the
  hardware reciprocal (2 u) and one product: (3 D + 6) u.
* so gates are within (6 D + n + 16) u, n = E (softmax) or k (renormalised)
  bounded by E; probability sums over T tokens add T u; the loss 2 u.
* gradients are sums and products of those: with M the same sums over
  magnitudes (the oracle's second result), 2 (6 D + n + 16) u M, plus half a
  bfloat16 step, 2^-8, of the value where it is stored so.
Values under 2^-126 may flush to zero: 1e-37 absolute.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import formats as F
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


def _logits(seed, T, E, dtype="f32", kind="normal", closed=0.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)).astype(np.float32)
    if kind == "ties":
        x = (np.round(x * 2) / 2).astype(np.float32)
    elif kind == "zero":
        x[:] = 0
    elif kind == "wide":
        x *= 20
    elif kind == "signed_zero":
        x = np.where(rng.random((T, E)) < 0.5, np.float32(0.0), np.float32(-0.0))
    if closed:
        x[rng.random((T, E)) < closed] = -np.inf
        x[0] = -np.inf                              # one row with nothing left
    return gen.to_bf16_bits(x) if dtype == "bf16" else x


def _spread(x, score):
    """D: largest distance of an open logit from its row's largest (softmax) or from 0."""
    x = R._vals(x)
    x = x[np.isfinite(x).any(axis=1)]
    f = np.isfinite(x)
    if not f.any():
        return 0.0
    if score == "sigmoid":
        return float(np.abs(np.where(f, x, 0)).max())
    top = x.max(axis=1, keepdims=True)
    return float(np.where(f, top - np.where(f, x, 0), 0).max())


def _close(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    d = np.abs(got - ref)
    bad = ~(d <= bound + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} out of bound, worst {d.max():.3e} of {np.abs(ref).max():.3e}"


SHAPES = [
    # T, E, k: one token, one expert, powers of two, odd sizes, the largest
    (1, 1, 1), (1, 384, 8), (5, 2, 2), (4096, 8, 2), (1000, 16, 16), (333, 33, 5), (700, 64, 6),
    (129, 65, 8), (257, 130, 7), (300, 200, 64), (2050, 384, 8), (100, 500, 10), (65, 1000, 16),
    (40, 1024, 64),
]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("form", ["softmax", "softmax-sum", "sigmoid", "sigmoid-bias"])
@pytest.mark.parametrize("dtype,kind,closed,masked", [
    ("f32", "normal", 0.0, False), ("bf16", "normal", 0.3, True), ("f32", "ties", 0.9, True),
    ("bf16", "zero", 0.0, False), ("f32", "wide", 0.0, False), ("f32", "signed_zero", 0.0, False),
])
def test_moe_route(nv, T, E, k, form, dtype, kind, closed, masked):
    x = _logits(hash((T, E, k)) % 1000 + 7, T, E, dtype, kind, closed)
    rng = np.random.default_rng(T + E)
    score = form.split("-")[0]
    renorm = form != "softmax"
    bias = (0.2 * rng.normal(size=E)).astype(np.float32) if form == "sigmoid-bias" else None
    mask = rng.random(T) < 0.7 if masked else None
    o = nv.moe_route(to_dev(x), k, score=score, renorm=renorm, scale=2.5,
                     bias=None if bias is None else to_dev(bias),
                     token_mask=None if mask is None else to_dev(mask), stats=True)
    r = R.route(x, k, score, renorm, 2.5, bias, mask)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    assert np.array_equal(from_dev(o["counts"]), r["counts"])
    D = _spread(x, score)
    rel = (6 * D + E + 16) * U
    _close(from_dev(o["gate"]), r["gate"], rel * r["gate"], "gate")
    _close(from_dev(o["prob_sum"]), r["prob_sum"], (rel + T * U) * r["prob_sum"], "prob_sum")
    loss = nv.moe_balance_loss(o["counts"], o["prob_sum"], k, 0.01)
    ref = R.balance_loss(r["counts"], r["prob_sum"], k, 0.01)
    _close(from_dev(loss)[0], ref, (rel + (T + 2) * U) * ref, "loss")
    # without the statistics: the same choice, gates and empty slots
    p = nv.moe_route(to_dev(x), k, score=score, renorm=renorm, scale=2.5,
                     bias=None if bias is None else to_dev(bias),
                     token_mask=None if mask is None else to_dev(mask))
    assert set(p) == {"topk_ids", "gate"}
    assert np.array_equal(from_dev(p["topk_ids"]), r["topk_ids"])
    _close(from_dev(p["gate"]), r["gate"], rel * r["gate"], "gate without statistics")


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score,renorm,dtype,balance,closed", [
    ("softmax", True, "f32", True, 0.0), ("softmax", False, "bf16", True, 0.3),
    ("softmax", True, "bf16", False, 0.9), ("softmax", False, "f32", False, 0.0),
    ("sigmoid", True, "f32", True, 0.3), ("sigmoid", False, "bf16", True, 0.0),
    ("sigmoid", True, "bf16", False, 0.0), ("sigmoid", False, "f32", False, 0.9),
])
def test_moe_route_bwd(nv, T, E, k, score, renorm, dtype, balance, closed):
    import torch
    x = _logits(T + 3 * E + k, T, E, dtype, "normal", closed)
    rng = np.random.default_rng(E)
    ids = R.select(R._vals(x), k, score, None, rng.random(T) < 0.8)
    dg = rng.normal(size=(T, k)).astype(np.float32)
    dg[ids < 0] = np.nan                            # empty slots are not read
    counts = R.route(x, k, score)["counts"] if balance else None
    dloss = np.array([0.75], np.float32)
    got = nv.moe_route_bwd(to_dev(x), to_dev(ids), to_dev(dg), score=score, renorm=renorm, scale=2.5,
                           counts=to_dev(counts) if balance else None, alpha=T * 0.5,
                           dloss=to_dev(dloss))
    assert got.dtype == (torch.bfloat16 if dtype == "bf16" else torch.float32)
    got = R._vals(from_dev(got))
    ref, mag = R.route_bwd(x, ids, dg, score, renorm, 2.5, counts, T * 0.5, 0.75)
    bound = 2 * (6 * _spread(x, score) + E + 16) * U * mag
    _close(got, ref, bound + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0), "dlogits")
    assert np.all(got[ids[:, 0] < 0] == 0)
    # the loss's gradient alone, a gradient of 1 by default; in place over the logits
    if balance:
        b = to_dev(x)
        out = nv.moe_route_bwd(b, to_dev(ids), score=score, renorm=renorm, counts=to_dev(counts),
                               alpha=T * 0.5, dlogits=b)
        ref, mag = R.route_bwd(x, ids, None, score, renorm, 1.0, counts, T * 0.5)
        bound = 2 * (6 * _spread(x, score) + E + 16) * U * mag
        _close(R._vals(from_dev(out)), ref,
               bound + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0), "dlogits of the loss")


ALONE = [
    # T, E, k on both sides of what one workgroup takes with its statistics
    (16, 384, 8), (17, 384, 8), (15, 1024, 64), (33, 300, 9), (1024, 8, 8), (1025, 8, 2), (1000, 7, 3), (4097, 8, 2), (63, 3, 1),
    (64, 64, 6), (65, 64, 6), (63, 33, 17), (64, 128, 4), (3, 5, 5), (2000, 1, 1),
]


@pytest.mark.parametrize("T,E,k", ALONE)
@pytest.mark.parametrize("form", ["softmax", "sigmoid-bias"])
def test_moe_route_few_rows(nv, T, E, k, form):
    x = _logits(T, T, E, "f32", "normal", 0.2)
    score = form.split("-")[0]
    bias = (0.2 * np.random.default_rng(E).normal(size=E)).astype(np.float32) if score == "sigmoid" else None
    o = nv.moe_route(to_dev(x), k, score=score, renorm=False, bias=None if bias is None else to_dev(bias),
                     stats=True)
    r = R.route(x, k, score, False, 1.0, bias)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    assert np.array_equal(from_dev(o["counts"]), r["counts"])
    rel = (6 * _spread(x, score) + E + 16) * U
    _close(from_dev(o["gate"]), r["gate"], rel * r["gate"], "gate")
    _close(from_dev(o["prob_sum"]), r["prob_sum"], (rel + T * U) * r["prob_sum"], "prob_sum")


LONG = [
    # T, E, k, form, dtype: enough rows for one thread each, whole and odd row lengths
    (9001, 8, 2, "softmax", "bf16"), (6000, 5, 3, "softmax-sum", "f32"), (17000, 16, 4, "sigmoid", "f32"),
    (31000, 30, 16, "softmax-sum", "bf16"), (33000, 32, 5, "softmax", "f32"),
    (66001, 64, 6, "sigmoid", "bf16"), (65536, 64, 2, "softmax-sum", "f32"),
    (60000, 57, 3, "softmax", "f32"), (40000, 8, 8, "sigmoid-bias", "f32"),
    (33001, 7, 2, "sigmoid-bias", "bf16"), (300000, 1, 1, "softmax", "f32"),
    (70000, 20, 17, "softmax-sum", "f32"),
]


@pytest.mark.parametrize("T,E,k,form,dtype", LONG)
@pytest.mark.parametrize("kind,closed", [("normal", 0.1), ("ties", 0.0)])
def test_moe_route_long(nv, T, E, k, form, dtype, kind, closed):
    """Many rows of few experts, both directions, with padding."""
    x = _logits(T + E, T, E, dtype, kind, closed)
    rng = np.random.default_rng(E)
    score = form.split("-")[0]
    renorm = form != "softmax"
    bias = (0.2 * rng.normal(size=E)).astype(np.float32) if form == "sigmoid-bias" else None
    mask = rng.random(T) < 0.7
    xm = x.copy()
    xm[~mask] = 0x7FC0 if dtype == "bf16" else np.nan            # padding holds anything
    o = nv.moe_route(to_dev(xm), k, score=score, renorm=renorm, scale=2.5,
                     bias=None if bias is None else to_dev(bias), token_mask=to_dev(mask), stats=True)
    p = nv.moe_route(to_dev(xm), k, score=score, renorm=renorm, scale=2.5,
                     bias=None if bias is None else to_dev(bias), token_mask=to_dev(mask))
    r = R.route(x, k, score, renorm, 2.5, bias, mask)
    rel = (6 * _spread(x, score) + E + 16) * U
    for got in (o, p):
        assert np.array_equal(from_dev(got["topk_ids"]), r["topk_ids"])
        _close(from_dev(got["gate"]), r["gate"], rel * r["gate"], "gate")
    assert np.array_equal(from_dev(o["counts"]), r["counts"])
    _close(from_dev(o["prob_sum"]), r["prob_sum"], (rel + T * U) * r["prob_sum"], "prob_sum")
    dg = rng.normal(size=(T, k)).astype(np.float32)
    dg[r["topk_ids"] < 0] = np.nan
    for with_loss in (True, False):
        got = nv.moe_route_bwd(to_dev(xm), o["topk_ids"], to_dev(dg), score=score, renorm=renorm,
                               scale=2.5, counts=o["counts"] if with_loss else None, alpha=T * 0.5)
        ref, mag = R.route_bwd(x, r["topk_ids"], dg, score, renorm, 2.5,
                               r["counts"] if with_loss else None, T * 0.5)
        bound = 2 * rel * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
        _close(R._vals(from_dev(got)), ref, bound, "dlogits")


def test_moe_route_bwd_foreign_indices(nv):
    """Indices outside [0, E) are empty slots; one expert twice counts twice."""
    T, E, k = 3, 40, 4
    x = _logits(5, T, E)
    ids = np.array([[1, -1, 40, 3], [-7, 2 ** 31 - 1, 40, -1], [9, 9, 2, -1]], np.int32)
    dg = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    clean = np.where((ids < 0) | (ids >= E), -1, ids).astype(np.int32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = from_dev(nv.moe_route_bwd(to_dev(x), to_dev(ids), to_dev(dg), score=score, renorm=renorm))
            ref, mag = R.route_bwd(x, clean, dg, score, renorm)
            _close(got, ref, 2 * (6 * _spread(x, score) + E + 16) * U * mag, f"{score} {renorm}")


def test_moe_route_nan_never_selected(nv):
    x = _logits(6, 64, 100)
    x[3, 5] = np.nan
    x[4] = np.nan
    o = nv.moe_route(to_dev(x), 8, stats=True)
    ids = from_dev(o["topk_ids"])
    assert ids.min() >= -1 and ids.max() < 100
    assert 5 not in ids[3] and (ids[4] == -1).all()
    keep = np.arange(64) > 4
    assert np.array_equal(ids[keep], R.select(R._vals(x[keep]), 8))


def test_moe_route_empty_and_no_tokens(nv):
    import torch
    o = nv.moe_route(torch.empty((0, 16), device="cuda"), 4, stats=True)
    assert o["topk_ids"].shape == (0, 4) and from_dev(o["counts"]).sum() == 0
    assert from_dev(nv.moe_balance_loss(o["counts"], o["prob_sum"], 4, 1.0))[0] == 0
    x = torch.full((70, 16), -float("inf"), device="cuda")
    o = nv.moe_route(x, 4, stats=True)
    assert (from_dev(o["topk_ids"]) == -1).all() and (from_dev(o["gate"]) == 0).all()
    assert from_dev(o["counts"]).sum() == 0 and (from_dev(o["prob_sum"]) == 0).all()
    d = nv.moe_route_bwd(x, o["topk_ids"], torch.full((70, 4), float("nan"), device="cuda"),
                         counts=o["counts"], alpha=1.0)
    assert (from_dev(d) == 0).all()
    assert nv.moe_route_bwd(x[:0], o["topk_ids"][:0]).shape == (0, 16)


@pytest.mark.parametrize("E", [7, 64, 130])
def test_moe_route_unaligned_views(nv, E):
    """Rows of a larger buffer at an odd offset, buffers behind them untouched."""
    import torch
    T, k = 50, 3
    x = _logits(8, T + 1, E, "bf16")
    o = {"topk_ids": torch.full((T + 1, k), -9, dtype=torch.int32, device="cuda"),
         "gate": torch.full((T + 1, k), -9.0, device="cuda")}
    nv.moe_route(to_dev(x)[1:], k, out={n: b[:T] for n, b in o.items()})
    r = R.route(x[1:], k)
    assert np.array_equal(from_dev(o["topk_ids"])[:T], r["topk_ids"])
    assert (from_dev(o["topk_ids"])[T:] == -9).all() and (from_dev(o["gate"])[T:] == -9).all()
    buf = torch.full((T + 2, E), 7.0, dtype=torch.bfloat16, device="cuda")
    dg = np.random.default_rng(2).normal(size=(T, k)).astype(np.float32)
    nv.moe_route_bwd(to_dev(x)[1:], to_dev(r["topk_ids"]), to_dev(dg), dlogits=buf[1:T + 1])
    got = R._vals(from_dev(buf))
    assert (got[0] == 7).all() and (got[T + 1] == 7).all()
    ref, mag = R.route_bwd(x[1:], r["topk_ids"], dg)
    _close(got[1:T + 1], ref, 2 * (6 * _spread(x, "softmax") + E + 16) * U * mag + 2.0 ** -8 * np.abs(ref), "view")


def test_moe_route_many_tokens_repeatable(nv):
    """The persistent grid's later rounds; the same bits on every call."""
    import torch
    T, E, k = 70001, 48, 4
    x = _logits(9, T, E)
    xd = to_dev(x)
    a = nv.moe_route(xd, k, score="sigmoid", stats=True)
    b = nv.moe_route(xd, k, score="sigmoid", stats=True)
    assert all(torch.equal(a[n], b[n]) for n in a)
    r = R.route(x, k, "sigmoid")
    assert np.array_equal(from_dev(a["topk_ids"]), r["topk_ids"])
    assert np.array_equal(from_dev(a["counts"]), r["counts"])
    rel = (6 * _spread(x, "sigmoid") + E + 16 + T) * U
    _close(from_dev(a["prob_sum"]), r["prob_sum"], rel * r["prob_sum"], "prob_sum")


def test_moe_route_refuses(nv):
    import torch
    x = torch.zeros((8, 16), device="cuda")
    with pytest.raises(ValueError):
        nv.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        nv.moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        nv.moe_route(x, 2, score="tanh")
    with pytest.raises(ValueError):
        nv.moe_route(x, 2, score="sigmoid", bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        nv.moe_route(x, 2, token_mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        nv.moe_route(x, 2, out={"gate": torch.empty((8, 3), device="cuda")})
    with pytest.raises(TypeError):
        nv.moe_route(x, 2, token_mask=[True] * 8)
    nv.moe_route(x, 2, scale=np.float32(2.5))                            # any number
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_route(x, 2, bias=torch.zeros(16, device="cuda"))          # softmax
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_route(x, 17)
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_route(x.repeat(1000, 1), 2, stats=True,
                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    ids = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        nv.moe_route_bwd(x, ids, torch.zeros((8, 3), device="cuda"))
    with pytest.raises(ValueError):
        nv.moe_route_bwd(x, ids[:4])
    with pytest.raises(ValueError):
        nv.moe_route_bwd(x, ids, dlogits=torch.zeros((8, 16), dtype=torch.bfloat16, device="cuda"))


def test_route_graphs_and_streams(nv):
    """Two captured graphs (each with its own workspace) replayed in turn on
    two streams with eager work between them give the eager bits."""
    import torch
    T, E, k = 3000, 130, 6
    xs = [to_dev(_logits(20 + i, T, E)) for i in range(2)]
    dg = to_dev(np.random.default_rng(3).normal(size=(T, k)).astype(np.float32))

    def step(x):
        o = nv.moe_route(x, k, stats=True)
        loss = nv.moe_balance_loss(o["counts"], o["prob_sum"], k, 0.1)
        return [*o.values(), loss, nv.moe_route_bwd(x, o["topk_ids"], dg, counts=o["counts"], alpha=0.1)]

    ref = [[t.clone() for t in step(x)] for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        step(xs[0])
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            assert all(torch.equal(a, b) for a, b in zip(o, r))


def test_route_past_32_bit_offsets(nv):
    """More than 2^32 logits: rows at both ends against the oracle, equal rows
    between (which go to the lowest experts) counted whole."""
    import torch
    T, E, k = 4_300_000, 1000, 2
    tail = 70
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    ends = _logits(11, 2 * tail, E, "bf16")
    x[:tail], x[-tail:] = to_dev(ends[:tail]), to_dev(ends[tail:])
    o = nv.moe_route(x, k, stats=True)
    r = R.route(ends, k)
    ids = o["topk_ids"]
    assert np.array_equal(from_dev(torch.cat([ids[:tail], ids[-tail:]])), r["topk_ids"])
    assert bool((ids[tail:-tail] == torch.arange(k, device="cuda", dtype=torch.int32)).all())
    want = r["counts"].copy()
    want[:k] += T - 2 * tail
    want[E] = T
    assert np.array_equal(from_dev(o["counts"]), want)
    dg = torch.ones((T, k), device="cuda")
    dg[:, 1] = -1.0
    d = nv.moe_route_bwd(x, ids, dg, dlogits=x)                  # in place
    ref, mag = R.route_bwd(ends, r["topk_ids"], np.tile([1.0, -1.0], (2 * tail, 1)))
    got = R._vals(from_dev(torch.cat([d[:tail], d[-tail:]])))
    _close(got, ref, 2 * (6 * _spread(ends, "softmax") + E + 16) * U * mag + 2.0 ** -8 * np.abs(ref), "ends")
    assert bool((d[tail:-tail, 0] == 0.5).all()) and bool((d[tail:-tail, 1] == -0.5).all())
    assert int(torch.count_nonzero(d[tail:-tail])) == 2 * (T - 2 * tail)


def test_route_lowest_values_are_open(nv):
    """The type's lowest value is a logit like any other: selected behind the
    others, never in place of -inf; extreme spreads stay finite."""
    lowest = np.finfo(np.float32).min
    x = np.full((40, 70), lowest, np.float32)
    x[1, 3] = 5
    x[2, ::2] = -np.inf
    x[3, 69] = np.finfo(np.float32).max
    x[4] = np.linspace(-3e38, 3e38, 70, dtype=np.float32)
    for k in (1, 8, 40):
        for score in ("softmax", "sigmoid"):
            o = nv.moe_route(to_dev(x), k, score=score, renorm=False, stats=True)
            r = R.route(x, k, score, False)
            assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
            assert np.array_equal(from_dev(o["counts"]), r["counts"])
            assert np.allclose(from_dev(o["gate"]), r["gate"], rtol=1e-5, atol=1e-30)
            d = from_dev(nv.moe_route_bwd(to_dev(x), o["topk_ids"], o["gate"], score=score,
                                          renorm=False, counts=o["counts"], alpha=1.0))
            assert np.isfinite(d).all()


@pytest.mark.parametrize("E,k", [(12, 3), (100, 8), (384, 8)])
def test_route_near_ties_under_a_bias(nv, E, k):
    """Keys that float32 cannot tell apart: saturated scores, biases of one
    float32 step, equal experts; infinite biases close or force an expert."""
    T = 200
    rng = np.random.default_rng(E)
    x = (12 + 8 * rng.random((T, E))).astype(np.float32)         # sigmoid within 1e-5 of 1
    x[::3] = np.round(x[::3])
    bias = (1 + rng.integers(0, 4, size=E) * 2.0 ** -23).astype(np.float32)
    bias[E - 1] = -np.inf
    bias[E - 2] = np.inf
    o = nv.moe_route(to_dev(x), k, score="sigmoid", bias=to_dev(bias))
    ids = from_dev(o["topk_ids"])
    assert np.array_equal(ids, R.select(R._vals(x), k, "sigmoid", bias))
    assert (ids[:, 0] == E - 2).all() and not (ids == E - 1).any()
    zero = np.zeros((T, E), np.float32)
    same = nv.moe_route(to_dev(zero), k, score="sigmoid", bias=to_dev(np.zeros(E, np.float32)))
    assert (from_dev(same["topk_ids"]) == np.arange(k)).all()


def test_route_two_eager_streams(nv):
    """Calls of two streams at once, each with its own workspace from torch."""
    import torch
    xs = [to_dev(_logits(30 + i, 20000, 130)) for i in range(2)]
    ref = [nv.moe_route(x, 6, stats=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                outs.append(nv.moe_route(x, 6, stats=True))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert all(torch.equal(o[n], ref[i % 2][n]) for n in o)


@pytest.mark.parametrize("T,E,k", [(40, 7, 2), (40, 60, 5), (40, 300, 8), (33000, 8, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_tiny_sigmoid_scores(nv, T, E, k, renorm):
    """Scores down to 2^-126: their quotients and gradients are those of any
    other row's, though 1 / (a sum of them) squared is far out of range. A
    product of scores that is below 2^-126 may be 0: 2^-126 times the gradient
    and the loss's coefficient, absolute."""
    rng = np.random.default_rng(T + E)
    x = (-86 + 4 * rng.random((T, E))).astype(np.float32)
    x[::2] += 60
    dg = (50 * rng.normal(size=(T, k))).astype(np.float32)
    o = nv.moe_route(to_dev(x), k, score="sigmoid", renorm=renorm, stats=True)
    r = R.route(x, k, "sigmoid", renorm)
    assert np.array_equal(from_dev(o["topk_ids"]), r["topk_ids"])
    rel = (6 * _spread(x, "sigmoid") + E + 16) * U
    _close(from_dev(o["gate"]), r["gate"], rel * r["gate"], "gate")
    _close(from_dev(o["prob_sum"]), r["prob_sum"], (rel + T * U) * r["prob_sum"], "prob_sum")
    got = from_dev(nv.moe_route_bwd(to_dev(x), o["topk_ids"], to_dev(dg), score="sigmoid", renorm=renorm,
                                    counts=o["counts"], alpha=float(T)))
    ref, mag = R.route_bwd(x, r["topk_ids"], dg, "sigmoid", renorm, 1.0, r["counts"], float(T))
    _close(got, ref, 2 * rel * mag + 2.0 ** -126 * 200, "dlogits")


@pytest.mark.parametrize("T,E,k", [(100, 384, 8), (300, 64, 6), (40000, 8, 2)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd_scales_with_its_gradients(nv, T, E, k, renorm, score):
    """The backward is linear in dgate and alpha: 2^80 times both (exact in
    every product and sum, and far inside the range) gives 2^80 times the bits."""
    rng = np.random.default_rng(T + E)
    x = to_dev((2 * rng.normal(size=(T, E))).astype(np.float32))
    dg = rng.normal(size=(T, k)).astype(np.float32)
    o = nv.moe_route(x, k, score=score, renorm=renorm, stats=True)
    got = [from_dev(nv.moe_route_bwd(x, o["topk_ids"], to_dev(dg * np.float32(c)), score=score,
                                     renorm=renorm, counts=o["counts"], alpha=float(T) * c))
           for c in (1.0, 2.0 ** 80)]
    assert np.array_equal(got[0] * np.float32(2.0 ** 80), got[1])
