"""Gradient lists on the GPU beyond single launches and single looks: tensors
that change under a handle. Bounds as derived in test_gpu_gradclip."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
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


def test_handle_of_a_tensor_cut_short(nv):
    """The same address with fewer elements: the sum leaves out what is no
    longer the tensor's, and a clip in place leaves it as it is."""
    import torch
    m = torch.full((5000,), 3.0, device="cuda")
    t = m[:]
    h = nv.GradList([t])
    assert from_dev(nv.moe_grad_sumsq(h))[0] == 9.0 * 5000
    t.data = m[:16]
    s = nv.moe_grad_sumsq(h)
    assert from_dev(s)[0] == 9.0 * 16
    nv.moe_grad_clip(h, s, 6.0)                               # norm 12: halved
    assert from_dev(m[:16]) == pytest.approx([1.5] * 16, rel=1e-6)
    assert (from_dev(m[16:]) == 3.0).all()


def test_handle_of_a_tensor_of_another_type(nv):
    """The same address as the other type, in the sum and as an output."""
    import torch
    bits = gen.to_bf16_bits(np.random.default_rng(1).normal(size=6000).astype(np.float32))
    m = to_dev(bits)                                          # pairs of them are finite float32 too
    t = m.view(torch.float32)
    h = nv.GradList([t])
    nv.moe_grad_sumsq(h)
    t.data = m[:3000]
    s = nv.moe_grad_sumsq(h)
    assert from_dev(s)[0] == pytest.approx(R.sumsq([bits[:3000]]), rel=2.0 ** -52 * 3008)
    f = torch.zeros(3000, device="cuda")
    with pytest.raises(ValueError):                           # float32 gradients, bfloat16 outputs
        nv.moe_grad_clip([f], s, 1.0, outs=h)


def test_handle_within_a_graph_keeps_what_was_captured(nv):
    """A replay uses what the capture took; the next eager call what is there."""
    import torch
    m = torch.full((100,), 2.0, device="cuda")
    t = m[:]
    h = nv.GradList([t])
    nv.moe_grad_sumsq(h)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = nv.moe_grad_sumsq(h)
    t.data = m[:10]
    for _ in range(3):
        s.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert from_dev(s)[0] == 400.0 and from_dev(nv.moe_grad_sumsq(h))[0] == 40.0


@pytest.mark.parametrize("bad", [None, "inf", "-inf", "nan"])
@pytest.mark.parametrize("max_norm", ["inf", "1e300", "1.0", "0.0"])
@pytest.mark.parametrize("in_place", [True, False])
def test_infinite_bound_and_norm(nv, bad, max_norm, in_place):
    """No bound leaves every gradient its bits, with a norm of infinity too (a
    bound past float32 is one of infinity there); a NaN norm makes all NaN."""
    import torch
    host = [np.array([3.0, -4.0, 0.0], np.float32), gen.to_bf16_bits(np.full(9, 2.0, np.float32))]
    if bad:
        host[0][2] = float(bad)
    ts = [to_dev(h) for h in host]
    outs = ts if in_place else [torch.empty_like(t) for t in ts]
    s = nv.moe_grad_sumsq(ts)
    norm = nv.moe_grad_clip(ts, s, float(max_norm), outs=None if in_place else outs)
    total = R.sumsq(host)
    with np.errstate(invalid="ignore"):                       # infinity by a factor of 0
        ref_norm, ref = R.clip(host, total, float(max_norm))
    assert np.array_equal(from_dev(norm), np.array([ref_norm], np.float32), equal_nan=True)
    for o, r, h in zip(outs, ref, host):
        got = R._vals(from_dev(o))
        if float(max_norm) > 1e30 and bad != "nan":
            assert np.array_equal(from_dev(o), h)
        else:
            assert np.array_equal(np.isnan(got), np.isnan(r))
            ok = ~np.isnan(r)
            eps = 3 * 2.0 ** -24 + (2.0 ** -8 if h.dtype == np.uint16 else 0.0)
            assert (np.abs(got[ok] - r[ok]) <= eps * np.abs(r[ok]) + 1e-37).all()


# Tables hold 280 tensors of a sum's launch, 180 of a scaling's, 16 of a short
# list's; chunks have 2^11 elements up to 2^23 of them in all, then 2^12, 2^13
# and 2^14; above 2048 chunks a workgroup goes through several, of several
# tensors where those are short.
LONG = {
    "180": [700 + i for i in range(180)],
    "181": [700 + i for i in range(181)],
    "280": [300 + i % 7 for i in range(280)],
    "281": [300 + i % 7 for i in range(281)],
    "600-with-empty": [(i * 977) % 5003 * (i % 5 > 0) for i in range(600)],
    "561-of-one": [1] * 561,
    "runs-over-tensors": [50000 + i for i in range(120)],
    "runs-over-short-ones": [3] * 100 + [7_000_000] + [5] * 60,
    "chunks-of-2^12": [6_000_001, 1, 4097, 3_000_000, 70_000],
    "chunks-of-2^13": [9_000_000, 0, 8_191, 8_192, 8_193, 12_000_001],
    "chunks-of-2^14": [30_000_001] + [2, 16384, 0, 16385] * 10 + [20_000_003],
    "three-chunks-a-run": [60_000_000] + [1, 2, 3] * 20 + [45_000_001, 16_383] + [9] * 17,
}


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("types", ["f32", "mixed"])
@pytest.mark.parametrize("in_place", [True, False])
def test_long_lists(nv, name, types, in_place):
    """The sum and every element, against 64-bit torch: random values without
    zeros (a chunk left out or scaled twice shows), tensors one element off the
    16-byte grid, memory between them left as it is."""
    import torch
    sizes = LONG[name]
    kinds = [torch.bfloat16 if types == "mixed" and i % 2 else torch.float32 for i in range(len(sizes))]
    gen_ = torch.Generator(device="cuda").manual_seed(len(sizes))

    def flat(t, fill):
        n = sum(m + 1 for m, u in zip(sizes, kinds) if u == t) + 1
        if not fill:
            return torch.full((n,), 7.0, dtype=t, device="cuda")
        f = torch.rand(n, generator=gen_, device="cuda") + 0.5
        return (f * torch.where(torch.rand(n, generator=gen_, device="cuda") < 0.5, -1e-2, 1e-2)).to(t)

    def views(buf):
        at, out = dict.fromkeys(buf, 1), []
        for m, t in zip(sizes, kinds):
            out.append(buf[t][at[t]:at[t] + m])
            at[t] += m + 1
        return out

    buf = {t: flat(t, True) for t in dict.fromkeys(kinds)}
    obuf = buf if in_place else {t: flat(t, False) for t in buf}
    before = {t: b.clone() for t, b in buf.items()}
    used = {t: torch.zeros(b.numel(), dtype=torch.bool, device="cuda") for t, b in buf.items()}
    for v in views(used):
        v.fill_(True)
    grads, outs = nv.GradList(views(buf)), nv.GradList(views(obuf))
    s = nv.moe_grad_sumsq(grads)
    total = sum(float(b[used[t]].double().square().sum()) for t, b in before.items())
    assert float(s) == pytest.approx(total, rel=2.0 ** -52 * (sum(sizes) + 8))
    bound = 0.3 * np.sqrt(total)
    norm = nv.moe_grad_clip(grads, s, bound, outs=outs)
    assert float(norm) == pytest.approx(np.sqrt(total), rel=2.0 ** -23)
    coef = bound / (np.sqrt(total) + 1e-6)
    for t, b in obuf.items():
        want = before[t][used[t]].double() * coef
        eps = 3 * 2.0 ** -24 + (2.0 ** -8 if t == torch.bfloat16 else 0.0)
        assert bool(((b[used[t]].double() - want).abs() <= eps * want.abs()).all())
        rest = before[t][~used[t]] if in_place else torch.full_like(b[~used[t]], 7.0)
        assert torch.equal(b[~used[t]], rest)
        if not in_place:
            assert torch.equal(buf[t], before[t])
