"""GPU parity of the global gradient norm and the clipping, against float64.

The sum of squares is formed in 64 bits: within n 2^-52 of the oracle's.
max_norm reaches the library as a float32 (the tests' bounds are not float32
values: one rounding, a relative 2^-24 of the factor), the factor is rounded
once to float32 and multiplied once: 3 * 2^-24 relative, plus half a bfloat16
step (2^-8) where the tensor is bfloat16; the float32 norm is rounded once.
"""

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


def _grads(seed, sizes, types, scale=1.0):
    rng = np.random.default_rng(seed)
    out = []
    for n, t in zip(sizes, types):
        g = (rng.normal(size=n) * scale).astype(np.float32)
        out.append(gen.to_bf16_bits(g) if t == "bf16" else g)
    return out


def _check(got, ref, bits, what):
    got = R._vals(got)
    bound = (3 * 2.0 ** -24 + (2.0 ** -8 if bits else 0.0)) * np.abs(ref) + 1e-37
    assert (np.abs(got - ref) <= bound).all(), what


LISTS = [
    [1], [0, 3, 0], [4096, 17], [16384], [16385], [2048] * 8, [2048] * 8 + [1], [100] * 16, [100] * 17,
    [16385, 1, 16383], [100000, 7, 65536, 3],
    [3] * 95, [3] * 96, [5, 0] * 97, [1000 + 37 * i for i in range(200)], [3000001],
]


@pytest.mark.parametrize("sizes", LISTS, ids=[f"{len(s)}x{max(s)}" for s in LISTS])
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_and_clip(nv, sizes, types, shift):
    """Every list in place and into copies, clipped and within the bound; with
    shift, every tensor starts off the 16-byte grid inside a larger buffer
    whose other elements stay as they are."""
    import torch
    kinds = [types if types != "mixed" else ("bf16" if i % 2 else "f32") for i in range(len(sizes))]
    host = _grads(len(sizes), sizes, kinds, 1e-2)
    total = R.sumsq(host)

    def put(fill):
        bufs, views = [], []
        for h, t in zip(host, kinds):
            b = torch.full((len(h) + 8,), 7.0, dtype=torch.bfloat16 if t == "bf16" else torch.float32,
                           device="cuda")
            v = b[shift:shift + len(h)]
            if fill:
                v.copy_(to_dev(h))
            bufs.append(b)
            views.append(v)
        return bufs, views

    for share in (0.3, 2.0):
        max_norm = share * np.sqrt(total)
        for in_place in (True, False):
            bufs, views = put(True)
            obufs, oviews = (bufs, views) if in_place else put(False)
            s = nv.moe_grad_sumsq(views)
            norm = nv.moe_grad_clip(views, s, max_norm, outs=None if in_place else oviews)
            assert from_dev(s)[0] == pytest.approx(total, rel=2.0 ** -52 * (sum(sizes) + 8))
            ref_norm, ref = R.clip(host, total, max_norm)
            assert from_dev(norm)[0] == pytest.approx(ref_norm, rel=2.0 ** -23)
            for b, r, t, h in zip(obufs, ref, kinds, host):
                g = from_dev(b)
                _check(g[shift:shift + len(h)], r, t == "bf16", "clipped")
                rest = R._vals(np.concatenate([g[:shift], g[shift + len(h):]]))
                assert (rest == 7).all()
            if not in_place:
                for v, h in zip(views, host):
                    assert np.array_equal(from_dev(v), h)


def test_extreme_scales(nv):
    """Squares that would overflow or vanish in 32 bits; NaN and infinity show."""
    import torch
    big = torch.tensor([3e30, 4e30], device="cuda")
    norm = nv.moe_grad_clip([big], nv.moe_grad_sumsq([big]), 1.0)
    assert from_dev(norm)[0] == pytest.approx(5e30, rel=1e-6)
    assert from_dev(big) == pytest.approx([0.6, 0.8], rel=1e-6)
    tiny = torch.tensor([3e-30, 4e-30], device="cuda")
    assert from_dev(nv.moe_grad_sumsq([tiny]))[0] == pytest.approx(25e-60, rel=1e-6)
    bad = [torch.tensor([1.0, float("nan")], device="cuda"), torch.ones(3, device="cuda")]
    norm = nv.moe_grad_clip(bad, nv.moe_grad_sumsq(bad), 1.0)
    assert np.isnan(from_dev(norm)[0]) and np.isnan(from_dev(bad[1])).all()
    inf = [torch.tensor([float("inf")], device="cuda"), torch.ones(3, device="cuda")]
    norm = nv.moe_grad_clip(inf, nv.moe_grad_sumsq(inf), 1.0)
    assert np.isinf(from_dev(norm)[0]) and (from_dev(inf[1]) == 0).all()
    zero = torch.zeros(5, device="cuda")
    assert from_dev(nv.moe_grad_clip([zero], nv.moe_grad_sumsq([zero]), 1.0))[0] == 0
    one = torch.ones(4, device="cuda")
    nv.moe_grad_clip([one], nv.moe_grad_sumsq([one]), 0.0)
    assert (from_dev(one) == 0).all()


def test_empty_list_and_added_sums(nv):
    import torch
    s = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
    nv.moe_grad_sumsq([], sumsq=s)
    assert from_dev(s)[0] == 0
    assert from_dev(nv.moe_grad_clip([], s + 9.0, 1.0))[0] == 3
    # two ranks' sums added: both clip by the joint norm
    a, b = torch.full((3,), 2.0, device="cuda"), torch.full((4,), 1.0, device="cuda")
    joint = nv.moe_grad_sumsq([a]) + nv.moe_grad_sumsq([b])
    nv.moe_grad_clip([a], joint, 1.0)
    assert from_dev(a) == pytest.approx([0.5] * 3, rel=1e-6)


def test_large_offsets(nv):
    """Elements past 2^31 of one tensor are read, scaled and written."""
    import torch
    n = (1 << 31) + 16385
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1] = 3.0
    g[0] = 4.0
    s = nv.moe_grad_sumsq([g])
    assert from_dev(s)[0] == 25.0
    nv.moe_grad_clip([g], s, 2.5)
    assert float(g[-1]) == 1.5 and float(g[0]) == 2.0 and int(torch.count_nonzero(g)) == 2


def test_grad_list_handle(nv):
    """A list made once follows tensors whose memory is replaced, and gives the
    same bits on every call."""
    import torch
    host = _grads(5, [70000, 33], ["f32", "f32"])
    ts = [to_dev(h) for h in host]
    h = nv.GradList(ts)
    assert len(h) == 2
    a, b = nv.moe_grad_sumsq(h), nv.moe_grad_sumsq(h)
    assert torch.equal(a, b)
    ts[1].data = torch.full((50,), 2.0, device="cuda")
    assert from_dev(nv.moe_grad_sumsq(h))[0] == pytest.approx(R.sumsq(host[:1]) + 200.0, rel=1e-12)
    ts[0].data = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        nv.moe_grad_sumsq(h)


def test_refusals(nv):
    import torch
    a, b = torch.ones(8, device="cuda"), torch.ones(9, device="cuda")
    s = nv.moe_grad_sumsq([a, b])
    with pytest.raises(ValueError):
        nv.GradList([a, a])
    with pytest.raises(ValueError):
        nv.GradList([b[:5], b[4:]])
    with pytest.raises(ValueError):
        nv.GradList([a.half()])
    with pytest.raises(ValueError):
        nv.GradList([torch.ones((4, 4), device="cuda").t()])
    with pytest.raises(ValueError):
        nv.moe_grad_sumsq([])
    with pytest.raises(ValueError):
        nv.moe_grad_clip([a], s, 1.0, outs=[b])                  # sizes
    with pytest.raises(ValueError):
        nv.moe_grad_clip([a], s, 1.0, outs=[a.bfloat16()])       # types
    with pytest.raises(ValueError):
        nv.moe_grad_clip([b[:4], b[5:]], s, 1.0, outs=[a[:4], b[1:5]])   # an out over a gradient
    with pytest.raises(ValueError):
        nv.moe_grad_clip([a], s.float(), 1.0)
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_grad_clip([a], s, -1.0)
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_grad_sumsq([torch.ones(1 << 20, device="cuda")],
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_graph_replays(nv):
    """Captured with its workspace, replayed over changing gradients."""
    import torch
    host = [_grads(30 + i, [50000, 1000], ["f32", "bf16"]) for i in range(3)]
    ts = [to_dev(h) for h in host[0]]
    outs = [torch.empty_like(t) for t in ts]
    grads, clipped = nv.GradList(ts), nv.GradList(outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = nv.moe_grad_sumsq(grads)
        norm = nv.moe_grad_clip(grads, s, 0.5, outs=clipped)
    for h in host * 2:
        for t, v in zip(ts, h):
            t.copy_(to_dev(v))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in ts]
        n = nv.moe_grad_clip(ts, nv.moe_grad_sumsq(ts), 0.5, outs=want)
        assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(want, outs))
        assert from_dev(norm)[0] == pytest.approx(np.sqrt(R.sumsq(h)), rel=2.0 ** -23)
