"""GPU parity of the MXFP4 calls against the oracle.

Bit-exact: codes, scales, values, grouping, re-quantized MXFP8. The product:
sums of a block of 32 are exact, so K / 32 additions of float32 round, each by
at most one unit of 2^-23 of the running magnitude (the matrix unit may cut
where it adds): (K / 32 + 1) 2^-23 times the sum over magnitudes, and half a
bfloat16 step, 2^-8 of the value, where it is stored so.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import formats as F
from oracle import gemm as GM
from oracle import mxfp4 as M4
from oracle import mxfp8 as MX
from oracle import permute as PM
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


def _rows(seed, rows, cols, dtype):
    """Values over many binades, with zeros, signed zeros and whole blocks of one value."""
    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(rows, cols)) * np.exp2(rng.integers(-8, 8, (rows, cols)))).astype(np.float32)
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[rng.random((rows, cols)) < 0.05] = -0.0
    x[::3, :32] = 0.0
    x[1::5, -32:] = 2.5
    return gen.to_bf16_bits(x) if dtype == "bf16" else x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (64, 256), (129, 1056), (7, 8192), (1031, 32), (2, 16416)])
def test_quantize(nv, rows, cols, dtype):
    x = _rows(rows + cols, rows, cols, dtype)
    codes, scales = nv.mxfp4_quantize(to_dev(x))
    rc, rs = M4.quantize(x)
    assert np.array_equal(from_dev(scales), rs)
    assert np.array_equal(from_dev(codes), rc)
    v = nv.mxfp4_dequantize(codes, scales)
    assert np.array_equal(from_dev(v), M4.dequantize(rc, rs).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_every_exponent(nv, dtype):
    """Every block exponent, with the values at and next to the ties of each code."""
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.96875, 6], np.float64)
    near = np.concatenate([ties, -ties])
    if dtype == "f32":
        up = np.nextafter(near.astype(np.float32), np.float32(7)).astype(np.float64)
        near = np.stack([near, up, np.nextafter(near.astype(np.float32), np.float32(-7)).astype(np.float64)])
        near = near.clip(-6, 6)
    else:
        near = near[None]
    e = np.arange(-140, 126, dtype=np.float64)
    with np.errstate(over="ignore"):
        x = (near[None] * np.exp2(e)[:, None, None]).reshape(-1, 32).astype(np.float32)
    x = x[np.isfinite(x).all(axis=1)]
    if dtype == "bf16":
        x = gen.to_bf16_bits(x)
    codes, scales = nv.mxfp4_quantize(to_dev(x))
    rc, rs = M4.quantize(x)
    assert np.array_equal(from_dev(scales), rs)
    bad = np.nonzero((from_dev(codes) != rc).any(axis=1))[0]
    assert bad.size == 0, (bad[:8], rs[bad[:8], 0], from_dev(codes)[bad[0]], rc[bad[0]])


def test_quantize_largest_and_smallest(nv):
    big, tiny = np.finfo(np.float32).max, np.float32(2.0 ** -149)
    x = np.zeros((6, 32), np.float32)
    x[0] = big
    x[1, 3], x[1, 4] = -big, tiny
    x[2] = tiny
    x[3, 0] = np.float32(2.0 ** -126)
    x[4, :2] = 1.0, 2.0 ** -140
    codes, scales = nv.mxfp4_quantize(to_dev(x))
    rc, rs = M4.quantize(x)
    assert np.array_equal(from_dev(scales), rs) and np.array_equal(from_dev(codes), rc)


@pytest.mark.parametrize("out", ["float32", "bfloat16"])
def test_dequantize_every_code_and_scale(nv, out):
    import torch
    dt = getattr(torch, out)
    codes = np.tile((np.arange(16) | (np.arange(16)[::-1] << 4)).astype(np.uint8), (255, 1))
    scales = np.arange(255, dtype=np.uint8)[:, None]
    got = nv.mxfp4_dequantize(to_dev(codes), to_dev(scales), out_dtype=dt)
    with np.errstate(over="ignore"):
        ref = M4.dequantize(codes, scales).astype(np.float32)      # 6 * 2^127 is infinite
    assert np.array_equal(got.float().cpu().numpy(), ref)
    e4 = np.tile(np.delete(np.arange(256, dtype=np.uint8), [0x7F, 0xFF])[:224], (255, 1))
    e8 = np.tile(scales, (1, 7))
    got = nv.mxfp8_dequantize(to_dev(e4), to_dev(e8), out_dtype=dt)
    with np.errstate(over="ignore"):
        ref = MX.dequantize(e4, e8).astype(np.float32)
    if dt == torch.bfloat16:
        want = torch.from_numpy(ref).bfloat16()
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    else:
        assert np.array_equal(from_dev(got), ref)


def test_quantize_live_rows_only(nv):
    import torch
    x = to_dev(_rows(5, 100, 160, "bf16"))
    for live in (0, 1, 37, 100, 1000):
        codes = torch.full((100, 80), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((100, 5), 0x5A, dtype=torch.uint8, device="cuda")
        nv.mxfp4_quantize(x, offsets=torch.tensor([0, live], device="cuda"), codes=codes, scales=scales)
        n = min(live, 100)
        rc, rs = nv.mxfp4_quantize(x)
        assert torch.equal(codes[:n], rc[:n]) and torch.equal(scales[:n], rs[:n])
        assert (codes[n:] == 0xA5).all() and (scales[n:] == 0x5A).all()
    assert nv.mxfp4_quantize(x[:0])[0].shape == (0, 80)


def _routed(seed, T, k, n_experts, e0, G, how="uniform"):
    if how == "uniform":
        return gen.route_uniform(seed, T, n_experts, k)
    if how == "one":                                       # everything on one expert
        return np.full((T, k), e0 + G - 1, np.int32) if k == 1 else gen.route_uniform(seed, T, k, k) + e0
    return np.full((T, k), e0 - 1 if e0 else n_experts + 5, np.int32)     # nothing local


@pytest.mark.parametrize("T,k,n_experts,e0,G,how", [
    (1, 1, 4, 0, 4, "uniform"), (300, 2, 8, 2, 4, "uniform"), (64, 3, 12, 0, 12, "uniform"),
    (5000, 4, 16, 4, 8, "uniform"), (200, 2, 8, 0, 8, "one"), (77, 2, 8, 3, 4, "none"),
])
def test_group(nv, T, k, n_experts, e0, G, how):
    ids = _routed(T, T, k, n_experts, e0, G, how)
    o = nv.moe_group(to_dev(ids), e0, G)
    off, pad, tok, slot = PM.permute(ids, e0, G)
    M = off[-1]
    assert np.array_equal(from_dev(o["offsets"]), off) and np.array_equal(from_dev(o["padded_offsets"]), pad)
    assert np.array_equal(from_dev(o["row_token"])[:M], tok) and np.array_equal(from_dev(o["row_slot"])[:M], slot)
    pair = np.full((T, k), -1, np.int32)
    pair[tok, slot] = np.arange(M)
    assert np.array_equal(from_dev(o["pair_row"]), pair)
    assert "pair_row" not in nv.moe_group(to_dev(ids), e0, G, out={})


def _check_product(nv, a, b, off, N, K, dtype, row_token=None, cap=None, m_extra=0):
    import torch
    dt = getattr(torch, dtype)
    M = int(off[-1])
    cap = (len(a[0]) if row_token is None else len(row_token)) if cap is None else cap
    y = torch.full((cap, N), -7.0, dtype=dt, device="cuda")
    got = nv.moe_fwd_grouped_gemm_mxfp4(to_dev(a[0]), to_dev(a[1]), to_dev(b[0]), to_dev(b[1]), to_dev(off),
                                        row_token=None if row_token is None else to_dev(row_token), y=y)
    got = got.double().cpu().numpy()
    ref, mag = M4.fwd_grouped(a, b, off, N, row_token)
    bound = (K / 32 + 1) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0.0)
    d = np.abs(got[:M] - ref)
    assert (d <= bound).all(), f"worst {np.max(d / np.maximum(bound, 1e-300)):.3f} of the bound"
    assert (got[M:] == -7.0).all(), "rows behind the last group"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 128), ([0, 3, 0, 1, 0], 128, 256), ([31, 32, 33, 0], 384, 384), ([64, 130, 7], 256, 640),
    ([300, 0, 257, 256, 255, 1], 256, 256), ([700, 20], 640, 1152), ([513], 1280, 128), ([0, 0], 128, 128),
    ([16, 17, 2, 9, 40, 0, 15, 1, 3], 512, 2048),
])
def test_product(nv, counts, N, K, gather, dtype):
    rng = np.random.default_rng(N + K + len(counts))
    G, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    T = max(1, M // 2 + 3) if gather else M + 5
    a = M4.quantize(rng.normal(size=(T, K)).astype(np.float32))
    b = M4.quantize((rng.normal(size=(G * N, K)) * 0.02).astype(np.float32))
    tok = None
    if gather:
        tok = np.concatenate([rng.integers(0, T, M), [-1, T, 1 << 30]]).astype(np.int32)
    _check_product(nv, a, b, off, N, K, dtype, tok)


@pytest.mark.parametrize("kind", ["wide", "ends", "zero", "alternating"])
def test_product_scales(nv, kind):
    """Scales far apart within a row, at the ends of their range, zero blocks, and sums that cancel."""
    rng = np.random.default_rng(9)
    G, N, K = 3, 256, 512
    off = np.array([0, 40, 41, 300])
    a = [rng.integers(0, 256, (300, K // 2)).astype(np.uint8), rng.integers(120, 134, (300, K // 32)).astype(np.uint8)]
    b = [rng.integers(0, 256, (G * N, K // 2)).astype(np.uint8), rng.integers(120, 134, (G * N, K // 32)).astype(np.uint8)]
    if kind == "wide":
        a[1] = rng.integers(90, 160, a[1].shape).astype(np.uint8)
    elif kind == "ends":
        a[1][:] = np.where(rng.random(a[1].shape) < 0.5, 1, 240)
        b[1][:] = 127
    elif kind == "zero":
        a[0][::2], b[0][::3], a[1][::2], b[1][::3] = 0, 0, 0, 0
    else:
        a[0][:, 1::2] = a[0][:, ::2] ^ 0x88
        b[0][:, 1::2] = b[0][:, ::2]
    _check_product(nv, tuple(a), tuple(b), off, N, K, "float32")


def test_product_views_and_shapes(nv):
    """[G, N, K] weights, a row slice of a larger buffer, offsets of a capacity-sized call."""
    import torch
    rng = np.random.default_rng(11)
    G, N, K, T, k = 4, 256, 256, 500, 2
    ids = gen.route_uniform(3, T, 16, k)
    a = M4.quantize(rng.normal(size=(T + 8, K)).astype(np.float32))
    b = M4.quantize((rng.normal(size=(G * N, K)) * 0.02).astype(np.float32))
    o = nv.moe_group(to_dev(ids), 4, G)
    ac, as_ = to_dev(a[0])[8:], to_dev(a[1])[8:]
    y = nv.moe_fwd_grouped_gemm_mxfp4(ac, as_, to_dev(b[0]).view(G, N, K // 2), to_dev(b[1]).view(G, N, K // 32),
                                      o["offsets"], row_token=o["row_token"], out_dtype=torch.bfloat16)
    off, _, tok, _ = PM.permute(ids, 4, G)
    ref, mag = M4.fwd_grouped((a[0][8:], a[1][8:]), b, off, N, tok)
    assert y.shape == (T * k, N)
    d = np.abs(y[:off[-1]].double().cpu().numpy() - ref)
    assert (d <= 9 * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("cols", [128, 384])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 5, 0, 32, 33], [128, 1, 300], [0, 0]])
def test_requant_rows(nv, counts, cols, gather):
    import torch
    rng = np.random.default_rng(cols + len(counts))
    G, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    pad = MX.padded_offsets_from_offsets(off)
    P = int(pad[-1]) + 64
    T = M // 2 + 2 if gather else M + 3
    q = M4.quantize(_rows(cols + M, T, cols, "f32"))
    tok = np.concatenate([rng.integers(0, T, M), [-1, 5]]).astype(np.int32) if gather else None
    out = torch.full((cols, P), 0x55, dtype=torch.uint8, device="cuda")
    e8 = torch.full((cols, P // 32), 0x55, dtype=torch.uint8, device="cuda")
    nv.mxfp8_requant_sr_mxfp4(to_dev(q[0]), to_dev(q[1]), to_dev(off), to_dev(pad), P, 0x5EED0001 << 8, 4,
                              row_token=None if tok is None else to_dev(tok), out=out, out_e8=e8)
    r4, r8 = M4.requant_sr(*q, off, pad, P, 0x5EED0001 << 8, 4, tok)
    n = int(pad[-1])
    assert np.array_equal(from_dev(e8)[:, :n // 32], r8[:, :n // 32])
    assert np.array_equal(from_dev(out)[:, :n], r4[:, :n])
    assert (from_dev(out)[:, n:] == 0x55).all() and (from_dev(e8)[:, n // 32:] == 0x55).all()


def test_requant_rows_outside_the_source_are_zero(nv):
    q = M4.quantize(_rows(1, 6, 128, "f32"))
    tok = np.array([0, -1, 6, 1 << 30, 5], np.int32)
    off, pad = np.array([0, 5]), np.array([0, 32])
    got, e8 = nv.mxfp8_requant_sr_mxfp4(to_dev(q[0]), to_dev(q[1]), to_dev(off), to_dev(pad), 32, 1, 0,
                                        row_token=to_dev(tok))
    v = MX.dequantize(from_dev(got), from_dev(e8))
    assert (v[:, 1:4] == 0).all() and (v[:, [0, 4]] != 0).any()


@pytest.mark.parametrize("G,N,K", [(1, 32, 128), (3, 96, 256), (4, 256, 128)])
def test_requant_weights(nv, G, N, K):
    q = M4.quantize(_rows(G * N, G * N, K, "f32"))
    off = np.arange(G + 1) * N
    got, e8 = nv.mxfp8_requant_sr_mxfp4(to_dev(q[0]), to_dev(q[1]), to_dev(off), to_dev(off), G * N, 77, 1,
                                        rows_per_group=N)
    from helpers import w8_blocked
    r4, r8 = M4.requant_sr(*q, off, off, G * N, 77, 1)
    assert np.array_equal(from_dev(got), w8_blocked(r4, G)) and np.array_equal(from_dev(e8), w8_blocked(r8, G))


def test_requant_every_scale(nv):
    """All scale bytes of finite float32 values, the smallest (subnormal values) among them."""
    codes = np.tile((np.arange(16) | (np.arange(16)[::-1] << 4)).astype(np.uint8), (252, 4))
    scales = np.tile(np.arange(252, dtype=np.uint8)[:, None], (1, 4))
    scales[0] = [0, 1, 2, 3]
    off, pad = np.array([0, 252]), np.array([0, 256])
    # neighbours of 32 rows are 32 binades apart: many elements fall below the block's grid
    got, e8 = nv.mxfp8_requant_sr_mxfp4(to_dev(codes), to_dev(scales), to_dev(off), to_dev(pad), 256, 5, 2)
    r4, r8 = M4.requant_sr(codes, scales, off, pad, 256, 5, 2)
    assert np.array_equal(from_dev(e8), r8)
    assert np.array_equal(from_dev(got), r4)


def test_step(nv):
    """The layer's step in MXFP4, each call checked on the GPU's own inputs to it."""
    import torch
    from precision_moe_numerics_nvfp4_amd.layer import MXFP4LayerStep
    T, K, N, E, k, n, e0 = 300, 256, 256, 4, 2, 12, 4
    w = gen.moe_case(31, T, K, N, E, k, n_experts=n, e0=e0)
    S = MXFP4LayerStep(T, K, N, E, k, e0=e0)
    S.dx.fill_(-7)
    S.step(to_dev(w["x"]), to_dev(w["w"]), to_dev(w["topk"]), to_dev(w["dy"]))
    torch.cuda.synchronize()
    xq, wq = M4.quantize(w["x"]), M4.quantize(w["w"])
    for got, ref in zip(S.xq + S.wq, xq + wq):
        assert np.array_equal(from_dev(got), ref)
    off, pad, tok, _ = PM.permute(w["topk"], e0, E)
    M = int(off[-1])
    ref, mag = M4.fwd_grouped(xq, wq, off, N, tok)
    assert (np.abs(from_dev(S.y)[:M] - ref) <= (K / 32 + 1) * 2.0 ** -23 * mag).all()
    x4, x8 = M4.requant_sr(*xq, off, pad, S.P, S.seed, 0, tok)
    p = int(pad[-1])
    assert np.array_equal(from_dev(S.xT[0])[:, :p], x4[:, :p])
    from helpers import w8_blocked
    w_off = np.arange(E + 1) * N
    w4, w8 = M4.requant_sr(*wq, w_off, w_off, E * N, S.seed, 1)
    assert np.array_equal(from_dev(S.wT[0]), w8_blocked(w4, E)) and np.array_equal(from_dev(S.wT[1]), w8_blocked(w8, E))
    # gradients: the MXFP8 products of these operands, to their own contract
    d4, d8 = MX.quantize_rowwise(w["dy"][:M])
    dx = GM.dgrad_grouped(d4, d8, w4, w8, off, N, "fp64")
    t4, t8 = MX.quantize_colwise_grouped(w["dy"], off, pad, S.P)
    dw = GM.wgrad_grouped(t4, t8, x4, x8, pad, "fp64")
    for g in range(E):
        s = slice(off[g], off[g + 1])
        assert np.abs(from_dev(S.dx)[s] - dx[s]).max() <= 1e-3 * np.abs(dx[s]).max()
        assert np.abs(from_dev(S.dw)[g] - dw[g]).max() <= 1e-3 * np.abs(dw[g]).max()


def test_step_graph(nv):
    """Captured once, replayed with eager steps on other inputs in between."""
    import torch
    from precision_moe_numerics_nvfp4_amd.layer import MXFP4LayerStep
    T, K, N, E, k = 600, 256, 512, 4, 2
    cases = []
    for s in (51, 52):
        w = gen.moe_case(s, T, K, N, E, k)
        cases.append([to_dev(w[i]) for i in ("x", "w", "topk", "dy")])
    S = MXFP4LayerStep(T, K, N, E, k, out_dtype=torch.bfloat16)
    outs = lambda: [S.y, S.dx, S.dw, *S.xT, *S.wT, S.perm["offsets"]]
    refs = []
    for c in cases:
        S.step(*c)
        torch.cuda.synchronize()
        refs.append([t.clone() for t in outs()])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.step(*cases[0])
    for _ in range(3):
        S.step(*cases[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[1], outs()))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[0], outs()))


def test_refusals(nv):
    import torch
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")
    off = torch.tensor([0, 4], device="cuda")
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(z(4, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(z(4, 64, dt=torch.float32).t())
    with pytest.raises(nv.Nvfp4moeError):
        nv.mxfp4_quantize(z(4, 48, dt=torch.float32))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(z(4, 64, dt=torch.float32), codes=z(4, 64))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(z(4, 64, dt=torch.float32), offsets=off.cpu())
    with pytest.raises(ValueError):
        nv.mxfp4_dequantize(z(4, 32), z(4, 3))
    with pytest.raises(ValueError):
        nv.mxfp4_dequantize(z(4, 32), z(4, 2), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        nv.mxfp8_dequantize(z(4, 64), z(4, 3))
    q = lambda r, c: (z(r, c // 2), z(r, c // 32))
    f = nv.moe_fwd_grouped_gemm_mxfp4
    with pytest.raises(ValueError):
        f(*q(4, 128), *q(128, 256), off)
    with pytest.raises(ValueError):
        f(*q(4, 128), *q(129, 128), torch.tensor([0, 2, 4], device="cuda"))
    with pytest.raises(ValueError):
        f(*q(4, 128), *q(128, 128), off, row_token=z(4, dt=torch.int64))
    with pytest.raises(ValueError):
        f(*q(4, 128), *q(128, 128), off, y=z(5, 128, dt=torch.float32))
    with pytest.raises(nv.Nvfp4moeError):
        f(*q(4, 128), *q(64, 128), off)
    r = nv.mxfp8_requant_sr_mxfp4
    with pytest.raises(ValueError):
        r(*q(64, 128), off, off, 64, 1, 0, rows_per_group=32)
    with pytest.raises(ValueError):
        r(*q(4, 128), off, off[:1], 64, 1, 0)
    with pytest.raises(nv.Nvfp4moeError):
        r(*q(4, 128), off, off, 33, 1, 0)
    with pytest.raises(ValueError):
        r(*q(32, 128), off, off, 32, 1, 0, rows_per_group=32, row_token=z(4, dt=torch.int32))
    with pytest.raises(nv.Nvfp4moeError):
        nv.moe_group(z(4, 2, dt=torch.int32), 0, 1025)
    with pytest.raises(ValueError):
        nv.moe_group(z(4, 2, dt=torch.int32), 1 << 33, 8)


def test_product_gathers_past_32_bits(nv):
    """Activations of more than 2 GiB: rows at both ends of them."""
    import torch
    T, K, N, G = 1050000, 4096, 128, 2
    codes = torch.zeros(T, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, K // 32), 127, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 31
    rng = np.random.default_rng(17)
    tok = np.array([0, T - 1, 1048577, 5, T - 2, 1048575], np.int32)
    a = M4.quantize(rng.normal(size=(6, K)).astype(np.float32))
    codes[to_dev(tok.astype(np.int64))], scales[to_dev(tok.astype(np.int64))] = to_dev(a[0]), to_dev(a[1])
    b = M4.quantize((rng.normal(size=(G * N, K)) * 0.02).astype(np.float32))
    off = np.array([0, 2, 6])
    y = nv.moe_fwd_grouped_gemm_mxfp4(codes, scales, to_dev(b[0]), to_dev(b[1]), to_dev(off), row_token=to_dev(tok))
    ref, mag = M4.fwd_grouped(a, b, off, N)
    assert (np.abs(from_dev(y) - ref) <= (K / 32 + 1) * 2.0 ** -23 * mag).all()
    # in place, the tile's own rows are addressed: the last ones lie past 2 GiB too
    off = np.array([0, 1048570, T])
    y = nv.moe_fwd_grouped_gemm_mxfp4(codes, scales, to_dev(b[0]), to_dev(b[1]), to_dev(off), out_dtype=torch.bfloat16)
    for r, i in ((T - 1, 1), (1048577, 2), (5, 3)):
        ref, mag = M4.fwd_grouped((a[0][i:i + 1], a[1][i:i + 1]), tuple(v[(r >= 1048570) * N:][:N] for v in b), [0, 1], N)
        d = np.abs(y[r].double().cpu().numpy() - ref[0])
        assert (d <= (K / 32 + 1) * 2.0 ** -23 * mag[0] + 2.0 ** -8 * np.abs(ref[0])).all()
