"""The few-token expert layer on values whose result is exact.

Weights of zeros and ones pick single inputs, the gates are 1 (one expert a
token, renormalised), so every product, sum and rounding of the definition is
exact in float32 and the kernels have to give the definition's bits.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import formats as F
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


ONE = 2                                                # E2M1 code of 1
assert F.e2m1_decode(np.array([ONE], np.uint8))[0] == 1.0 and F.e4m3_decode(np.array([0x38], np.uint8))[0] == 1.0


def _picking(picks, rows, cols, fmt, experts):
    """The weight of `experts` equal experts whose row r sums the columns picks[r]."""
    codes = np.zeros((rows, cols), np.uint8)
    for r, cs in enumerate(picks):
        codes[r, list(cs)] = ONE
    codes = np.tile(codes[:, ::2] | codes[:, 1::2] << 4, (experts, 1))
    if fmt == "mxfp4":
        return codes, np.full((experts * rows, cols // 32), 127, np.uint8)
    return codes, np.full((experts * rows, cols // 16), 0x38, np.uint8), np.ones(experts, np.float32)


def _run(nv, x, w1, w2, experts, seed=3, **how):
    """out as float32, one expert a token, drawn."""
    import torch
    lg = np.random.default_rng(seed).normal(size=(len(x), experts)).astype(np.float32)
    up = lambda w: tuple(to_dev(v) for v in w)
    bits = gen.to_bf16_bits(x.astype(np.float32))
    assert np.array_equal(F.bf16_bits_to_f32(bits), x.astype(np.float32), equal_nan=True)
    o = nv.moe_ffn_tokens(to_dev(bits), to_dev(lg), 1, up(w1), up(w2), out_dtype=torch.float32, **how)
    assert (from_dev(o["gate"]) == 1.0).all()
    return from_dev(o["out"])


# tokens and experts: the second product's lists of 8, and (more than 7 tokens an expert) of 16
SIZES = [(1, 1), (9, 4), (20, 2), (64, 6)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,E", SIZES)
def test_h_is_a_float32(nv, T, E, gated, fmt):
    """h takes 24 significant bits, and all of them reach the output."""
    Fw, K = 128, 512
    rng = np.random.default_rng(T)
    part = 2 * rng.integers(0, 64, (3, T, Fw)) + 1                   # odd, 7 bits
    part[0] += 128                                                   # the first of 8
    x = np.zeros((T, K))
    x[:, :384] = np.concatenate([part[0] * 65536.0, part[1] * 256.0, part[2]], axis=1)
    x *= rng.choice([-1, 1], (T, 1))
    x[:, 384] = 1.0
    picks = [(j, 128 + j, 256 + j) for j in range(Fw)] + ([(384,)] * Fw if gated else [])
    w1 = _picking(picks, len(picks), K, fmt, E)
    w2 = _picking([(r % Fw,) for r in range(K)], K, Fw, fmt, E)
    got = _run(nv, x, w1, w2, E, act="none", gated=gated)
    h = x[:, :128] + x[:, 128:256] + x[:, 256:384]
    assert (np.abs(h) >= 2.0 ** 23).all() and (h % 2 == 1).all()     # all 24 bits are used
    assert np.array_equal(got, np.tile(h, (1, 4)).astype(np.float32))


@pytest.mark.parametrize("T,E", SIZES)
def test_h_next_to_the_largest_float32(nv, T, E):
    """Values that bfloat16 would round to infinity."""
    x = np.zeros((T, 128))
    x[:, 0], x[:, 1], x[:, 2] = 255 * 2.0 ** 120, 255 * 2.0 ** 112, 255 * 2.0 ** 104
    x[::2] *= -1
    w1 = _picking([(0, 1, 2)] * 128, 128, 128, "mxfp4", E)
    w2 = _picking([(r,) for r in range(128)], 128, 128, "mxfp4", E)
    got = _run(nv, x, w1, w2, E, act="none")
    big = np.finfo(np.float32).max
    want = np.where(np.arange(T)[:, None] % 2 == 0, -big, big) * np.ones((1, 128))
    assert np.array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu2", "silu"])
@pytest.mark.parametrize("T,E", SIZES)
def test_nan_reaches_its_token_and_no_other(nv, T, E, act, gated, fmt):
    """A NaN in x, or in an expert's outer scale, is NaN in the output of the tokens that meet it; the others keep
    their bits."""
    rng = np.random.default_rng(T + E)
    cols = lambda n, rows: [rng.choice(n, 3, replace=False) for _ in range(rows)]
    w1 = _picking(cols(256, 256 if gated else 128), 256 if gated else 128, 256, fmt, E)
    w2 = _picking(cols(128, 256), 256, 128, fmt, E)
    x = rng.integers(-8, 9, (T, 256)).astype(np.float64)
    clean = _run(nv, x, w1, w2, E, act=act, gated=gated)
    assert np.isfinite(clean).all()
    bad = np.arange(T) % 3 == 0
    x[bad, rng.integers(0, 256, bad.sum())] = np.nan
    got = _run(nv, x, w1, w2, E, act=act, gated=gated)
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])
    if fmt == "nvfp4":
        x[bad] = 1.0
        clean = _run(nv, x, w1, w2, E, act=act, gated=gated)
        lg = np.random.default_rng(3).normal(size=(T, E)).astype(np.float32)
        met = lg.argmax(axis=1) == lg[0].argmax()
        for i in (0, 1):
            w = [list(w1), list(w2)]
            w[i][2] = w[i][2].copy()
            w[i][2][lg[0].argmax()] = np.nan
            got = _run(nv, x, *map(tuple, w), E, act=act, gated=gated)
            assert np.isnan(got[met]).all() and np.array_equal(got[~met], clean[~met])


@pytest.mark.parametrize("E", [8, 80])
def test_the_largest_h(nv, E):
    """512 pairs of 2^20 values: the parts of h end past 3 GiB. Lists of 16 and of 8."""
    import torch
    T, k, K, Fw, local = 64, 8, 128, 1 << 20, 7
    rng = np.random.default_rng(E)
    x = rng.choice([-1.0, 1.0], (T, K)) * rng.integers(1, 257, (T, K))
    lg = np.full((T, E), -20.0, np.float32)
    lg[:, :k] = 4.0                                      # slot j is expert j, its gate 1/8; one of them is local
    w1c = np.zeros((Fw, K // 2), np.uint8)
    j = np.arange(Fw)
    col = (j * 37 + j // K) % K                          # h[j] = x[col[j]]
    w1c[j, col // 2] = np.where(col % 2, ONE << 4, ONE)
    w2c = np.zeros((K, Fw // 2), np.uint8)
    pick = np.concatenate([rng.integers(0, Fw, (K, 4)), Fw - 1 - np.arange(K)[:, None], np.arange(K)[:, None]], axis=1)
    for r in range(K):
        for c in set(pick[r].tolist()):
            w2c[r, c // 2] |= ONE << 4 if c % 2 else ONE
    ones = lambda rows, cols: torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    o = nv.moe_ffn_tokens(to_dev(gen.to_bf16_bits(x.astype(np.float32))), to_dev(lg), k, (to_dev(w1c), ones(Fw, K)),
                          (to_dev(w2c), ones(K, Fw)), act="none", e0=local, out_dtype=torch.float32)
    assert (from_dev(o["topk_ids"]) == np.arange(k)).all() and (from_dev(o["gate"]) == 0.125).all()
    want = np.stack([x[:, col[sorted(set(pick[r].tolist()))]].sum(axis=1) for r in range(K)], axis=1) / 8
    assert np.array_equal(from_dev(o["out"]), want.astype(np.float32))
