"""Pins of the MXFP4 oracle: exponent and rounding by brute force, exact round
trips, the product by exact rational sums, the re-quantization against the
MXFP8 oracle, the few-token layer by plain loops (CPU only)."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import formats as F
from oracle import mxfp4 as M4
from oracle import mxfp8 as MX
from oracle import nvfp4 as Q
from oracle import route as R

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_exponent_at_and_next_to_every_boundary():
    for e in range(-127, 125):
        top = np.float32(6.0 * 2.0 ** e)
        for v, want in ((top, e), (np.nextafter(top, np.float32(np.inf), dtype=np.float32), e + 1)):
            if not np.isfinite(v):
                continue
            x = np.zeros((1, 32), np.float32)
            x[0, 7] = -v
            assert M4.block_exponents(x)[0, 0] == want, (e, v)
    assert M4.block_exponents(np.zeros((1, 32), np.float32))[0, 0] == -127
    assert M4.block_exponents(np.full((1, 32), 2.0 ** -149, np.float32))[0, 0] == -127


def test_codes_are_the_nearest():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(40, 64)) * np.exp2(rng.integers(-30, 30, (40, 64)))).astype(np.float32)
    codes, scales = M4.quantize(x)
    c = Q.unpack_codes(codes)
    for (r, j), v in np.ndenumerate(x.astype(np.float64)):
        y = v / 2.0 ** (int(scales[r, j // 32]) - 127)
        d = [abs(abs(y) - g) for g in GRID]
        best = [i for i, q in enumerate(d) if q == min(d)]
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert int(c[r, j]) == want | (8 if v < 0 else 0)


def test_every_code_and_scale_comes_back():
    codes = np.tile((np.arange(16) | (np.arange(16)[::-1] << 4)).astype(np.uint8), (254, 1))
    codes[:, 0] = 7                                       # a 6 in the block keeps its exponent
    scales = np.arange(254, dtype=np.uint8)[:, None]
    v = M4.dequantize(codes, scales)
    keep = np.abs(v).max(axis=1) <= np.finfo(np.float32).max
    got, gs = M4.quantize(v[keep].astype(np.float32))
    assert np.array_equal(gs, scales[keep]) and np.array_equal(got, codes[keep])


def test_product_is_the_exact_sum():
    rng = np.random.default_rng(1)
    a = M4.quantize(rng.normal(size=(5, 64)).astype(np.float32))
    b = M4.quantize((rng.normal(size=(2 * 3, 64)) * 0.02).astype(np.float32))
    tok = np.array([4, 0, 0, 2, 3])
    y, _ = M4.fwd_grouped(a, b, [0, 2, 5], 3, tok)
    A, B = M4.dequantize(*a), M4.dequantize(*b)
    for r in range(5):
        for n in range(3):
            g = 0 if r < 2 else 1
            want = sum(Fraction(A[tok[r], i]) * Fraction(B[g * 3 + n, i]) for i in range(64))
            assert Fraction(y[r, n]) == want              # every partial sum fits 53 bits here


def test_requant_equals_mxfp8_of_the_values():
    rng = np.random.default_rng(2)
    q = M4.quantize(rng.normal(size=(40, 128)).astype(np.float32))
    off, pad, P = np.array([0, 7, 7, 40]), np.array([0, 32, 32, 96]), 96
    e4, e8 = M4.requant_sr(*q, off, pad, P, 0x5EED, 3)
    v = MX.dequantize(e4, e8)
    x = M4.dequantize(*q)
    for g in range(3):
        for i, r in enumerate(range(off[g], off[g + 1])):
            got, want = v[:, pad[g] + i], x[r]
            # a neighbour of the value: E4M3 steps are at most 1/8 of it, or 2^-9 of the block's scale
            step = np.maximum(np.abs(want) / 8, np.repeat(0, 128) + 2.0 ** (e8[:, (pad[g] + i) // 32].astype(float) - 136))
            assert (np.abs(got - want) <= step).all()
    assert (v[:, 7:32] == 0).all() and (v[:, 65:] == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("gated,act", [(False, "relu2"), (True, "silu")])
def test_ffn_tokens_by_loops(fmt, gated, act):
    rng = np.random.default_rng(3)
    T, K, Fw, n, E, e0, k = 3, 32, 32, 2, 5, 1, 2
    x = rng.normal(size=(T, K)).astype(np.float32)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    m = 2 if gated else 1
    q = (lambda w, rows: M4.quantize(w)) if fmt == "mxfp4" else (lambda w, rows: Q.quantize(w, rows))
    w1 = q(rng.normal(size=(n * m * Fw, K)).astype(np.float32), m * Fw)
    w2 = q(rng.normal(size=(n * K, Fw)).astype(np.float32), K)
    got = M4.ffn_tokens(x, logits, k, w1, w2, act=act, gated=gated, e0=e0, n_local=n)
    W1, W2 = M4.weight(w1), M4.weight(w2)
    r = R.route(logits, k)
    for t in range(T):
        want = np.zeros(K)
        for j in range(k):
            e = r["topk_ids"][t, j] - e0
            if not 0 <= e < n:
                continue
            h = []
            for f in range(Fw):
                v = sum(float(W1[e * m * Fw + f, i]) * float(x[t, i]) for i in range(K))
                v = v / (1 + math.exp(-v)) if act == "silu" else max(v, 0.0) ** 2
                if gated:
                    v *= sum(float(W1[e * m * Fw + Fw + f, i]) * float(x[t, i]) for i in range(K))
                h.append(v)
            for c in range(K):
                want[c] += r["gate"][t, j] * sum(float(W2[e * K + c, f]) * h[f] for f in range(Fw))
        assert np.allclose(got["out"][t], want, rtol=1e-10, atol=1e-10)
    if fmt == "nvfp4":                                    # the NVFP4 oracle's own values (its outer product rounds)
        assert np.allclose(W1, Q.dequantize(*w1, rows_per_group=m * Fw), rtol=2.0 ** -23)
