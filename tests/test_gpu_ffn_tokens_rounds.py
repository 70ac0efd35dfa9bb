"""The few-token layer where a workgroup has several jobs one after another.

A workgroup that goes on to its next job reuses its columns, scales and joined
sums, and loads for a list of another length. Values are whole numbers times
powers of two whose sums stay below 2^24 of their unit (checked), so every order
of additions is exact and the results have to be the definition's bits. Each
weight row and token is different: anything stale shows.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import formats as F
from oracle import nvfp4 as Q
from workloads import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


def _weight(rng, fmt, experts, rows, cols, share=1.0):
    """Any codes in a share of the places, zeros in the others; scales of 1 or 2."""
    codes = rng.integers(0, 256, (experts * rows, cols // 2), dtype=np.uint8)
    if share < 1.0:
        codes[rng.random(codes.shape, dtype=np.float32) >= share] = 0
    s = rng.integers(0, 2, (experts * rows, cols // (32 if fmt == "mxfp4" else 16)), dtype=np.int8)
    if fmt == "mxfp4":
        return codes, (s + 127).astype(np.uint8)
    return codes, (0x38 + 8 * s).astype(np.uint8), np.exp2(rng.integers(0, 2, experts)).astype(np.float32)


PAIR = F.e2m1_decode(Q.unpack_codes(np.arange(256, dtype=np.uint8)[:, None])).astype(np.float32)


def _values(w, e, rows):
    """float32 values (exact) of expert e's rows."""
    s = slice(e * rows, (e + 1) * rows)
    scale = np.exp2(w[1][s].astype(np.float32) - 127) if len(w) == 2 else F.e4m3_decode(w[1][s]).astype(np.float32)
    v = PAIR[w[0][s]].reshape(rows, scale.shape[1], -1) * scale[:, :, None]
    return v.reshape(rows, -1) * (1 if len(w) == 2 else w[2][e])


# Workgroups with several jobs: of the first product where F is the larger, of the second where K is. T * k more than
# seven times the experts makes lists of 16, else they are of 8.
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,k,E,K,Fw,gated", [
    (40, 4, 24, 128, 8192, False), (64, 4, 24, 128, 8192, False), (64, 4, 16, 640, 8192, False),
    (28, 4, 16, 640, 4096, True), (64, 8, 16, 256, 4096, True), (9, 4, 24, 128, 16384, False),
    (40, 4, 24, 8192, 128, False), (64, 4, 24, 8192, 128, False), (64, 4, 16, 8192, 640, False),
    (28, 4, 16, 8192, 384, True), (9, 4, 24, 16384, 128, False),
])
def test_several_jobs_a_workgroup(nv, T, k, E, K, Fw, gated, fmt):
    import torch
    rng = np.random.default_rng(T * k + K)
    # popularity falls with the expert's number: neighbouring lists differ in length, some experts have several
    p = 1.0 / (3 + np.arange(E))
    ids = np.sort(np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]), axis=1)
    lg = np.full((T, E), -20.0, np.float32)
    np.put_along_axis(lg, ids, np.float32(4.0), axis=1)
    x = (rng.choice([-1, 1], (T, K)) * (rng.random((T, K)) < 8 / K)).astype(np.float32)
    m = 2 if gated else 1
    w1, w2 = _weight(rng, fmt, E, m * Fw, K), _weight(rng, fmt, E, K, Fw, 8 / Fw)
    up = lambda w: tuple(to_dev(a) for a in w)
    o = nv.moe_ffn_tokens(to_dev(gen.to_bf16_bits(x)), to_dev(lg), k, up(w1), up(w2), act="none",
                          gated=gated, out_dtype=torch.float32)
    assert np.array_equal(from_dev(o["topk_ids"]), ids)
    assert (from_dev(o["gate"]) == 1.0 / k).all()          # k equal logits, k a power of two
    want, most = np.zeros((2, T, K), np.float32)          # sums of exact terms: float32 holds them
    for e in range(E):
        t = np.nonzero((ids == e).any(axis=1))[0]
        if not t.size:
            continue
        a, b = _values(w1, e, m * Fw), _values(w2, e, K)
        v = x[t] @ a.T
        h = v[:, :Fw] * v[:, Fw:] if gated else v
        # values are whole multiples of 1/2, of 1/4 where two are multiplied
        assert (np.abs(x[t]) @ np.abs(a).T).max() < 2.0 ** 23 and np.abs(h).max() < 2.0 ** 22
        want[t] += h @ b.T / k
        most[t] += np.abs(h) @ np.abs(b).T / k
    assert most.max() < 2.0 ** 24 * 2.0 ** -(m + 1) / k
    assert np.array_equal(from_dev(o["out"]), want)
