"""The MXFP4 product reads only the rows that its map names: what else lies in
the buffers (never written, or bytes that stand for NaN) changes no result.

The contraction lengths leave the last piece of a row half empty, where the
bytes that follow a row's scales are a neighbour's."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import mxfp4 as M4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


def _fill(q, rows):
    for part in q:
        part[rows] = 0xFF


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [128, 384, 640, 896])
@pytest.mark.parametrize("counts,N", [([1], 128), ([0, 40, 0, 100, 0], 384), ([300, 0, 150, 256, 0, 200], 256)])
def test_rows_that_nothing_reads(nv, counts, N, K, gather, dtype):
    import torch
    rng = np.random.default_rng(K + N)
    G, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    T = 2 * M + 1 if gather else M + 3
    a = M4.quantize(rng.normal(size=(T, K)).astype(np.float32))
    b = M4.quantize((rng.normal(size=(G * N, K)) * 0.02).astype(np.float32))
    tok = None
    if gather:                                           # even rows only, the last row among them
        tok = (2 * rng.permutation(M + 1)[:M]).astype(np.int32)
        tok[0] = 2 * M
        _fill(a, np.setdiff1d(np.arange(T), tok))
    else:
        _fill(a, slice(M, None))
    for g in np.nonzero(np.array(counts) == 0)[0]:       # weights that no row meets
        _fill(b, slice(g * N, (g + 1) * N))
    y = nv.moe_fwd_grouped_gemm_mxfp4(*map(to_dev, a), *map(to_dev, b), to_dev(off),
                                      row_token=None if tok is None else to_dev(tok), out_dtype=getattr(torch, dtype))
    ref, mag = M4.fwd_grouped(a, b, off, N, tok)
    # K / 32 additions of exact block sums, a unit of 2^-23 of the magnitude each; half a bfloat16 step where stored so
    bound = (K / 32 + 1) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0.0)
    got = y[:M].double().cpu().numpy()
    assert np.isfinite(got).all(), f"{(~np.isfinite(got)).any(axis=1).sum()} of {M} rows are not finite"
    assert (np.abs(got - ref) <= bound).all()
