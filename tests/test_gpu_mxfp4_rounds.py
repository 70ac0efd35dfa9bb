"""The MXFP4 product where a workgroup has several tiles one after another.

Whole tiles behind whole tiles (whose rows are still being written when the next
tile's loads are waited for), cut pieces ahead of whole tiles, groups of every
kind of height, both output types. Scales are 1 and 2 and all sums stay below
2^24 of their unit (checked), so float32 sums are exact in any order: every value
is compared, bit for bit.
"""

import numpy as np
import pytest

from helpers import ensure_built, to_dev
from oracle import formats as F
from oracle import nvfp4 as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


PAIR = F.e2m1_decode(Q.unpack_codes(np.arange(256, dtype=np.uint8)[:, None])).astype(np.float32)


def _tensor(rng, rows, K):
    return rng.integers(0, 256, (rows, K // 2), dtype=np.uint8), rng.integers(127, 129, (rows, K // 32), dtype=np.uint8)


def _values(q):
    v = PAIR[q[0]].reshape(len(q[0]), -1, 32) * np.exp2(q[1].astype(np.float32) - 127)[:, :, None]
    return v.reshape(len(q[0]), -1)


MIXED = [256, 512, 300, 40, 64, 1, 0, 200, 128, 700, 33]        # 14 tiles of 256 rows

# On 256 compute units, an eighth of the tiles to 32 of them: rounds, and what is left over
CASES = [
    (MIXED * 5, 1024, 384),             # 1 round, 3: quarters
    (MIXED * 6, 1024, 128),             # 1 round, 10: halves
    (MIXED * 9, 1024, 256),             # 1 round, 31: whole
    (MIXED * 11, 1024, 128),            # 2 rounds, 13: halves
    (MIXED * 7, 640, 640),              # the last tile of a row has 128 columns
    (MIXED * 8, 640, 256),
    ([256 * 66], 2048, 384),            # 2 rounds of whole tiles, 2: quarters
    ([256] * 100 + [250] * 180, 512, 128),
    ([60] * 300, 512, 256),             # 2 rounds, 11: halves of the columns
    ([60, 64, 5] * 92, 256, 1024),      # 1 round, 2 to 3
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_several_tiles_a_workgroup(nv, case, gather, dtype):
    import torch
    counts, N, K = CASES[case]
    rng = np.random.default_rng(case)
    G, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    T = M // 3 + 7 if gather else M + 5
    a, b = _tensor(rng, T, K), _tensor(rng, G * N, K)
    tok = rng.integers(0, T, M + 3).astype(np.int32) if gather else None
    dt = getattr(torch, dtype)
    y = torch.full((len(tok) if gather else T, N), -7.0, dtype=dt, device="cuda")
    nv.moe_fwd_grouped_gemm_mxfp4(*map(to_dev, a), *map(to_dev, b), to_dev(off),
                                  row_token=to_dev(tok) if gather else None, y=y)
    av, bv = _values(a), _values(b)
    rows = tok[:M] if gather else np.arange(M)
    want = np.empty((M, N), np.float32)
    for g in range(G):
        s = slice(off[g], off[g + 1])
        want[s] = av[rows[s]] @ bv[g * N:(g + 1) * N].T
    # values are multiples of 1/2, products of 1/4; 12 is the largest value
    assert np.abs(av).max() <= 12 and K * 144 < 2 ** 24 // 4
    got = y.cpu()
    want = torch.from_numpy(want).to(dt)
    bad = torch.nonzero((got[:M] != want).any(dim=1)).flatten()
    assert bad.numel() == 0, f"{bad.numel()} of {M} rows, first {bad[:8].tolist()}"
    assert (got[M:] == -7.0).all()
