"""The probability sums of the routing statistics: how their error goes with
the rows (it must not), for every form that takes them.

u = 2^-24. A row's probability is within rel u of its value, rel as derived in
test_gpu_route (6 D + E + 16; for equal logits the exponentials are 1 and their
sum E exactly, so it is a reciprocal's 2). At most 16 of them are added in 32
bits (16 u, and 4 u for the joins of a matrix accumulator's lanes), all above
that in 64; a workgroup's sum and the result are each rounded once: 22 u in all,
whatever the rows.
"""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev
from oracle import route as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUMS = 22 * U


@pytest.fixture(scope="module")
def nv():
    ensure_built()
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_moe_numerics_nvfp4_amd as nv
    return nv


@pytest.mark.parametrize("T,E,k,score", [
    ((1 << 22) + 7, 20, 17, "softmax"),       # a wavefront per row, 512 rows each
    (1 << 20, 200, 2, "sigmoid"),
    ((1 << 22) + 5, 100, 2, "softmax"),       # 16 lanes per row, 128 rows each
    ((1 << 24) + 9, 12, 2, "softmax"),        # a thread per row, 128 rows each
    ((1 << 24) + 9, 7, 1, "sigmoid"),
    (140000, 1000, 16, "softmax"),            # the most experts a lane, 18 rows each
    (140000, 500, 5, "sigmoid"),
])
def test_equal_rows_by_the_million(nv, T, E, k, score):
    import torch
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    o = nv.moe_route(x, k, score=score, stats=True)
    assert from_dev(o["counts"]).tolist() == [T] * k + [0] * (E - k) + [T]
    got = from_dev(o["prob_sum"]).astype(np.float64)
    # the sigmoid of 0 is 1/2 within 6 u, like every other of the row
    rel = (2 if score == "softmax" else 2 + 2 * 6) * U
    worst = np.abs(got / (T / E) - 1).max()
    assert worst <= rel + SUMS, f"{worst / U:.1f} u"
    loss = from_dev(nv.moe_balance_loss(o["counts"], o["prob_sum"], k, 0.25))[0]
    assert abs(loss - 0.25) <= 0.25 * (rel + SUMS + 2 * U)


FORMS = [
    # T, E, k, score, biased: one workgroup, a part of the device, all of it; each form
    (16, 384, 8, "softmax", False), (900, 8, 2, "sigmoid", True), (64, 50, 3, "softmax", False),
    (3000, 40, 4, "softmax", False), (5000, 384, 8, "sigmoid", True), (70000, 20, 17, "softmax", False),
    (200000, 100, 3, "sigmoid", False), (300000, 6, 2, "softmax", False), (250000, 30, 4, "softmax", False),
    (140000, 60, 5, "softmax", False), (132000, 520, 4, "sigmoid", True), (600000, 66, 3, "softmax", False), (50000, 8, 2, "sigmoid", True), (20000, 600, 9, "softmax", False),
]


@pytest.mark.parametrize("T,E,k,score,biased", FORMS)
def test_sums_within_their_depth(nv, T, E, k, score, biased):
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, E)).astype(np.float32)
    bias = (0.2 * rng.normal(size=E)).astype(np.float32) if biased else None
    mask = rng.random(T) < 0.9
    o = nv.moe_route(to_dev(x), k, score=score, bias=None if bias is None else to_dev(bias),
                     token_mask=to_dev(mask), stats=True)
    want = (R.probabilities(R._vals(x), score) * mask[:, None]).sum(axis=0)
    D = np.abs(x).max() if score == "sigmoid" else (x.max(axis=1) - x.min(axis=1)).max()
    got = from_dev(o["prob_sum"])
    assert from_dev(o["counts"])[E] == mask.sum()
    bad = np.abs(got - want) / want
    assert bad.max() <= (6 * D + E + 16) * U + SUMS, f"{bad.max() / U:.1f} u"
