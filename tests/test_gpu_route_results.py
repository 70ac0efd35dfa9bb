"""What the routing call hands back, apart from the values."""

import numpy as np
import pytest

from helpers import ensure_built, from_dev, to_dev

pytestmark = pytest.mark.gpu


def test_results_of_a_call_without_statistics():
    """Buffers of an earlier call's statistics are no results of this one."""
    ensure_built()
    import torch
    import precision_moe_numerics_nvfp4_amd as nv
    x = to_dev(np.random.default_rng(0).normal(size=(50, 20)).astype(np.float32))
    o = nv.moe_route(x, 3, stats=True)
    kept = {n: from_dev(t.clone()) for n, t in o.items()}
    p = nv.moe_route(-x, 3, out=o)
    assert set(p) == {"topk_ids", "gate"}
    assert p["topk_ids"] is o["topk_ids"] and p["gate"] is o["gate"]
    assert not np.array_equal(from_dev(p["topk_ids"]), kept["topk_ids"])
    assert all(np.array_equal(from_dev(o[n]), kept[n]) for n in ("counts", "prob_sum"))
    q = nv.moe_route(x, 3, stats=True, out=p)
    assert set(q) == {"topk_ids", "gate", "counts", "prob_sum"} and set(p) == {"topk_ids", "gate"}
    assert all(np.array_equal(from_dev(q[n]), kept[n]) for n in kept)
