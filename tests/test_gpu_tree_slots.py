"""ra_tree_attention with slot ids outside the pool, of prefix and of drafted tokens: flagged, and read as slot 0."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
from test_gpu_tree import BF, Case, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix,draft,n,hq,hkv,d", [
    (50, 7, 3, 8, 2, 64), (500, 8, 2, 32, 8, 128), (300, 6, 70, 32, 8, 128),        # narrow: small calls, the plan's
    (400, 16, 60, 32, 8, 128), (400, 40, 5, 32, 8, 128), (130, 70, 3, 64, 8, 128),  # wide: one query tile, two and more
])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_a_slot_outside_the_pool_is_read_as_slot_0(prefix, draft, n, hq, hkv, d, bad):
    rng = np.random.default_rng(prefix + draft)
    c = Case(rng, [prefix + b % 3 for b in range(n)], [draft] * n, hq, hkv, d, "chain", gap=1)
    c.k[0] = torch.randn(hkv, d, device=c.k.device).to(BF)
    c.v[0] = 3.0
    table = c.table.copy()
    b = n - 1
    for j in (3, int(c.P[b]) - 1, int(c.P[b]) + 1, int(c.P[b]) + draft - 1):
        table[c.rpi[b], j] = bad
        c.table[c.rpi[b], j] = 0
    o = c.run(table=i32(table))
    assert int(c.err.item()) == ra.DEVERR_SLOT
    c.check(o)
