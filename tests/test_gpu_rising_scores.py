"""Scores that climb from chunk to chunk of a key tile, so that the uncapped passes raise a row's reference several times within
a tile, for some rows of a warp and not for others, against 64-bit attention."""
import numpy as np
import pytest
import torch

import test_gpu_attention_mod as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 4000.0])   # 4,000 is far above the scores: the pass for large caps
@pytest.mark.parametrize("step", [50, 90])       # climb per 32 keys (a chunk's sum may hold 2^60, 41.6 of them)
def test_references_raised_within_a_tile(d, cap, step):
    c = A.Case(np.random.default_rng(d + step), [0, 300], [390, 200], 8, 2, d, cap=cap)
    # along the first dimension of K the key's position, in chunks of 32; the rows' first dimension says how fast they climb
    k, q = c.k.float(), c.q.float()
    for b in range(2):
        n = int(c.P[b] + c.E[b])
        slots = torch.from_numpy(c.table[c.rpi[b], :n]).long().to(A.DEV)
        k[slots, :, 0] = (torch.arange(n, device=A.DEV) // 32).float()[:, None]
    rate = torch.tensor([1.0, -1.0, 0.5, 0.0, 1.0, 1.0, 0.9, -0.2], device=A.DEV) * step / c.scale
    q[:, :, 0] = rate
    q[::3, :, 0] *= -1
    c.k, c.q = k.to(A.BF), q.to(A.BF)
    for _ in range(3):
        c.check(c.extend())
    assert int(c.err) == 0
