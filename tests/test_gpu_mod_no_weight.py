"""Rows that see keys, but none with a score above minus infinity: 0, whether their keys are one piece or several, beside
requests that they leave alone."""
import numpy as np
import pytest
import torch

import test_gpu_attention_mod as A

pytestmark = pytest.mark.gpu


def strike(c, b):
    """All keys of request b at minus infinity."""
    c.q = (c.q.abs() + 0.125).to(A.BF)
    n = int(c.P[b] + c.E[b])
    c.k[torch.from_numpy(c.table[c.rpi[b], :n]).long().to(A.DEV)] = -float("inf")


def check(c, o, b):
    assert int(c.err) == 0
    rows = slice(int(c.qo[b]), int(c.qo[b + 1]))
    assert (o[rows] == 0).all(), o[rows].flatten()[:4]
    o[rows] = 7.0
    c.check(o, [i for i in range(c.B) if i != b])


# contexts, heads; the struck request is the first: small calls of one and two requests a lane, calls with a plan of their own
# and few or many rows to merge, a request that is one piece
DECODE = [([2000], 8, 8), ([1500, 30, 900], 8, 2), ([900] + [40] * 39, 8, 2), ([9000] + [70] * 99, 8, 4),
          ([5000] + [64] * 79, 64, 8), ([20, 3000], 8, 2)]


@pytest.mark.parametrize("lens,hq,hkv", DECODE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(slopes=True), dict(window=700)])
def test_decode(lens, hq, hkv, d, kw):
    c = A.Case(np.random.default_rng(len(lens)), np.array(lens) - 1, [1] * len(lens), hq, hkv, d, **kw)
    strike(c, 0)
    check(c, c.decode(), 0)


@pytest.mark.parametrize("P,E", [([2000, 0], [40, 60]), ([0, 300], [200, 70]), ([3000], [1])])
@pytest.mark.parametrize("kw", [dict(), dict(slopes=True), dict(window=150)])
def test_extend(P, E, kw):
    c = A.Case(np.random.default_rng(len(P)), P, E, 8, 2, 64, **kw)
    strike(c, 0)
    check(c, c.extend(), 0)
