"""ra_tree_commit for requests of which a drafted token has no slot: skipped as a whole, wherever the token is, so that the
dummy slot reaches neither the table nor the free list."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R
from test_gpu_commit_paths import Trees, host, i32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("page", [-3, 1 << 31, 0])   # (as 32-bit words: negative, negative, the dummy slot's own page)
@pytest.mark.parametrize("nth", [0, 1, 3, 6])        # the page of the list's end that is wrong
def test_a_wrong_page_in_the_middle_of_a_tree(page, nth):
    B, T = 3, 5
    prefix, rows = [4, 0, 9], [2, 0, 1]
    pages = np.arange(1, B * T + 4)
    pages[-1 - (T + nth if nth < T else nth - T)] = np.int64(page).astype(np.int32)
    struck = 1 if nth < T else 0
    table = i32(np.arange(3 * 40).reshape(3, 40) + 500)
    before = host(table)
    free, count = i32(pages), i32([len(pages)])
    loc, pos = (torch.full((B * T,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    qo, ends, seq = i32(np.zeros(B + 1)), i32(np.zeros(B)), i32(prefix)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_step_slots(table, i32(rows), seq, i32([T] * B), free, count, loc, pos, qo, ends, device_error=err)
    assert int(err) == (ra.DEVERR_SLOT if page else 0)
    got = host(loc).reshape(B, T)
    assert (got == 0).sum() == 1 and got[struck, nth if nth < T else nth - T] == 0
    err.zero_()
    left, mid = int(count), host(free)
    path = np.array([[0, 2, 3, -1, -1]] * B)
    want = R.commit(host(table), np.delete(rows, struck), np.delete(prefix, struck), [T] * (B - 1),
                    np.delete(host(qo)[:-1], struck), host(loc), np.delete(path, struck, 0), [3] * (B - 1), mid, left)
    ra.ra_tree_commit(table, i32(rows), seq, i32([T] * B), qo, loc, i32(path), i32([3] * B), seq, free, count,
                      device_error=err)
    assert int(err) == ra.DEVERR_SLOT
    assert np.array_equal(host(table), want[0]) and np.array_equal(host(free), want[1]) and int(count) == want[2]
    assert 0 not in host(free)[:int(count)]
    assert host(seq).tolist() == [n + (0 if b == struck else 3) for b, n in enumerate(prefix)]
    assert np.array_equal(host(table)[rows[struck], :prefix[struck]], before[rows[struck], :prefix[struck]])


@pytest.mark.parametrize("batch,longest", [(40, 64), (700, 30)])
def test_wrong_slots_and_wrong_paths_among_many(batch, longest):
    rng = np.random.default_rng(batch)
    t = Trees(rng, rng.integers(2, longest + 1, batch), longest, 3)
    pick = rng.permutation(batch)
    for b in pick[:batch // 8]:
        t.loc[t.qo[b] + rng.integers(0, t.drafts[b])] = -rng.integers(0, 5)
    for b in pick[batch // 8 - 3:batch // 4]:                   # (three of them with wrong paths as well)
        t.path[b, t.accepted[b] - 1] = t.drafts[b] + 7
    t.check(sorted(pick[:batch // 4].tolist()), ra.DEVERR_SLOT | ra.DEVERR_LENGTH)


def test_the_last_slot_of_the_longest_tree():
    t = Trees(np.random.default_rng(2), [1024, 9], 1024)
    t.loc[1023] = 0
    t.check([0], ra.DEVERR_SLOT)
