"""ra_tree_commit with paths that do not ascend within their tree: flagged, the request skipped, and neither the other
requests' entries nor anything around the free list touched."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 1100  # words in front of and behind the list (a tree holds up to 1,024 nodes)


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def host(t):
    return t.cpu().numpy()


class Trees:
    def __init__(self, rng, drafts, widest, held=0):
        B = len(drafts)
        self.B, self.drafts, self.total = B, np.asarray(drafts), int(np.sum(drafts))
        self.prefix = rng.integers(0, 30, B)
        self.qo = np.concatenate([[0], np.cumsum(drafts)])
        self.table = rng.integers(1, 999, (B + 1, 40 + widest)).astype(np.int32)
        self.rpi = rng.permutation(B + 1)[:B]
        self.loc = (rng.permutation(self.total) + 1000).astype(np.int32)
        self.path = np.full((B, widest), -1, np.int32)
        self.accepted = np.zeros(B, np.int64)
        for b, T in enumerate(drafts):
            keep = [0] + [i for i in range(1, T) if rng.random() < 0.4] if T else []
            self.path[b, :len(keep)], self.accepted[b] = keep, len(keep)
        self.held = held  # entries in the list before the call
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(self, wrong, flags=ra.DEVERR_LENGTH):
        """Requests `wrong` are flagged and skipped, the others committed."""
        big = np.full(2 * GUARD + self.held + self.total, -5, np.int32)
        big[GUARD:GUARD + self.held] = 1 + np.arange(self.held)
        words = i32(big)
        free = words[GUARD:GUARD + self.held + self.total]
        table, count = i32(self.table), i32([self.held])
        seq = torch.full((self.B,), -7, dtype=torch.int32, device=DEV)
        self.err.zero_()
        ra.ra_tree_commit(table, i32(self.rpi), i32(self.prefix), i32(self.drafts), i32(self.qo), i32(self.loc),
                          i32(self.path), i32(self.accepted), seq, free, count, device_error=self.err)
        good = [b for b in range(self.B) if b not in wrong]
        ref = R.commit(self.table, self.rpi[good], self.prefix[good], self.drafts[good], self.qo[good], self.loc,
                       self.path[good], self.accepted[good], big[GUARD:GUARD + self.held + self.total], self.held)
        assert int(self.err) == (flags if wrong else 0)
        assert np.array_equal(host(table), ref[0])
        big[GUARD:GUARD + self.held + self.total] = ref[1]
        assert np.array_equal(host(words), big)
        assert int(count) == ref[2]
        lens = self.prefix.copy()
        lens[good] = ref[3]
        assert np.array_equal(host(seq), lens)


BAD = [[0, 0], [0, -1], [-1, -1, -1], [0, -1, -1], [5, 2, 0], [0, 3, 3], [0, 2, 1], [1, 0], [0, 6], [0, 1 << 30], [-9], [6],
       [0, 1, 2, 3, 4, 4], [1, 2, 3, 4, 5, 6]]


@pytest.mark.parametrize("path", BAD)
@pytest.mark.parametrize("held", [0, 5])
@pytest.mark.parametrize("at", [0, 2])
def test_paths_that_do_not_ascend(path, held, at):
    t = Trees(np.random.default_rng(len(path) + held), [6, 5, 6], 6, held)
    t.path[at] = -1
    t.path[at, :len(path)], t.accepted[at] = path, len(path)
    t.check([at])


@pytest.mark.parametrize("batch,longest", [(40, 64), (600, 40), (1500, 9)])
def test_several_of_many_requests(batch, longest):
    """More than one round of 512 requests, and clusters of 1 to 8 CTAs."""
    rng = np.random.default_rng(batch)
    t = Trees(rng, rng.integers(2, longest + 1, batch), longest, 3)
    t.check([])
    wrong = sorted(rng.choice(batch, batch // 5, replace=False).tolist())
    for b in wrong:
        n = int(t.accepted[b])
        kind = rng.integers(0, 3)
        if kind == 0:
            t.path[b, n - 1] = t.drafts[b]                       # behind the tree
        elif kind == 1 and n >= 2:
            t.path[b, n - 1] = t.path[b, n - 2]
        elif n < t.drafts[b]:
            t.accepted[b] = n + 1                                # more than the path holds
        else:
            t.path[b, 0] = -1
    t.check(wrong)


def test_the_longest_paths():
    """Every entry of a path of 1,024 nodes counts, the last of 32 and the first of the next 32 among them."""
    t = Trees(np.random.default_rng(1), [1024, 1000], 1024)
    t.path[0], t.accepted[0] = np.arange(1024), 1024
    t.check([])
    for k in (0, 1, 31, 32, 33, 1022, 1023):
        keep = t.path[0, k]
        t.path[0, k] = keep + 1 if k < 1023 else 1022
        t.check([0])
        t.path[0, k] = keep
