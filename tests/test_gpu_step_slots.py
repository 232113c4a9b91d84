"""ra_step_slots and ra_tree_commit against their definitions: pages and single slots, empty and padded batches, more
requests than one round of the scan, outputs in place, bad requests, graphs."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def host(t):
    return t.cpu().numpy()


class Step:
    def __init__(self, rng, cur, new, page, pad=0, spare=3):
        self.cur, self.new, self.page = np.asarray(cur), np.asarray(new), page
        B = len(self.cur)
        pages = -(-self.cur // page)
        self.need = -(-(self.cur + self.new) // page) - pages
        ids = rng.permutation(int(pages.sum() + self.need.sum()) + spare) + 1
        self.table = np.full((B + 2, int((self.cur + self.new).max(initial=0)) + 2), -1, np.int32)
        self.rpi = rng.permutation(B + 2)[:B]
        at = 0
        for b in range(B):
            slots = (ids[at:at + pages[b], None] * page + np.arange(page)).ravel()
            self.table[self.rpi[b], :self.cur[b]] = slots[:self.cur[b]]
            at += pages[b]
        self.free = ids[at:].astype(np.int32)
        self.n = int(self.new.sum()) + pad
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **over):
        a = dict(table=i32(self.table), rpi=i32(self.rpi), cur=i32(self.cur), new=i32(self.new), free=i32(self.free),
                 count=i32([len(self.free)]), n=self.n)
        a.update(over)
        B = a["rpi"].shape[0]
        loc, pos = (torch.full((a["n"],), -7, dtype=torch.int32, device=DEV) for _ in range(2))
        qo, seq = torch.full((B + 1,), -7, dtype=torch.int32, device=DEV), torch.full((B,), -7, dtype=torch.int32, device=DEV)
        left = torch.full((1,), -7, dtype=torch.int32, device=DEV)
        ra.ra_step_slots(a["table"], a["rpi"], a["cur"], a["new"], a["free"], a["count"], loc, pos, qo, seq,
                         page_size=self.page, free_count_out=left, device_error=self.err)
        return [host(x) for x in (a["table"], loc, pos, qo, seq)] + [int(left)]

    def ref(self):
        return R.step_slots(self.table, self.rpi, self.cur, self.new, self.free, len(self.free), self.page, self.n)


def same(got, ref):
    for i, (x, y) in enumerate(zip(got, ref)):
        assert np.array_equal(x, y), i


CASES = [([0], [1], 1), ([7], [0], 4), ([5, 0, 16, 31], [1, 1, 1, 1], 16), ([0, 3, 8, 9], [5, 0, 8, 23], 4),
         ([100, 0, 63, 64, 65], [900, 65, 64, 1, 200], 64), ([11] * 40, [1] * 40, 1), ([4000, 1], [5000, 4095], 16),
         ([0, 0, 9], [0, 0, 1], 3), (list(range(700)), [i % 7 for i in range(700)], 5),
         ([i % 50 for i in range(1500)], [1] * 1500, 16)]


@pytest.mark.parametrize("cur,new,page", CASES)
@pytest.mark.parametrize("pad", [0, 70])
def test_step_slots(cur, new, page, pad):
    s = Step(np.random.default_rng(len(cur) + page), cur, new, page, pad)
    same(s.run(), s.ref())
    assert int(s.err) == 0


@pytest.mark.parametrize("batch,longest", [(1, 1), (13, 40), (512, 60), (513, 9), (2000, 40), (5, 20000)])
def test_step_slots_random(batch, longest):
    rng = np.random.default_rng(batch)
    s = Step(rng, rng.integers(0, 300, batch), rng.integers(0, longest + 1, batch), int(rng.choice([1, 16, 24])), 11)
    same(s.run(), s.ref())
    assert int(s.err) == 0


def test_step_slots_in_place_and_chained():
    """Three steps over the same buffers, the lengths and the list's count written in place; then no request."""
    rng = np.random.default_rng(3)
    s = Step(rng, [5, 0, 30], [4, 17, 2], 8, spare=40)
    table, cur, free, count = i32(s.table), i32(s.cur), i32(s.free), i32([len(s.free)])
    ref_table, ref_cur, left = s.table, s.cur, len(s.free)
    wide = torch.full((5, 120), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    ref_table = host(wide)
    loc, pos = (torch.zeros(30, dtype=torch.int32, device=DEV) for _ in range(2))
    qo = torch.zeros(4, dtype=torch.int32, device=DEV)
    for new in ([4, 17, 2], [1, 1, 1], [9, 0, 12]):
        ra.ra_step_slots(wide, i32(s.rpi), cur, i32(new), free, count, loc, pos, qo, cur, page_size=8)
        ref = R.step_slots(ref_table, s.rpi, ref_cur, new, s.free, left, 8, 30)
        same([host(wide), host(loc), host(pos), host(qo), host(cur), int(count)], ref)
        ref_table, ref_cur, left = ref[0], ref[4], ref[5]
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    ra.ra_step_slots(wide, none, none, none, free, count, loc, pos, qo[:1], none)
    assert int(count) == left and int(qo[0]) == 0 and not host(loc).any()


def test_step_slots_flags_bad_requests():
    rng = np.random.default_rng(4)
    s = Step(rng, [5, 6, 7, 8], [3, 2, 4, 1], 4)
    good = s.ref()

    def check(flag, wrong, **over):
        s.err.zero_()
        table, loc, pos, qo, seq, left = s.run(**over)
        assert int(s.err) == flag
        for b in range(4):
            rows, r = slice(qo[b], qo[b + 1]), s.rpi[b]
            if b in wrong:
                assert not loc[rows].any() and np.array_equal(table[r], s.table[r])
            else:
                assert (loc[rows] > 0).all() and seq[b] == s.cur[b] + s.new[b]
        return table, loc, pos, qo, seq, left

    bad = s.rpi.copy()
    bad[1] = 99
    check(ra.DEVERR_TABLE, [1], rpi=i32(bad))
    bad[1] = -1
    check(ra.DEVERR_TABLE, [1], rpi=i32(bad))
    out = check(ra.DEVERR_LENGTH, [2], new=i32([3, 2, 4000, 1]), n=5000)
    assert out[4][2] == 7
    out = check(ra.DEVERR_LENGTH, [0], new=i32([-3, 2, 4, 1]))
    assert out[3].tolist() == [0, 0, 2, 6, 7] and out[4][0] == 5
    out = check(ra.DEVERR_LENGTH, [3], n=9)             # the last request's token has no row
    assert out[3].tolist() == [0, 3, 5, 9, 9] and out[4][3] == 8
    # pages for the first request only: the others that need one are refused
    need = s.need
    first_two = int(need[:2].sum())
    out = check(ra.DEVERR_FULL, [b for b in range(4) if need[b] and need[:b + 1].sum() > first_two],
                count=i32([first_two]), free=i32(s.free))
    assert out[5] == 0
    out = check(ra.DEVERR_LENGTH, [], count=i32([10 ** 6]))   # clamped to the list's size
    assert out[5] == good[5]
    s.err.zero_()
    _, loc, *_ = s.run(free=i32(-s.free))
    assert int(s.err) == ra.DEVERR_SLOT and loc.min() >= 0


def tables(rng, prefix, drafts, gap=0):
    B = len(prefix)
    total = int(np.sum(drafts)) + gap * B
    qo = np.concatenate([[0], np.cumsum(np.asarray(drafts) + gap)])
    table = rng.integers(1, 999, (B + 1, int((np.asarray(prefix) + drafts).max()) + 3)).astype(np.int32)
    loc = (rng.permutation(total + 5)[:total] + 1000).astype(np.int32)
    widest = max(int(np.max(drafts)), 1)
    path = np.full((B, widest), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    for b, T in enumerate(drafts):
        if T == 0:
            continue
        keep = [0] + [i for i in range(1, T) if rng.random() < 0.3]
        accepted[b] = len(keep)
        path[b, :len(keep)] = keep
    free = np.concatenate([rng.integers(1, 99, 4), np.zeros(total + 2)]).astype(np.int32)
    return dict(table=table, rpi=rng.permutation(B + 1)[:B], prefix=np.asarray(prefix), drafts=np.asarray(drafts), qo=qo,
                loc=loc, path=path, accepted=accepted, free=free, count=4)


def run_commit(c, err=None, **over):
    a = {k: i32([v] if k == "count" else v) for k, v in c.items()}
    a.update(over)
    seq = torch.full((len(c["prefix"]),), -7, dtype=torch.int32, device=DEV)
    left = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    ra.ra_tree_commit(a["table"], a["rpi"], a["prefix"], a["drafts"], a["qo"], a["loc"], a["path"], a["accepted"], seq,
                      a["free"], a["count"], free_count_out=left, device_error=err)
    return host(a["table"]), host(a["free"]), int(left), host(seq)


@pytest.mark.parametrize("prefix,drafts,gap", [([0], [1], 0), ([9, 0, 300], [8, 1, 5], 0), ([5, 6], [0, 3], 2),
                                               ([40] * 600, [1 + i % 9 for i in range(600)], 0), ([7, 100], [1024, 700], 0),
                                               ([1] * 224, [32 + i % 33 for i in range(224)], 1)])
def test_tree_commit(prefix, drafts, gap):
    c = tables(np.random.default_rng(len(prefix)), prefix, drafts, gap)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    same(run_commit(c, err), R.commit(**c))
    assert int(err) == 0


def test_tree_commit_flags_bad_requests():
    c = tables(np.random.default_rng(9), [9, 4, 30], [6, 5, 8])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for key, value, flag in (("rpi", -2, ra.DEVERR_TABLE), ("drafts", -1, ra.DEVERR_LENGTH), ("drafts", 9, ra.DEVERR_LENGTH),
                             ("accepted", 6, ra.DEVERR_LENGTH), ("prefix", 10 ** 6, ra.DEVERR_LENGTH),
                             ("qo", 10 ** 6, ra.DEVERR_LENGTH)):
        bad = c[key].copy()
        bad[1] = value
        err.zero_()
        table, free, left, seq = run_commit(c, err, **{key: i32(bad)})
        assert int(err) == flag, key
        rest = {k: (v[[0, 2]] if k in ("rpi", "prefix", "drafts", "path", "accepted") else v) for k, v in c.items()}
        rest["qo"] = c["qo"][[0, 2]]
        ref = R.commit(**rest)
        assert np.array_equal(table, ref[0]) and np.array_equal(free, ref[1]) and left == ref[2], key
    err.zero_()                                    # no room for the last slots
    room = 4 + int((c["drafts"] - c["accepted"]).sum()) - 2
    table, free, left, _ = run_commit(c, err, free=i32(c["free"][:room]))
    ref = R.commit(**c)
    assert int(err) == ra.DEVERR_FULL and left == room and np.array_equal(free, ref[1][:room])
    assert np.array_equal(table, ref[0])
    err.zero_()                                    # a path that descends: flagged, nothing outside the request written
    bad = c["path"].copy()
    bad[0, :3], c["accepted"][0] = [5, 2, 0], 3
    table, *_ = run_commit(c, err, path=i32(bad))
    other = np.delete(np.arange(4), c["rpi"][0])
    assert np.array_equal(table[other], R.commit(**c)[0][other])


def test_step_and_commit_in_a_graph():
    """Lengths that change between replays of one captured step."""
    rng = np.random.default_rng(12)
    B, T = 6, 4
    table = torch.full((B, 400), -1, dtype=torch.int32, device=DEV)
    rpi, cur, new = i32(np.arange(B)), torch.zeros(B, dtype=torch.int32, device=DEV), i32([T] * B)
    free, count = i32(rng.permutation(2000) + 1), i32([2000])
    loc, pos = (torch.zeros(B * T + 3, dtype=torch.int32, device=DEV) for _ in range(2))
    qo, seq = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    path, accepted = i32([[0, 2, -1, -1]] * B), i32([2] * B)

    def step():
        ra.ra_step_slots(table, rpi, cur, new, free, count, loc, pos, qo, seq)
        ra.ra_tree_commit(table, rpi, cur, new, qo, loc, path, accepted, cur, free, count)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        t, f, c = np.full((B, 400), -1, np.int32), host(free).copy(), 2000
        lens = np.zeros(B, np.int64)
        for k in range(5):
            accepted.copy_(i32(1 + (np.arange(B) + k) % 2))
            graph.replay()
            t, l, _, q, _, c = R.step_slots(t, np.arange(B), lens, [T] * B, f, c, 1, B * T)
            n = 1 + (np.arange(B) + k) % 2
            t, f, c, lens = R.commit(t, np.arange(B), lens, [T] * B, q, l, host(path), n, f, c)
    torch.cuda.synchronize()
    assert np.array_equal(host(table), t) and int(count) == c and np.array_equal(host(cur), lens)
    assert np.array_equal(host(free), f)
    assert sorted(set(host(free)[:c]) | set(t[t >= 0])) == list(range(1, 2001))   # no slot lost or doubled


@pytest.mark.parametrize("pages", [0, 3, 9])
def test_requests_without_slots_are_not_committed(pages):
    """Too few free pages: the requests that got the dummy slot keep their lengths and rows, and it is not freed."""
    B, T = 4, 3
    table = i32(np.arange(B * 30).reshape(B, 30) + 100)
    before = host(table)
    rpi, cur, new = i32([2, 0, 3, 1]), i32([5, 0, 7, 20]), i32([T] * B)
    free, count = i32(list(range(1, pages + 1)) + [-9] * (B * T - pages)), i32([pages])
    loc, pos = (torch.full((B * T,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    qo, seq = torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_step_slots(table, rpi, cur, new, free, count, loc, pos, qo, seq, device_error=err)
    assert int(err) == ra.DEVERR_FULL
    err.zero_()
    ra.ra_tree_commit(table, rpi, cur, new, qo, loc, i32([[0, 2, -1]] * B), i32([2] * B), seq, free, count, device_error=err)
    assert int(err) == ra.DEVERR_SLOT
    placed = pages // T
    assert int(count) == pages - 2 * placed
    row = host(table)
    held = [row[r, p:p + 2] for r, p in zip([2, 0, 3, 1][:placed], [5, 0, 7, 20])]
    slots = np.concatenate(held + [host(free)[:int(count)]])
    assert sorted(slots.tolist()) == list(range(1, pages + 1))
    assert host(seq).tolist() == [n + (2 if b < placed else 0) for b, n in enumerate([5, 0, 7, 20])]
    for b in range(placed, B):
        assert np.array_equal(row[[2, 0, 3, 1][b]], before[[2, 0, 3, 1][b]])
