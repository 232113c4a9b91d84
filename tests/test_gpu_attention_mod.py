"""ra_extend_attention_mod and ra_decode_attention_mod against 64-bit attention: caps, biases, windows, documents, shared
prefixes and their combinations, rows that see nothing, values that are not finite outside what a row sees, scores far
beyond the cap, references that move, bad requests, streams and graphs."""
import numpy as np
import pytest
import torch

import mod_ref as M
import prefix_shared_kv_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def i32(a):
    return None if a is None else torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """Requests of P cached and E new tokens (decode: E = 1)."""

    def __init__(self, rng, P, E, hq, hkv, d, cap=0.0, window=0, slopes=False, doc=0, full=None, sharp=1.0, grow=0.0, gap=0):
        self.hq, self.hkv, self.d = hq, hkv, d
        self.P, self.E = np.asarray(P), np.asarray(E)
        self.B = len(self.P)
        lens = self.P + self.E
        S = int(lens.sum()) + 9
        perm = rng.permutation(S)
        k, v = rng.normal(size=(S, hkv, d)), rng.normal(size=(S, hkv, d))
        self.table = np.full((self.B + 2, int(lens.max()) + 3), -1, np.int32)
        self.rpi = rng.permutation(self.B + 2)[:self.B]
        at = 0
        for b, n in enumerate(lens):
            slots = perm[at:at + n]
            at += n
            self.table[self.rpi[b], :n] = slots
            if grow:
                k[slots] *= (1 + grow * np.arange(n) / 64)[:, None, None]
        k[perm[at:]] = v[perm[at:]] = np.nan
        self.k = torch.from_numpy(k.astype(np.float32)).to(DEV).to(BF)
        self.v = torch.from_numpy(v.astype(np.float32)).to(DEV).to(BF)
        self.qo = np.concatenate([[0], np.cumsum(self.E + gap)])
        self.total = int(self.qo[-1])
        self.q = torch.from_numpy((sharp * rng.normal(size=(self.total, hq, d))).astype(np.float32)).to(DEV).to(BF)
        self.scale, self.cap, self.window = d ** -0.5, cap, window
        self.slopes = (2.0 ** (-6 * (np.arange(hq) + 1) / hq)).astype(np.float32) if slopes else None
        self.full = None if full is None else np.asarray(full)
        self.first = None
        if doc:
            self.first = np.zeros(self.total, np.int64)
            for b in range(self.B):
                p = self.P[b] + np.arange(self.E[b])
                self.first[self.qo[b]:self.qo[b] + self.E[b]] = p // doc * doc
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def kw(self):
        return dict(sm_scale=self.scale, score_cap=self.cap, window=self.window, device_error=self.err,
                    slopes=None if self.slopes is None else torch.from_numpy(self.slopes).to(DEV), first_key=i32(self.first))

    def extend(self, **over):
        o = torch.full_like(self.q, 7.0)
        ws = torch.full((ra.ra_extend_mod_workspace_bytes(self.B, self.total, self.hq, self.hkv),), 0xFF, dtype=torch.uint8,
                        device=DEV)
        a = dict(self.kw(), full_lens=i32(self.full), max_extend_len=max(1, int(self.E.max())),
                 max_prefix_len=int(self.P.max()), workspace=ws)
        t = dict(rpi=self.rpi, P=self.P, E=self.E, qo=self.qo)
        t.update({k: over.pop(k) for k in list(over) if k in t})
        a.update(over)
        ra.ra_extend_attention_mod(self.k, self.v, self.q, o, i32(self.table), i32(t["rpi"]), i32(t["P"]), i32(t["E"]),
                                   i32(t["qo"]), **a)
        return o

    def decode(self, **over):
        o = torch.full_like(self.q, 7.0)
        longest = int((self.P + 1).max())
        ws = torch.full((ra.ra_decode_workspace_bytes(self.B, self.hq, self.hkv, self.d, longest),), 0xFF, dtype=torch.uint8,
                        device=DEV)
        a = dict(self.kw(), max_seq_len=longest, workspace=ws)
        t = dict(rpi=self.rpi, L=self.P + 1)
        t.update({k: over.pop(k) for k in list(over) if k in t})
        a.update(over)
        ra.ra_decode_attention_mod(self.k, self.v, self.q, o, i32(self.table), i32(t["rpi"]), i32(t["L"]), **a)
        return o

    def check(self, o, requests=None):
        k, v, q, o = f64(self.k), f64(self.v), f64(self.q), f64(o)
        written = np.zeros(self.total, bool)
        for b in range(self.B) if requests is None else requests:
            P, E, q0 = int(self.P[b]), int(self.E[b]), int(self.qo[b])
            rows = slice(q0, q0 + E)
            written[rows] = True
            slots = self.table[self.rpi[b], :P + E]
            full = 0 if self.full is None else min(int(self.full[b]), P + E)
            ref, bound = M.attend(q[rows], k[slots], v[slots], self.scale, P + np.arange(E), self.cap, self.slopes, self.window,
                                  None if self.first is None else self.first[rows], full)
            bad = ~(np.abs(o[rows] - ref) <= bound)
            assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(o[rows] - ref)[bad][:4], bound[bad][:4])
        assert (o[~written] == 7.0).all()


EXTEND = [
    # P, E, hq, hkv, d, what
    ([0], [1], 8, 2, 64, dict(cap=30.0)),
    ([0, 5], [1, 3], 32, 8, 128, dict()),
    ([1000], [33], 32, 8, 128, dict(cap=50.0)),
    ([100, 0, 513], [129, 200, 64], 16, 4, 128, dict(cap=5.0, sharp=4.0)),
    ([700, 31], [100, 257], 8, 8, 64, dict(window=1)),
    ([700, 31], [100, 257], 8, 8, 64, dict(window=128, slopes=True)),
    ([300], [500], 32, 8, 128, dict(window=100, cap=30.0)),
    ([2000, 10], [40, 300], 64, 8, 128, dict(window=1024, cap=20.0, sharp=3.0)),
    ([0, 0], [800, 333], 4, 4, 128, dict(doc=57)),
    ([90], [400], 16, 16, 64, dict(doc=130, slopes=True, cap=50.0)),
    ([0, 40], [600, 300], 32, 8, 128, dict(full=[200, 100])),
    ([0, 40], [600, 300], 8, 1, 128, dict(full=[700, 35], slopes=True)),
    ([17, 260], [300, 90], 32, 32, 128, dict(full=[150, 340], cap=30.0, window=200, slopes=True, doc=64)),
    ([130], [140], 5, 5, 64, dict(window=7, doc=11)),
    ([65, 0, 9], [200, 0, 1], 16, 1, 64, dict(cap=10.0, sharp=6.0, gap=3)),
    ([50], [130], 128, 1, 64, dict(window=20, slopes=True)),
    ([500, 3], [260, 9], 12, 12, 128, dict(cap=1e-3, sharp=2.0)),
    ([500, 3], [260, 9], 8, 2, 128, dict(cap=1e6, sharp=3.0, grow=0.5)),
    ([200], [300], 8, 2, 64, dict(slopes=True, grow=0.4)),
    ([200], [300], 8, 2, 64, dict(cap=40.0, grow=2.0, sharp=2.0)),
]


@pytest.mark.parametrize("i", range(len(EXTEND)))
def test_extend(i):
    P, E, hq, hkv, d, what = EXTEND[i]
    c = Case(np.random.default_rng(i), P, E, hq, hkv, d, **what)
    c.check(c.extend())
    assert int(c.err) == 0


DECODE = [
    ([0], 8, 2, 64, dict(cap=30.0)), ([0, 1, 15, 16, 127, 128], 32, 8, 128, dict(slopes=True)),
    ([1500], 32, 8, 128, dict(cap=50.0)), ([900, 3, 4000], 64, 8, 128, dict(cap=20.0, sharp=3.0, window=1024)),
    ([700] * 30, 8, 8, 64, dict(window=1)), ([700] * 30, 8, 1, 64, dict(window=129, slopes=True)),
    (list(range(0, 2000, 23)), 16, 4, 128, dict(window=333, cap=30.0, slopes=True)),
    ([5000, 200], 5, 5, 64, dict(cap=1e-3)), ([5000, 200], 14, 2, 128, dict(cap=1e6, grow=0.1)),
    ([3000, 20], 32, 32, 128, dict(doc=257, cap=50.0, slopes=True)), ([3000, 20], 32, 8, 128, dict(grow=0.5, cap=40.0)),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i):
    P, hq, hkv, d, what = DECODE[i]
    c = Case(np.random.default_rng(100 + i), P, [1] * len(P), hq, hkv, d, **what)
    c.check(c.decode())
    assert int(c.err) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(d):
    """First keys behind the row, a window before the document: such rows give 0, the others are as ever."""
    rng = np.random.default_rng(d)
    for cap in (0.0, 30.0):
        c = Case(rng, [20, 300, 0], [150, 70, 33], 8, 2, d, cap=cap)
        c.first = rng.integers(-5, 400, c.total)
        c.first[100:150] = 10 ** 9
        c.first[-33:] = 2 ** 31 - 1
        o = c.extend()
        c.check(o)
        assert not o[100:150].any() and not o[-33:].any()
        c = Case(rng, [20, 300, 0, 5000, 77], [1] * 5, 8, 2, d, cap=cap)
        c.first = np.array([21, 299, 1, 2 ** 31 - 1, -9])
        o = c.decode()
        c.check(o)
        assert not o[0].any() and not o[2:4].any() and o[1].any()
        assert int(c.err) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_outside_what_a_row_sees(d, cap, value):
    """K and V that are not finite: rows that do not see them are as ever, rows that see V of one are not finite in the
    dimension where it is."""
    rng = np.random.default_rng(3)
    c = Case(rng, [150], [300], 8, 2, d, cap=cap, window=100)
    slots = torch.from_numpy(c.table[c.rpi[0]].astype(np.int64)).to(DEV)
    clean_v, clean_k = c.v.clone(), c.k.clone()
    bad = [60, 200, 201, 333, 449]                       # positions
    c.v[slots[bad], 0, 3] = value
    c.v[slots[bad], 1, d - 1] = value
    o = f64(c.extend())
    pos = 150 + np.arange(300)
    sees = np.any([(pos >= b) & (pos - b < 100) for b in bad], 0)
    assert not np.isfinite(o[sees][:, :4, 3]).any() and not np.isfinite(o[sees][:, 4:, d - 1]).any()
    c.v = clean_v
    ref = f64(c.extend())
    c.check(torch.from_numpy(ref).to(DEV))
    # the rows that see none are within the bound of the clean result, as are the other dimensions of the rest
    k, v, q = f64(c.k), f64(clean_v), f64(c.q)
    rows = c.table[c.rpi[0], :450]
    exact, bound = M.attend(q, k[rows], v[rows], c.scale, pos, cap, None, 100)
    hit = np.zeros(o.shape, bool)
    hit[:, :4, 3] = sees[:, None]
    hit[:, 4:, d - 1] = sees[:, None]
    assert (np.abs(o - exact) <= bound)[~hit].all()
    # keys: a row sees none of the bad ones
    c.k = clean_k.clone()
    c.k[slots[bad]] = value
    o = f64(c.extend())
    assert (np.abs(o - exact) <= bound)[~sees].all()
    c.k = clean_k
    # decode: values before the window, and behind the context (not in any request's keys)
    c = Case(rng, [500, 90], [1, 1], 8, 2, d, cap=cap, window=100)
    for b, hidden in ((0, slice(0, 401)), (1, slice(0, 0))):
        at = torch.from_numpy(c.table[c.rpi[b]].astype(np.int64)).to(DEV)[hidden]
        c.k[at] = c.v[at] = value
    c.check(c.decode())


def test_scores_far_beyond_the_cap_and_the_reference():
    """Scores of thousands: capped they stay within the cap; uncapped with a bias the reference has to move."""
    rng = np.random.default_rng(4)
    c = Case(rng, [300], [200], 16, 4, 128, cap=15.0, sharp=300.0)
    c.check(c.extend())
    c = Case(rng, [300], [200], 16, 4, 128, cap=15.0, sharp=2.0)
    at = torch.from_numpy(c.table[c.rpi[0], 100:101].astype(np.int64)).to(DEV)
    c.k[at] *= 200                                      # one key leaves the polynomial's range
    c.check(c.extend())
    c = Case(rng, [700, 200], [1, 1], 16, 4, 128, cap=15.0, sharp=300.0)
    c.check(c.decode())
    c = Case(rng, [700], [300], 8, 8, 64, slopes=True)
    c.slopes = np.linspace(-0.5, 3.0, 8).astype(np.float32)   # negative: the farthest key weighs most
    c.check(c.extend())
    c = Case(rng, [700, 2000], [1, 1], 8, 8, 64, slopes=True)
    c.slopes = np.linspace(-0.5, 3.0, 8).astype(np.float32)
    c.check(c.decode())


def test_without_changes_they_are_the_plain_calls():
    """No cap, bias or mask: within rounding of the plain calls; a window of the whole context changes no bit."""
    rng = np.random.default_rng(5)
    c = Case(rng, [400, 0], [100, 300], 32, 8, 128)
    a, b = c.extend(), c.extend(window=100000)
    assert torch.equal(a, b)
    c.check(a)
    c = Case(rng, [400, 0, 3000], [1, 1, 1], 32, 8, 128)
    a, b = c.decode(), c.decode(window=100000)
    assert torch.equal(a, b)
    o = torch.empty_like(c.q)
    ws = torch.empty(ra.ra_decode_workspace_bytes(3, 32, 8, 128, 3001), dtype=torch.uint8, device=DEV)
    ra.ra_decode_attention(c.k, c.v, c.q, o, i32(c.table), i32(c.rpi), i32(c.P + 1), max_seq_len=3001, sm_scale=c.scale,
                           workspace=ws)
    c.check(o)


def test_bad_requests_are_flagged():
    rng = np.random.default_rng(6)
    c = Case(rng, [30, 400, 5], [60, 20, 130], 8, 2, 64, cap=30.0, window=50)
    good = c.extend()
    for key, value, flag in (("rpi", 99, ra.DEVERR_TABLE), ("P", -1, ra.DEVERR_LENGTH), ("P", 401, ra.DEVERR_LENGTH),
                             ("E", -1, ra.DEVERR_LENGTH), ("qo", c.total, ra.DEVERR_LENGTH), ("qo", -1, ra.DEVERR_LENGTH)):
        bad = np.array(getattr(c, key))
        bad[1] = value
        for first in (None, np.zeros(c.total)):
            c.err.zero_()
            o = c.extend(**{key: bad}, first_key=i32(first))
            assert int(c.err) == flag, (key, value)
            assert torch.equal(o[:60], good[:60]) and torch.equal(o[80:], good[80:]) and (o[60:80] == 7.0).all()
    c.err.zero_()
    c.table[c.rpi[1], 401] = 10 ** 8
    c.extend()
    assert int(c.err) == ra.DEVERR_SLOT
    c = Case(rng, [30, 400, 5], [1, 1, 1], 8, 2, 64, cap=30.0, window=50)
    good = c.decode()
    for key, value, flag in (("rpi", -1, ra.DEVERR_TABLE), ("L", 0, ra.DEVERR_LENGTH), ("L", -5, ra.DEVERR_LENGTH)):
        bad = np.array(c.rpi if key == "rpi" else c.P + 1)
        bad[1] = value
        c.err.zero_()
        o = c.decode(**{key: bad})
        assert int(c.err) == flag and (o[1] == 7.0).all() and torch.equal(o[::2], good[::2])


def test_two_streams_and_graphs():
    """Calls at once on two streams; captured calls replayed after their lengths, masks and queries changed."""
    rng = np.random.default_rng(7)
    cases = [Case(rng, [300] * 6, [90] * 6, 32, 8, 128, cap=30.0, window=200) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            outs.append([c.extend() for _ in range(4)])
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o[3])
        assert all(torch.equal(o[0], x) for x in o)
    a, b = cases
    t = [a.k, a.v, a.q, torch.empty_like(a.q), i32(a.table), i32(a.rpi), i32(a.P), i32(a.E), i32(a.qo)]
    first, full = torch.zeros(a.total, dtype=torch.int32, device=DEV), torch.zeros(6, dtype=torch.int32, device=DEV)
    d = [a.k, a.v, a.q[:6].clone(), torch.empty_like(a.q[:6]), t[4], t[5], i32([390, 1, 77, 200, 128, 5])]
    dfirst = torch.zeros(6, dtype=torch.int32, device=DEV)
    ws = torch.empty(ra.ra_extend_mod_workspace_bytes(6, a.total, 32, 8), dtype=torch.uint8, device=DEV)
    dws = torch.empty(ra.ra_decode_workspace_bytes(6, 32, 8, 128, 400), dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            ra.ra_extend_attention_mod(*t, max_extend_len=90, max_prefix_len=300, sm_scale=a.scale, workspace=ws, score_cap=30.0,
                                       first_key=first, full_lens=full)
            ra.ra_decode_attention_mod(*d, max_seq_len=391, sm_scale=a.scale, workspace=dws, score_cap=30.0, first_key=dfirst)
        a.window, a.full = 0, np.array([0, 100, 320, 5, 390, 390])
        a.first = rng.integers(0, 300, a.total)
        first.copy_(i32(a.first))
        full.copy_(i32(a.full))
        t[2].copy_(b.q)
        t[6].copy_(i32([300, 10, 0, 299, 128, 77]))
        a.P = np.array([300, 10, 0, 299, 128, 77])
        dfirst.copy_(i32([300, 0, 70, 0, 127, 4]))
        graph.replay()
    torch.cuda.synchronize()
    a.check(t[3])
    one = Case(rng, [389, 0, 76, 199, 127, 4], [1] * 6, 32, 8, 128, cap=30.0)
    one.k, one.v, one.q, one.table, one.rpi, one.first = a.k, a.v, d[2], a.table, a.rpi, np.array([300, 0, 70, 0, 127, 4])
    one.check(d[3])


def test_pools_past_32_bits():
    rng = np.random.default_rng(8)
    S, hq, hkv, d = 2_200_000, 16, 8, 128
    c = Case(rng, [400], [70], hq, hkv, d, cap=30.0, window=300, slopes=True)
    k, v = (torch.zeros(S, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    slots = S - 1 - np.arange(470)
    old = torch.from_numpy(c.table[c.rpi[0], :470].astype(np.int64)).to(DEV)
    new = torch.from_numpy(slots).to(DEV)
    k[new], v[new] = c.k[old], c.v[old]
    small = (c.k, c.v)
    table = c.table.copy()
    c.k, c.v = k, v
    c.table[c.rpi[0], :470] = slots
    o = c.extend()
    (c.k, c.v), c.table = small, table
    c.check(o)
    one = Case(rng, [469], [1], hq, hkv, d, cap=30.0, window=300, slopes=True)
    one.k, one.v, one.table, one.rpi = k, v, np.full((2, 475), -1, np.int32), np.array([1])
    one.table[1, :470] = slots
    o = one.decode()
    one.k, one.v, one.table, one.rpi = c.k, c.v, c.table, c.rpi
    one.check(o)
    assert int(c.err) == 0 and int(one.err) == 0


@pytest.mark.parametrize("cap", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("split", [False, True])
def test_finite_dimensions_beside_values_that_are_not(cap, split):
    """A visible V value that is not finite: its dimension is not finite, every other one within the bound; a row that sees
    nothing gives 0 beside NaN; values whose products overflow behind capped weights do not."""
    rng = np.random.default_rng(13)
    n = 64 if split else 3000                               # few rows: split key ranges; many: whole ones
    c = Case(rng, [500], [n], 8, 2, 128, cap=cap, sharp=2.0)
    c.first = np.zeros(n, np.int64)
    c.first[5:9] = 10 ** 6                                  # rows that see nothing
    slots = torch.from_numpy(c.table[c.rpi[0]].astype(np.int64)).to(DEV)
    clean = c.v.clone()
    for value in (float("nan"), float("inf")):
        c.v = clean.clone()
        c.v[slots[7], 0, 11] = value                        # seen by all other rows
        c.v[slots[500 + n - 1], 1, 64] = value              # seen by the last row only
        o = f64(c.extend())
        k, v = f64(c.k)[c.table[c.rpi[0], :500 + n]], f64(clean)[c.table[c.rpi[0], :500 + n]]
        some = np.r_[0:40, n - 24:n]
        ref, bound = M.attend(f64(c.q)[some], k, v, c.scale, 500 + some, cap, None, 0, c.first[some], 0)
        hit = np.zeros(ref.shape, bool)
        hit[:, :4, 11] = (c.first[some] == 0)[:, None]
        hit[-1, 4:, 64] = True
        assert not np.isfinite(o[some][hit]).any()
        assert (np.abs(o[some] - ref) <= bound)[~hit].all()
        assert not o[5:9].any()
    c.v = clean.clone()
    c.v[slots[:500], 1] = 2.0 ** 100                        # times weights of up to 2^43: past fp32
    c.k[slots[:500], 1] = c.q[20, 4].sign() * 8.0
    o = f64(c.extend())
    k, v = f64(c.k)[c.table[c.rpi[0], :500 + n]], f64(c.v)[c.table[c.rpi[0], :500 + n]]
    some = np.r_[0:5, 18:24]
    ref, bound = M.attend(f64(c.q)[some], k, v, c.scale, 500 + some, cap)
    assert np.isfinite(o[some]).all() and (np.abs(o[some] - ref) <= bound).all()


@pytest.mark.parametrize("batch,longest", [(1, 8300), (70, 2870), (70, 301)])
def test_documents_over_many_query_tiles(batch, longest):
    """Two tokens a query tile: more tiles than the plan keeps first keys for, more requests than a warp has lanes, and
    requests without new tokens among them."""
    rng = np.random.default_rng(batch + longest)
    E = rng.integers(0, 9, batch)
    E[batch // 2] = longest
    P = rng.integers(0, 20, batch)
    c = Case(rng, P, E, 128, 1, 64, cap=20.0, doc=7, slopes=True)
    o = c.extend()
    assert c.err.item() == 0
    k, v, q, o = f64(c.k), f64(c.v), f64(c.q), f64(o)
    for b in range(batch):
        slots = c.table[c.rpi[b], :P[b] + E[b]]
        for at in range(0, P[b] + E[b], 70):  # whole documents: no row sees outside
            pos = np.arange(max(at, P[b]), min(at + 70, P[b] + E[b]))
            if len(pos) == 0:
                continue
            rows = c.qo[b] + pos - P[b]
            keys = slots[at:at + 70]
            ref, bound = M.attend(q[rows], k[keys], v[keys], c.scale, pos - at, c.cap, c.slopes, 0, c.first[rows] - at, 0)
            bad = ~(np.abs(o[rows] - ref) <= bound)
            assert not bad.any(), (b, at, np.argwhere(bad)[:4])


@pytest.mark.parametrize("shift", [16, 48])
def test_workspaces_at_16_byte_boundaries(shift):
    """Split ranges, so that partial rows are written; old bytes around the workspace stay."""
    kw = dict(cap=30.0, slopes=True)
    e, c = (Case(np.random.default_rng(shift), [900, 20], E, 16, 4, 128, **kw) for E in ([40, 3], [1, 1]))
    for call, size in ((e.extend, ra.ra_extend_mod_workspace_bytes(2, e.total, 16, 4)),
                       (c.decode, ra.ra_decode_workspace_bytes(2, 16, 4, 128, 901))):
        big = torch.full((size + 128,), 0xA5, dtype=torch.uint8, device=DEV)
        assert big.data_ptr() % 64 == 0
        assert torch.equal(call(workspace=big[shift:shift + size]), call())
        assert (big[:shift] == 0xA5).all() and (big[shift + size:] == 0xA5).all()


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("hidden", [1, 70, 600])
def test_scores_of_minus_infinity(hidden, slopes):
    """Keys that rows see with a score of minus infinity weigh nothing, also where a whole tile, slab or piece has no other."""
    rng = np.random.default_rng(hidden)
    e, c = (Case(rng, [700, 640], E, 8, 2, 64, slopes=slopes) for E in ([40, 3], [1, 1]))
    for case, call in ((e, e.extend), (c, c.decode)):
        case.q = (case.q.abs() + 0.125).to(BF)
        for b in range(2):
            case.k[torch.from_numpy(case.table[case.rpi[b], :hidden]).long().to(DEV)] = -float("inf")
        o = f64(call())
        assert int(case.err) == 0
        k, v, q = f64(case.k), f64(case.v), f64(case.q)
        for b in range(2):
            P, E, q0 = int(case.P[b]), int(case.E[b]), int(case.qo[b])
            slots = case.table[case.rpi[b], hidden:P + E]
            ref, bound = M.attend(q[q0:q0 + E], k[slots], v[slots], case.scale, P + np.arange(E) - hidden, 0.0, case.slopes)
            bad = ~(np.abs(o[q0:q0 + E] - ref) <= bound)
            assert not bad.any(), (b, np.argwhere(bad)[:4])
