"""ra_tree_attention against 64-bit attention: lengths from none to long, trees and arbitrary masks, rows that
see nothing, values behind a mask that are not finite, splits and their merge, bad requests, graphs."""
import numpy as np
import pytest
import torch

import kv8_ref as R
import prefix_shared_kv_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def i32(a):
    return gpu(np.asarray(a, dtype=np.int32))


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def tree_masks(rng, T, kind):
    """[T, T] visibility among drafted tokens."""
    seen = np.eye(T, dtype=bool)
    if kind == "tree":
        for i in range(1, T):
            parent = rng.integers(-1, i)
            if parent >= 0:
                seen[i] |= seen[parent]
    elif kind == "chain":
        seen = np.tril(np.ones((T, T), bool))
    elif kind == "any":
        seen = rng.random((T, T)) < 0.4
    elif kind == "none":
        seen[:] = False
    return seen


class Case:
    def __init__(self, rng, prefix, draft, hq, hkv, d, kind="tree", words=None, gap=0, scale=None, grow=0.0):
        self.rng, self.hq, self.hkv, self.d = rng, hq, hkv, d
        self.P, self.T = np.asarray(prefix), np.asarray(draft)
        B = len(self.P)
        n = int((self.P + self.T).sum())
        S = n + 7
        perm = rng.permutation(S)
        self.k = gpu(rng.normal(size=(S, hkv, d)).astype(np.float32)).to(BF)
        self.v = gpu(rng.normal(size=(S, hkv, d)).astype(np.float32)).to(BF)
        for x in (self.k, self.v):                           # slots outside every context
            x[torch.from_numpy(perm[n:].copy()).to(DEV)] = float("nan")
        width = int((self.P + self.T).max())
        self.table = np.full((B + 1, width + 2), -1, np.int32)
        self.rpi = rng.permutation(B + 1)[:B]
        at = 0
        for b in range(B):
            m = self.P[b] + self.T[b]
            self.table[self.rpi[b], :m] = perm[at:at + m]
            if grow:  # keys whose scale grows along the context: the softmax's reference moves
                f = gpu((1 + grow * np.arange(m) / 64).astype(np.float32))[:, None, None]
                sl = torch.from_numpy(perm[at:at + m].copy()).to(DEV)
                self.k[sl] = (self.k[sl].float() * f).to(BF)
            at += m
        self.total = int(self.T.sum()) + gap * B
        self.qo = np.concatenate([[0], np.cumsum(self.T + gap)])
        self.max_t = max(int(self.T.max()), 1)
        self.words = words or -(-self.max_t // 32)
        bits = np.zeros((self.total, self.words * 32), bool)
        self.seen = []
        for b in range(B):
            s = tree_masks(rng, int(self.T[b]), kind)
            self.seen.append(s)
            bits[self.qo[b]:self.qo[b] + self.T[b], :self.T[b]] = s
            bits[self.qo[b]:self.qo[b] + self.T[b], self.T[b]:] = True   # bits past the drafted tokens: ignored
        self.mask = np.packbits(bits.reshape(self.total, self.words, 32), axis=-1, bitorder="little").view(np.int32)
        self.mask = self.mask.reshape(self.total, self.words)
        self.q = gpu(rng.normal(size=(self.total, hq, d)).astype(np.float32)).to(BF)
        self.scale = scale or d ** -0.5
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **over):
        a = dict(table=i32(self.table), rpi=i32(self.rpi), P=i32(self.P), T=i32(self.T), qo=i32(self.qo),
                 mask=gpu(self.mask), max_t=self.max_t, max_p=int(self.P.max()))
        a.update(over)
        o = torch.full_like(self.q, 7.0)
        ws = torch.full((ra.ra_tree_workspace_bytes(len(self.P), self.total, self.hq, self.hkv, self.d, a["max_t"]),),
                        0xFF, dtype=torch.uint8, device=DEV)
        ra.ra_tree_attention(self.k, self.v, self.q, o, a["table"], a["rpi"], a["P"], a["T"], a["qo"], a["mask"],
                             max_draft_len=a["max_t"], max_prefix_len=a["max_p"], sm_scale=self.scale, workspace=ws,
                             device_error=self.err)
        return o

    def check(self, o, requests=None, skip=()):
        written = np.zeros(self.total, bool)
        k, v = f64(self.k), f64(self.v)
        for b in range(len(self.P)) if requests is None else requests:
            P, T, q0 = int(self.P[b]), int(self.T[b]), int(self.qo[b])
            written[q0:q0 + T] = True
            if T == 0:
                continue
            slots = self.table[self.rpi[b], :P + T]
            seen = np.concatenate([np.ones((T, P), bool), self.seen[b]], 1)
            ref, a, x = R.attend(f64(self.q[q0:q0 + T]), k[slots], v[slots], self.scale, seen)
            bad = np.abs(f64(o[q0:q0 + T]) - ref) > R.attention_bound(ref, a, x, self.d, R.EPS_BF16)
            assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(f64(o[q0:q0 + T]) - ref).max())
        assert (o[torch.from_numpy(~written).to(DEV)] == 7.0).all()


CASES = [
    # prefix, draft, hq, hkv, d, kind
    ([0], [1], 8, 2, 64, "tree"), ([1], [1], 32, 8, 128, "tree"), ([0, 5], [3, 1], 32, 8, 128, "tree"),
    ([127, 128, 129], [1, 2, 3], 32, 8, 128, "tree"), ([100, 120, 126], [28, 8, 5], 8, 2, 64, "tree"),
    ([1000, 0, 77, 2049], [8, 8, 0, 5], 32, 8, 128, "tree"), ([1500], [64], 64, 8, 128, "tree"),
    ([300, 33], [65, 33], 64, 8, 128, "tree"), ([90, 511], [130, 257], 8, 2, 64, "tree"),
    ([640], [100], 16, 16, 128, "tree"), ([45, 700], [31, 32], 5, 5, 64, "tree"), ([200], [17], 12, 3, 128, "chain"),
    ([260, 10], [40, 96], 32, 8, 128, "any"), ([0, 0, 64], [40, 33, 9], 32, 8, 128, "any"),
    ([0, 130], [70, 70], 8, 2, 64, "none"), ([4000], [4], 8, 1, 128, "tree"), ([250], [12], 16, 1, 128, "tree"),
    ([20, 400], [1024, 700], 4, 1, 64, "tree"), ([70, 0], [1, 3], 32, 1, 128, "tree"), ([300], [5], 128, 1, 64, "tree"),
    ([150, 31], [2, 1], 64, 4, 128, "tree"), ([97], [6], 40, 20, 64, "any"), ([33, 500, 64], [32, 17, 1], 11, 11, 64, "tree"),
    ([33, 500, 64, 7], [16, 9, 1, 16], 16, 16, 64, "tree"), ([300, 15, 1], [8, 7, 1], 28, 14, 64, "any"),
    ([333, 17, 0], [9, 4, 6], 6, 6, 128, "tree"), ([333, 17, 0], [9, 4, 6], 7, 7, 128, "any"),
    (list(range(3, 640, 15)), [1 + i % 8 for i in range(43)], 16, 16, 64, "any"),
]


@pytest.mark.parametrize("prefix,draft,hq,hkv,d,kind", CASES)
def test_tree_matches_64_bit_attention(prefix, draft, hq, hkv, d, kind):
    c = Case(np.random.default_rng(sum(prefix) + sum(draft) + hq), prefix, draft, hq, hkv, d, kind)
    o = c.run()
    assert int(c.err.item()) == 0
    c.check(o)


@pytest.mark.parametrize("batch,longest,bound", [(32, 200, None), (33, 200, None), (6, 900, 1 << 20), (1, 5000, None)])
def test_tree_planned_by_the_warps_and_by_the_kernel(batch, longest, bound):
    """Narrow requests on both sides of the small-call rule, and under a loose bound."""
    rng = np.random.default_rng(batch + longest)
    prefix, draft = rng.integers(0, longest + 1, batch), rng.integers(0, 9, batch)
    prefix[0], draft[0] = longest, 8
    c = Case(rng, prefix, draft, 32, 8, 128, gap=1)
    if bound:
        wide = np.full((c.table.shape[0], bound), -1, np.int32)
        wide[:, :c.table.shape[1]] = c.table
        c.table = wide
    o = c.run(max_p=bound or longest)
    assert int(c.err.item()) == 0
    c.check(o)


@pytest.mark.parametrize("batch", [33, 50, 64, 65])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (5, 5, 64), (4, 1, 128)])
def test_tree_of_more_requests_than_lanes(batch, hq, hkv, d):
    """33 to 64 narrow requests (two per lane of a small call) and one more: empty and invalid ones, split and unsplit
    ones, and a drafted token whose V is not finite."""
    rng = np.random.default_rng(batch + hq)
    prefix, draft = rng.integers(0, 90, batch), rng.integers(0, 9, batch)
    prefix[[0, 31, 32, batch - 1]], draft[[0, 31, 32, batch - 1]] = [400, 60, 333, 250], [8, 1, 7, 5]
    draft[5] = 0
    c = Case(rng, prefix, draft, hq, hkv, d, gap=1)
    P = c.P.copy()
    P[batch - 2] = -1
    slot = int(c.table[c.rpi[32], int(prefix[32]) + 2])
    c.v[slot, 0, 7] = float("inf")
    o = c.run(P=i32(P))
    assert int(c.err.item()) == ra.DEVERR_LENGTH
    at = int(c.qo[batch - 2])
    assert (o[at:at + int(c.T[batch - 2])] == 7.0).all()
    k, v = f64(c.k), f64(c.v)
    for b in range(batch):
        if b == batch - 2 or c.T[b] == 0:
            continue
        Pb, T, q0 = int(c.P[b]), int(c.T[b]), int(c.qo[b])
        slots = c.table[c.rpi[b], :Pb + T]
        seen = np.concatenate([np.ones((T, Pb), bool), c.seen[b]], 1)
        vb = np.where(np.isfinite(v[slots]), v[slots], 0.0)
        ref, a, x = R.attend(f64(c.q[q0:q0 + T]), k[slots], vb, c.scale, seen)
        got = f64(o[q0:q0 + T])
        blind = ~c.seen[b][:, 2] if b == 32 else np.ones(T, bool)      # rows without the infinite value
        bad = np.abs(got - ref) > R.attention_bound(ref, a, x, d, R.EPS_BF16)
        assert not bad[blind].any(), b
        assert b != 32 or not np.isfinite(got[~blind][:, 0, 7]).any()


@pytest.mark.parametrize("hq,hkv,d,draft", [(32, 8, 128, 16), (8, 8, 64, 70), (8, 1, 128, 8), (16, 2, 64, 13)])
def test_tree_one_query_tile_on_the_wide_path(hq, hkv, d, draft):
    """Requests of 33..128 rows per kv head in calls that are not small: both query tiles of an item share out its
    key tiles (even and odd numbers of them, a single one), split (few kv heads) and unsplit."""
    rng = np.random.default_rng(hq + draft)
    prefix, drafts = rng.integers(0, 1100, 40), rng.integers(0, draft + 1, 40)
    prefix[:6], drafts[:6] = [0, 1, 127, 128, 129, 1500], [draft, 1, 1, draft, 1, draft]
    c = Case(rng, prefix, drafts, hq, hkv, d, gap=1)
    o = c.run(max_p=1 << 20 if hq == 32 else 1500, table=i32(np.pad(c.table, ((0, 0), (0, 1 << 20 if hq == 32 else 0)))))
    assert int(c.err.item()) == 0
    c.check(o)
    c = Case(rng, prefix[:34], np.minimum(drafts[:34], 9), hq, hkv, d, "chain", grow=3.0)
    c.max_t = draft
    c.words = -(-draft // 32)
    c.mask = np.pad(c.mask, ((0, 0), (0, c.words - c.mask.shape[1])))
    c.check(c.run())


def test_tree_many_requests_unsplit():
    """Enough items that nothing is split (the direct bf16 rows), with rows between the requests left alone."""
    rng = np.random.default_rng(2)
    c = Case(rng, rng.integers(0, 900, 70), rng.integers(0, 40, 70), 32, 8, 128, gap=2)
    o = c.run()
    assert int(c.err.item()) == 0
    c.check(o)


def test_tree_wider_mask_and_loose_bounds():
    rng = np.random.default_rng(3)
    c = Case(rng, [300, 64], [20, 7], 32, 8, 128, words=5)
    c.check(c.run(max_t=150, max_p=320))


def test_tree_moving_reference():
    """Scores that grow along the context, so that the softmax's reference moves in most tiles, and a first
    chunk whose keys a row does not see."""
    rng = np.random.default_rng(4)
    c = Case(rng, [1200, 0, 0], [40, 200, 90], 32, 8, 128, "chain", grow=4.0)
    c.check(c.run())
    # rows that see only the last drafted tokens, with scores far below zero
    c = Case(rng, [0], [160], 8, 2, 64, "none")
    c.seen[0][:, 150:] = True
    bits = np.zeros((160, 160), bool)
    bits[:, 150:] = True
    c.mask = np.packbits(bits.reshape(160, 5, 32), axis=-1, bitorder="little").view(np.int32).reshape(160, 5)
    c.q[:] = 20.0
    c.k[:] = -20.0
    c.v[:] = torch.randn(c.v.shape, device=DEV).to(BF)
    c.check(c.run())


def test_tree_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(5)
    for prefix in ([0], [0] * 80):
        c = Case(rng, prefix, [9] * len(prefix), 8, 2, 64, "none")
        o = c.run()
        assert not o.any()


@pytest.mark.parametrize("prefix,n,hq", [(0, 1, 32), (300, 1, 32), (2000, 1, 32), (200, 60, 32), (0, 2, 8), (299, 1, 8),
                                         (2000, 1, 8), (200, 60, 8), (999, 40, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_behind_the_mask_do_not_matter(prefix, n, hq, bad):
    """A drafted token whose K and V are not finite changes only rows that see it: wide (hq 32) and narrow (hq 8)
    requests, split and unsplit, planned by the kernel and by the warps."""
    rng = np.random.default_rng(6)
    g = hq // 8
    c = Case(rng, [prefix] * n, [24] * n, hq, 8, 128, "none")
    for s in c.seen:
        s[:] = np.eye(24, dtype=bool)
        s[:, 3] = False
        s[7, 3] = True
    bits = np.zeros((c.total, 32), bool)
    bits[:, :24] = np.concatenate(c.seen)
    c.mask = np.packbits(bits.reshape(c.total, 1, 32), axis=-1, bitorder="little").view(np.int32).reshape(c.total, 1)
    clean = c.run()
    c.check(clean)
    k0, v0 = f64(c.k), f64(c.v)
    slots = c.table[c.rpi, prefix + 3]
    at = torch.from_numpy(slots.astype(np.int64)).to(DEV)
    c.v[at, 2, 5] = bad
    c.k[at, 1, 0] = float("nan")
    o = c.run()
    # rows that do not see token 3 (row 3 itself sees nothing but the prefix): heads whose K and V are fine bit
    # for bit; the others within the bounds of the clean result (row 7's NaN score sends its warp through the
    # exact path, whose reference rounds other rows differently, and the bad V's head is recomputed in fp32)
    rest = np.setdiff1d(np.arange(c.total), np.arange(n) * 24 + 7)
    other = np.setdiff1d(np.arange(hq), np.arange(g, 3 * g))
    assert torch.equal(o[rest][:, other], clean[rest][:, other])
    for b in range(n):
        slots = c.table[c.rpi[b], :prefix + 24]
        seen = np.concatenate([np.ones((24, prefix), bool), c.seen[b]], 1)
        q0 = 24 * b
        ref, a, x = R.attend(f64(c.q[q0:q0 + 24]), k0[slots], v0[slots], c.scale, seen)
        off = np.abs(f64(o[q0:q0 + 24]) - ref) <= R.attention_bound(ref, a, x, c.d, R.EPS_BF16)
        assert np.delete(off, 7, 0).all()
    seeing = o[np.arange(n) * 24 + 7].float()
    assert not torch.isfinite(seeing[:, 2 * g:3 * g, 5]).any()
    assert torch.isnan(seeing[:, g:2 * g]).all()
    if bad != bad:
        assert torch.isnan(seeing[:, 2 * g:3 * g, 5]).all()
    assert torch.isfinite(seeing[:, 3 * g:]).all()


def test_bad_requests_are_flagged_and_skipped():
    rng = np.random.default_rng(7)
    c = Case(rng, [100, 200, 50], [5, 6, 7], 8, 2, 64)
    good = c.run()
    rows1 = slice(int(c.qo[1]), int(c.qo[2]))
    for field, value, bit in (("P", -1, ra.DEVERR_LENGTH), ("P", 201, ra.DEVERR_LENGTH), ("T", 8, ra.DEVERR_LENGTH),
                              ("T", -2, ra.DEVERR_LENGTH), ("rpi", 4, ra.DEVERR_TABLE), ("rpi", -1, ra.DEVERR_TABLE)):
        a = getattr(c, field).copy()
        a[1] = value
        c.err.zero_()
        o = c.run(**{field: i32(a)})
        assert int(c.err.item()) == bit, field
        assert (o[rows1] == 7.0).all()
        # (the others' split may differ once request 1 is gone: the same values up to rounding)
        c.check(o, requests=[0, 2])
    qo = c.qo.copy()
    qo[1] = c.total - 3                                      # rows past the end of q
    c.err.zero_()
    o = c.run(qo=i32(qo))
    assert int(c.err.item()) == ra.DEVERR_LENGTH
    c.check(o, requests=[0, 2])
    t = c.table.copy()
    t[c.rpi[2], 3] = c.k.shape[0]
    c.err.zero_()
    c.k[0] = 0.5
    c.v[0] = 0.25
    o = c.run(table=i32(t))
    assert int(c.err.item()) == ra.DEVERR_SLOT and torch.isfinite(o.float()).all()
    assert good.shape == o.shape


def test_tree_is_deterministic_and_replays_from_a_graph():
    rng = np.random.default_rng(8)
    c = Case(rng, [900, 30, 1800], [12, 64, 33], 32, 8, 128)
    args = [i32(c.table), i32(c.rpi), i32(c.P), i32(c.T), i32(c.qo), gpu(c.mask)]
    o = torch.empty_like(c.q)
    ws = torch.empty(ra.ra_tree_workspace_bytes(3, c.total, 32, 8, 128, 64), dtype=torch.uint8, device=DEV)

    def step():
        ra.ra_tree_attention(c.k, c.v, c.q, o, *args, max_draft_len=64, max_prefix_len=1800, sm_scale=c.scale,
                             workspace=ws)
    step()
    first = o.clone()
    step()
    assert torch.equal(o, first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.q.copy_(torch.randn_like(c.q, dtype=torch.float32).to(BF))
    c.P = c.P - np.array([400, 3, 1])                        # other lengths: another plan on replay
    for b in range(3):                                       # the drafted tokens' slots stay behind the prefix
        n = c.P[b] + c.T[b]
        c.table[c.rpi[b], c.P[b]:n] = c.table[c.rpi[b], c.P[b]:n]
    args[2].copy_(i32(c.P))
    g.replay()
    torch.cuda.synchronize()
    got = o.clone()
    c.check(got)
    step()
    assert torch.equal(o, got)


def test_verify_step_together():
    """A verify step as it is used: drafted tokens' projections normed, rotated and stored, then attended over
    the prefix with the tree's masks; the chain of one branch equals decode of its last token."""
    rng = np.random.default_rng(9)
    hq, hkv, d, P, T = 32, 8, 128, 333, 6
    S = P + T + 3
    kp, vp = (gpu(rng.normal(size=(S, hkv, d)).astype(np.float32)).to(BF) for _ in range(2))
    slots = rng.permutation(S)[:P + T]
    table = np.full((1, P + T), -1, np.int32)
    table[0] = slots
    qkv = gpu(rng.normal(size=(T, hq + 2 * hkv, d)).astype(np.float32)).to(BF)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    depth = np.array([0, 1, 1, 2, 2, 3])
    parent = [-1, 0, 0, 1, 2, 4]
    seen = np.eye(T, dtype=bool)
    for i in range(1, T):
        seen[i] |= seen[parent[i]]
    ang = np.arange(400)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    cs = gpu(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    w = torch.ones(d, dtype=BF, device=DEV)
    qo, o = torch.empty(T, hq, d, dtype=BF, device=DEV), torch.empty(T, hq, d, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_qk_norm_rope_store(q, k, v, w, w, i32(P + depth), cs, qo, kp, vp, i32(slots[P:]), device_error=err)
    bits = np.zeros((T, 32), bool)
    bits[:, :T] = seen
    mask = np.packbits(bits, axis=-1, bitorder="little").view(np.int32)
    ws = torch.empty(ra.ra_tree_workspace_bytes(1, T, hq, hkv, d, T), dtype=torch.uint8, device=DEV)
    ra.ra_tree_attention(kp, vp, qo, o, i32(table), i32([0]), i32([P]), i32([T]), i32([0, T]), gpu(mask),
                         max_draft_len=T, max_prefix_len=P, sm_scale=d ** -0.5, workspace=ws, device_error=err)
    k64, v64 = f64(kp)[slots], f64(vp)[slots]
    full = np.concatenate([np.ones((T, P), bool), seen], 1)
    ref, a, x = R.attend(f64(qo), k64, v64, d ** -0.5, full)
    assert (np.abs(f64(o) - ref) <= R.attention_bound(ref, a, x, d, R.EPS_BF16)).all()
    # branch 0 -> 2 -> 4 -> 5 as a sequence of its own: decode of its last token
    branch = np.concatenate([slots[:P], slots[P + np.array([0, 2, 4, 5])]])[None].astype(np.int32)
    od = torch.empty(1, hq, d, dtype=BF, device=DEV)
    wd = torch.empty(ra.ra_decode_workspace_bytes(1, hq, hkv, d, P + 4), dtype=torch.uint8, device=DEV)
    ra.ra_decode_attention(kp, vp, qo[5:6].contiguous(), od, i32(branch), i32([0]), i32([P + 4]), max_seq_len=P + 4,
                           sm_scale=d ** -0.5, workspace=wd, device_error=err)
    bound = R.attention_bound(ref[5:6], a[5:6], x[5:6], d, R.EPS_BF16)
    assert (np.abs(f64(od) - f64(o[5:6])) <= 2 * bound).all()
    assert int(err.item()) == 0
