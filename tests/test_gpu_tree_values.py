"""ra_tree_attention where drafted tokens' V hold values that are not finite: rows that do not see them, and dimensions
without them, are bit for bit what zeros in their place give; rows that see them get the infinity or NaN; and the
call's time does not grow with the prefix because of them."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
from test_gpu_tree import Case, gpu, i32

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def masked(c, seen):
    """Give every request of the case the visibility `seen` ([T, T], cut to its tokens)."""
    bits = np.zeros((c.total, c.words * 32), bool)
    for b, t in enumerate(c.T):
        c.seen[b] = seen[:t, :t]
        bits[c.qo[b]:c.qo[b] + t, :t] = c.seen[b]
    c.mask = np.packbits(bits.reshape(c.total, c.words, 32), axis=-1, bitorder="little").view(np.int32)
    c.mask = c.mask.reshape(c.total, c.words)


# prefix, drafted tokens, requests, q heads, kv heads, head dim
FORMS = [
    (5, 8, 1, 32, 8, 128), (300, 8, 3, 32, 8, 128),        # small calls: one piece, several
    (40, 4, 40, 16, 8, 128), (300, 8, 3, 16, 16, 64),      # 33 requests and more; one 16-row block per head
    (250, 12, 5, 8, 8, 128), (3000, 8, 2, 8, 1, 64),       # two row blocks; one head, many pieces
    (1900, 40, 2, 16, 16, 64),                             # several narrow items per request
    (700, 8, 80, 32, 8, 128), (2100, 6, 70, 5, 5, 64),     # narrow items from the plan kernel, unsplit and split
    (150, 16, 70, 32, 8, 128), (900, 16, 6, 64, 8, 128),   # wide, one query tile: unsplit, split
    (200, 70, 40, 32, 8, 128), (2500, 64, 3, 64, 8, 128), (100, 300, 2, 16, 2, 64),  # wide, two tiles and more
]


@pytest.mark.parametrize("prefix,draft,n,hq,hkv,d", FORMS)
def test_values_that_are_not_finite_reach_only_rows_that_see_them(prefix, draft, n, hq, hkv, d):
    rng = np.random.default_rng(prefix + draft + n)
    drafts = np.maximum(draft - np.arange(n) % 3, 1)
    c = Case(rng, [prefix + b % 5 for b in range(n)], drafts, hq, hkv, d, gap=1)
    seen = np.eye(draft, dtype=bool) | (rng.random((draft, draft)) < 0.3)
    first, last = 1, int(drafts.min()) - 1                  # two tokens, each with a value of its own
    seen[:, first] = np.arange(draft) % 2 == 1
    seen[:, last] = np.arange(draft) % 3 == 0
    masked(c, seen)
    heads = sorted({0, hkv - 1})
    at = {}
    for b in range(0, n, 2):                                # every other request
        row = c.table[c.rpi[b]]
        at[b] = [int(row[c.P[b] + first]), int(row[c.P[b] + last])]
        for h in heads:
            c.v[at[b], h] = torch.where(torch.isfinite(c.v[at[b], h]), c.v[at[b], h], torch.zeros_like(c.v[at[b], h]))
            c.v[at[b][0], h, 3] = 0
            c.v[at[b], h, d - 1] = 0
    clean = c.run()
    for b in at:
        for h in heads:
            c.v[at[b][0], h, 3] = -INF
            c.v[at[b][0], h, d - 1] = INF
            c.v[at[b][1], h, d - 1] = -INF if first != last else NAN
    o = c.run()
    want = clean.clone()
    g = hq // hkv
    for b in at:
        rows = np.arange(int(c.qo[b]), int(c.qo[b]) + int(c.T[b]))
        see = [c.seen[b][:, first], c.seen[b][:, last]]
        for h in heads:
            cols = slice(h * g, (h + 1) * g)
            want[rows[see[0]], cols, 3] = -INF
            if first != last:
                want[rows[see[0]], cols, d - 1] = INF
                want[rows[see[1]], cols, d - 1] = -INF
                want[rows[see[0] & see[1]], cols, d - 1] = NAN
            else:
                want[rows[see[0]], cols, d - 1] = NAN
    assert int(c.err.item()) == 0
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(o.float(), 0, 1e39, -1e39), torch.nan_to_num(want.float(), 0, 1e39, -1e39))


@pytest.mark.parametrize("prefix,draft,n,hq", [(300, 5, 2, 32), (300, 5, 60, 32), (300, 40, 3, 32), (300, 16, 50, 32)])
def test_prefix_values_reach_every_row(prefix, draft, n, hq):
    """A prefix token's V that is not finite, in the same key tile as drafted tokens with one of their own."""
    rng = np.random.default_rng(draft)
    c = Case(rng, [prefix] * n, [draft] * n, hq, 8, 128, "none")
    slot = [int(c.table[c.rpi[b], prefix - 1]) for b in range(n)]
    last = [int(c.table[c.rpi[b], prefix + draft - 1]) for b in range(n)]
    clean = c.run()
    c.v[slot, 2, 7] = NAN
    c.v[last, 2, 9] = NAN                                   # seen by no row
    o = c.run()
    g = hq // 8
    assert torch.isnan(o[:, 2 * g:3 * g, 7]).all()
    o[:, 2 * g:3 * g, 7] = clean[:, 2 * g:3 * g, 7]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("draft,n", [(8, 1), (64, 2)])
def test_values_that_are_not_finite_cost_little(draft, n):
    """A long prefix and one drafted value: at most a few times the clean call (a serial pass over the prefix for each
    row of the head would take 100 times as long and more)."""
    rng = np.random.default_rng(11)
    P, hq, hkv, d = 30_000, 64, 8, 128
    c = Case(rng, [P] * n, [draft] * n, hq, hkv, d, "chain")
    args = [i32(c.table), i32(c.rpi), i32(c.P), i32(c.T), i32(c.qo), gpu(c.mask)]
    o = torch.empty_like(c.q)
    ws = torch.empty(ra.ra_tree_workspace_bytes(n, c.total, hq, hkv, d, draft), dtype=torch.uint8, device=c.q.device)

    def timed():
        best = 1e9
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            ra.ra_tree_attention(c.k, c.v, c.q, o, *args, max_draft_len=draft, max_prefix_len=P, sm_scale=c.scale,
                                 workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    clean = timed()
    for b in range(n):
        c.v[int(c.table[c.rpi[b], P]), :, 5] = INF
    assert timed() <= 5 * clean + 1.0, "milliseconds"
    assert torch.isinf(o[:, :, 5]).all() and torch.isfinite(o[:, :, 6]).all()
