"""ra_tree_verify and ra_tree_verify_greedy against their definitions in 64 bits: drafts drawn and given, odd
vocabularies and row strides, repeated tokens, empty residuals, values that are not finite, the distribution of what
comes out, bad requests, streams and graphs."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def f32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV)


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Trees:
    def __init__(self, rng, drafts, vocab, spread=2.0, noise=0.7, gap=0):
        self.T, self.vocab = np.asarray(drafts), vocab
        self.B = len(self.T)
        self.total = int(self.T.sum()) + gap * self.B
        self.qo = np.concatenate([[0], np.cumsum(self.T + gap)])
        self.widest = max(int(self.T.max(initial=0)), 1)
        self.parents = np.full(self.total, -1)
        for b, T in enumerate(self.T):
            if T:
                self.parents[self.qo[b]:self.qo[b] + T] = R.tree(rng, T)
        logits = rng.normal(size=(self.total, vocab)) * spread
        self.target = softmax(logits)
        self.draft = softmax(logits + noise * rng.normal(size=logits.shape))
        self.tokens = rng.integers(0, vocab, self.total)
        for b, T in enumerate(self.T):
            for i in range(1, T):
                q0 = self.qo[b]
                q = self.draft[q0 + self.parents[q0 + i]].astype(np.float64)
                self.tokens[q0 + i] = rng.choice(vocab, p=q / q.sum())
        self.u, self.uf = rng.random(self.total, np.float32), rng.random(self.B, np.float32)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def outputs(self):
        return (torch.full((self.B, self.widest), -7, dtype=torch.int32, device=DEV),
                *(torch.full((self.B,), -7, dtype=torch.int32, device=DEV) for _ in range(2)))

    def run(self, drawn, stride=0, **over):
        def rows(x):
            t = f32(x)
            if stride:
                wide = torch.full((t.shape[0], self.vocab + stride), float("nan"), device=DEV)
                wide[:, 1:self.vocab + 1] = t
                t = wide[:, 1:self.vocab + 1]
            return t

        out = self.outputs()
        a = dict(tokens=i32(self.tokens), parents=i32(self.parents), T=i32(self.T), qo=i32(self.qo))
        a.update(over)
        ra.ra_tree_verify(rows(self.target), rows(self.draft) if drawn else None, a["tokens"], a["parents"], a["T"], a["qo"],
                          f32(self.u), f32(self.uf), *out, max_draft_len=self.widest, device_error=self.err)
        return [x.cpu().numpy() for x in out]

    def check(self, got, drawn, requests=None):
        path, accepted, nxt = got
        for b in range(self.B) if requests is None else requests:
            if self.T[b] == 0:
                assert accepted[b] == 0 and nxt[b] == 0 and (path[b] == -1).all()
                continue
            ref, token = R.verify(self.target, self.draft if drawn else None, self.tokens, self.parents, self.T[b],
                                  self.qo[b], self.u, self.uf[b])
            assert list(path[b]) == ref + [-1] * (self.widest - len(ref)), b
            assert accepted[b] == len(ref) and nxt[b] == token, (b, token, nxt[b])


CASES = [([1], 1), ([2], 2), ([3, 0, 7], 5), ([8] * 4, 32003), ([16] * 9, 1000), ([64, 33, 1], 4097), ([5] * 3, 100000),
         ([1024, 300], 61), ([4] * 100, 8191), ([2, 3], 65536), ([12] * 5, 4096)]


@pytest.mark.parametrize("drafts,vocab", CASES)
@pytest.mark.parametrize("drawn", [False, True])
def test_verify(drafts, vocab, drawn):
    t = Trees(np.random.default_rng(vocab + len(drafts)), drafts, vocab, gap=vocab % 2)
    t.check(t.run(drawn), drawn)
    assert int(t.err) == 0


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("stride", [2, 5])
def test_verify_strided_rows(drawn, stride):
    t = Trees(np.random.default_rng(stride), [9, 4, 17], 7001)
    t.check(t.run(drawn, stride), drawn)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_wide_nodes_with_repeated_tokens(drawn):
    """Every node a child of node 0, tokens repeated, numbers that refuse most; and ones that accept the last."""
    rng = np.random.default_rng(5)
    for low in (0.0, 0.9, 0.999):
        t = Trees(rng, [40, 700, 2], 37, spread=0.5)
        t.parents = np.where(t.parents >= 0, 0, -1)
        t.u = (low + (1 - low) * rng.random(t.total)).astype(np.float32)
        t.u[t.u >= 1] = np.float32(1 - 2 ** -24)
        t.check(t.run(drawn), drawn)
        assert int(t.err) == 0


def test_verify_empty_residuals():
    """q equal to p: a refusal (a number above 1 cannot be, but q(x) of a token is) leaves nothing, and p is drawn from;
    given drafts that held all of p likewise."""
    t = Trees(np.random.default_rng(6), [6] * 8, 50)
    t.target[:] = 1 / 64
    t.target[:, 32:] = 0                        # sums to 1/2, exactly
    t.draft[:] = t.target * 2                   # p - q <= 0 everywhere
    t.tokens = t.tokens % 32
    t.check(t.run(True), True)
    t.target[:] = 0
    t.target[:, 7] = 1
    t.tokens[:] = 7
    t.u[:] = np.float32(1 - 2 ** -24)
    t.check(t.run(False), False)                # accepted: u < 1
    t.target[:, 7] = 0.5                        # refused, and nothing else has weight
    t.check(t.run(False), False)
    assert int(t.err) == 0


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_ends_of_the_numbers(drawn):
    """u = 0 and the largest u below 1; zero weights at both ends of the vocabulary are never drawn."""
    t = Trees(np.random.default_rng(7), [3] * 64, 5000)
    t.target[:, :11] = 0
    t.target[:, -13:] = 0
    t.target[::5, :4990 - 13] = 0
    t.draft[:, :11] = t.draft[:, -13:] = 0
    t.uf[::2], t.uf[1::2] = 0, np.float32(1 - 2 ** -24)
    t.u[::3] = 0
    got = t.run(drawn)
    t.check(got, drawn)
    assert (got[2] >= 11).all() and (got[2] < 4987).all() and int(t.err) == 0


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_values_that_are_not_finite(drawn):
    """NaN and negative entries count as 0; a row of them, or with an infinity, is flagged and gives token 0; rows that
    no accepted node reaches have no influence."""
    t = Trees(np.random.default_rng(8), [1] * 6, 3000)
    t.target[0, 5::3] = np.nan
    t.target[1, 100:2900] = -1
    t.check(t.run(drawn), drawn)
    assert int(t.err) == 0
    for value in (np.nan, 0.0, -2.0):
        t.target[2] = value
        got = t.run(drawn)
        assert int(t.err) == ra.DEVERR_VALUE and got[2][2] == 0
        t.check(got, drawn, [0, 1, 3, 4, 5])
        t.err.zero_()
    t.target[2, 50] = np.inf
    got = t.run(drawn)
    assert int(t.err) == ra.DEVERR_VALUE and got[2][2] == 0
    t.check(got, drawn, [0, 1, 3, 4, 5])
    t = Trees(np.random.default_rng(9), [20] * 4, 500)
    reached = t.run(drawn)
    for b in range(4):
        for i in set(range(20)) - set(reached[0][b]):
            t.target[t.qo[b] + i] = np.nan
            t.draft[t.qo[b] + i] = np.nan
    t.check(t.run(drawn), drawn)
    assert int(t.err) == 0


def test_verify_flags_bad_requests():
    t = Trees(np.random.default_rng(10), [5, 6, 7], 300)
    for key, value, flag in (("T", 8, ra.DEVERR_LENGTH), ("T", -1, ra.DEVERR_LENGTH), ("qo", 18, ra.DEVERR_LENGTH),
                             ("qo", -1, ra.DEVERR_LENGTH)):
        bad = np.array(t.T if key == "T" else t.qo)
        bad[1] = value
        for drawn in (False, True):
            t.err.zero_()
            got = t.run(drawn, **{key: i32(bad)})
            assert int(t.err) == flag and got[1][1] == 0 and got[2][1] == 0 and (got[0][1] == -1).all()
            t.check(got, drawn, [0, 2])
    t.err.zero_()
    tokens = t.tokens.copy()
    tokens[t.qo[1] + 1], tokens[t.qo[2] + 1] = 300, -4          # (node 1 is a child of node 0)
    t.tokens = tokens
    for drawn in (False, True):
        t.check(t.run(drawn), drawn)
        assert int(t.err) == ra.DEVERR_VALUE
    parents = t.parents.copy()
    parents[t.qo[0] + 3], parents[t.qo[0] + 2] = 4, 99           # not before the node: never reached
    got = t.run(False, parents=i32(parents))
    t.parents[t.qo[0] + 3] = t.parents[t.qo[0] + 2] = -1
    t.check(got, False)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_keeps_the_targets_distribution(drawn):
    """The first token that comes out of 60,000 trees of three drafts at node 0 has the target's distribution: counts
    within 5 standard deviations of a binomial."""
    rng = np.random.default_rng(11)
    n, vocab = 60000, 6
    p, q = softmax(rng.normal(size=vocab) * 1.2), softmax(rng.normal(size=vocab) * 1.2)
    tokens = rng.choice(vocab, p=q.astype(np.float64) / q.astype(np.float64).sum(), size=(n, 4))
    if not drawn:
        tokens[:] = [0, 2, 5, 2]                                 # the same drafts each time, whatever q is
    parents = np.tile([-1, 0, 0, 0], n)
    out = (torch.empty(n, 4, dtype=torch.int32, device=DEV), *(torch.empty(n, dtype=torch.int32, device=DEV) for _ in "ab"))
    rows = lambda x: f32(x).expand(4 * n, vocab).contiguous()
    ra.ra_tree_verify(rows(p), rows(q) if drawn else None, i32(tokens.ravel()), i32(parents), i32([4] * n),
                      i32(4 * np.arange(n + 1)), f32(rng.random(4 * n, np.float32)), f32(rng.random(n, np.float32)), *out,
                      max_draft_len=4)
    path, accepted, nxt = [x.cpu().numpy() for x in out]
    first = np.where(accepted > 1, tokens[np.arange(n), np.maximum(path[:, 1], 0)], nxt)
    counts, want = np.bincount(first, minlength=vocab), p.astype(np.float64) / p.astype(np.float64).sum()
    assert (np.abs(counts - n * want) <= 5 * np.sqrt(n * want * (1 - want))).all()
    assert 0.2 < (accepted > 1).mean() < 1.0


def greedy_case(rng, drafts, vocab, dtype):
    t = Trees(rng, drafts, vocab)
    logits = f32(rng.normal(size=(t.total, vocab)) * 2).to(dtype)
    t.logits = logits
    wide = logits.float().cpu().numpy()
    for b, T in enumerate(t.T):
        for i in range(1, T):
            q0 = t.qo[b]
            if rng.random() < 0.7:
                t.tokens[q0 + i] = int(wide[q0 + t.parents[q0 + i]].argmax())
    return t


def run_greedy(t, logits=None):
    out = t.outputs()
    ra.ra_tree_verify_greedy(t.logits if logits is None else logits, i32(t.tokens), i32(t.parents), i32(t.T), i32(t.qo), *out,
                             max_draft_len=t.widest, device_error=t.err)
    return [x.cpu().numpy() for x in out]


def check_greedy(t, got):
    wide = t.logits.float().cpu().numpy()
    for b in range(t.B):
        if t.T[b] == 0:
            assert got[1][b] == 0 and got[2][b] == 0 and (got[0][b] == -1).all()
            continue
        ref, token = R.greedy(wide, t.tokens, t.parents, t.T[b], t.qo[b])
        assert list(got[0][b][:got[1][b]]) == ref and (got[0][b][got[1][b]:] == -1).all() and got[2][b] == token, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("drafts,vocab", [([1], 1), ([4, 0, 9], 3), ([8] * 4, 32003), ([64] * 3, 1000), ([16] * 40, 4099),
                                          ([5, 5], 128000), ([1024], 17)])
def test_greedy(dtype, drafts, vocab):
    t = greedy_case(np.random.default_rng(vocab), drafts, vocab, dtype)
    check_greedy(t, run_greedy(t))
    assert int(t.err) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy_ties_infinities_and_nan(dtype):
    t = greedy_case(np.random.default_rng(3), [1] * 12, 9001, dtype)
    x = t.logits
    x[0] = 1.5                                    # all equal
    x[1] = -float("inf")
    x[2] = 0.0
    x[2, 1234:] = -0.0                            # equal values of two signs
    x[2, :1000] = -1.0
    x[3, 17], x[3, 8000], x[3, 16] = float("inf"), float("inf"), float("nan")
    x[4, ::2] = float("nan")
    x[5] = -float("inf")
    x[5, 9000] = -3e38
    x[6, 8999:] = 9.0                             # ties at the end of the row
    x[7, [0, 8, 4096]] = 11.0
    x[8] = float("nan")
    x[8, 5000] = -float("inf")
    x[9], x[9, 3001:] = -0.0, 0.0
    check_greedy(t, run_greedy(t))
    assert int(t.err) == 0
    x[10] = float("nan")
    check_greedy(t, run_greedy(t))
    assert int(t.err) == ra.DEVERR_VALUE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy_strided_rows(dtype):
    """Rows at an odd stride from an odd start, values around them larger."""
    t = greedy_case(np.random.default_rng(4), [6, 11], 5003, dtype)
    for before, after in ((1, 0), (3, 4), (7, 2)):
        wide = torch.full((t.total, 5003 + before + after), 1e9, dtype=dtype, device=DEV)
        wide[:, before:before + 5003] = t.logits
        check_greedy(t, run_greedy(t, wide[:, before:before + 5003]))


def test_rows_past_32_bits():
    """A row whose first value is more than 2^32 values behind the first row's."""
    vocab, n = 1 << 20, 4200
    logits = torch.zeros(n, vocab, dtype=torch.bfloat16, device=DEV)
    logits[n - 2, 777], logits[n - 1, 1048575] = 2.0, 3.0
    out = (torch.empty(1, 2, dtype=torch.int32, device=DEV), *(torch.empty(1, dtype=torch.int32, device=DEV) for _ in "ab"))
    tokens, parents = i32(np.full(n, 777)), i32(np.where(np.arange(n) == n - 1, 0, -1))
    ra.ra_tree_verify_greedy(logits, tokens, parents, i32([2]), i32([n - 2, n]), *out, max_draft_len=2)
    assert out[0].tolist() == [[0, 1]] and out[2].tolist() == [1048575]
    del logits
    probs = torch.zeros(n, vocab, device=DEV)
    probs[n - 2, 777], probs[n - 1, 1000000] = 1.0, 1.0
    ra.ra_tree_verify(probs, None, tokens, parents, i32([2]), i32([n - 2, n]), f32(np.full(n, 0.5)), f32([0.5]), *out,
                      max_draft_len=2)
    assert out[0].tolist() == [[0, 1]] and out[2].tolist() == [1000000]


def test_two_streams_and_a_graph():
    a, b = (Trees(np.random.default_rng(s), [16] * 60, 20011) for s in (1, 2))
    tensors = [[f32(t.target), f32(t.draft), i32(t.tokens), i32(t.parents), i32(t.T), i32(t.qo), f32(t.u), f32(t.uf),
                *t.outputs()] for t in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x in zip(streams, tensors):
            ra.ra_tree_verify(*x, max_draft_len=16, stream=s)
    torch.cuda.synchronize()
    for t, x in zip((a, b), tensors):
        t.check([y.cpu().numpy() for y in x[8:]], True)
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            ra.ra_tree_verify(*tensors[0], max_draft_len=16)
        for i in range(8):
            tensors[0][i].copy_(tensors[1][i])
        graph.replay()
    torch.cuda.synchronize()
    b.check([y.cpu().numpy() for y in tensors[0][8:]], True)
