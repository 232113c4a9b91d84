"""Verification where requests without drafted tokens, and ones that are refused, leave their clusters of 2, 4 and 8 CTAs at
once, beside requests that stay, many calls in a row on the same buffers."""
import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


@pytest.mark.parametrize("vocab", [900, 4100, 9001, 17003])  # 1, 2, 4 and 8 CTAs a request
@pytest.mark.parametrize("mode", ["given", "drawn", "greedy"])
def test_requests_that_leave_at_once(vocab, mode):
    rng = np.random.default_rng(vocab)
    B, T = 12, 6
    lens = np.array([T, 0, 3, 99, T, 0, 0, 2, T, -1, 1, T])     # 99 and -1 are refused
    live = np.clip(np.where(lens == 99, 0, lens), 0, T)
    qo = np.arange(B + 1) * T
    parents = np.concatenate([R.tree(rng, T) for _ in range(B)])
    logits = (3 * rng.normal(size=(B * T, vocab))).astype(np.float32)
    tokens = rng.integers(0, vocab, B * T)
    for i in range(B * T):
        if parents[i] >= 0 and rng.random() < 0.7:
            tokens[i] = logits[i // T * T + parents[i]].argmax()
    p = np.exp(logits - logits.max(1, keepdims=True))
    p = (p / p.sum(1, keepdims=True)).astype(np.float32)
    q = np.roll(p, 1, 0)
    u, uf = rng.random(B * T, np.float32), rng.random(B, np.float32)
    path, acc, nxt = torch.zeros(B, T, dtype=torch.int32, device=DEV), i32(np.zeros(B)), i32(np.zeros(B))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tree = (i32(tokens), i32(parents), i32(lens), i32(qo))
    x, target, draft = (torch.from_numpy(a).to(DEV) for a in (logits, p, q))
    uu, uuf = torch.from_numpy(u).to(DEV), torch.from_numpy(uf).to(DEV)
    want_path, want_acc, want_next = np.full((B, T), -1), np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        if live[b] == 0:
            continue
        if mode == "greedy":
            walk, t = R.greedy(logits, tokens, parents, live[b], qo[b])
        else:
            walk, t = R.verify(p, q if mode == "drawn" else None, tokens, parents, live[b], qo[b], u, uf[b])
        want_path[b, :len(walk)], want_acc[b], want_next[b] = walk, len(walk), t
    for _ in range(50):
        path.fill_(-7)
        if mode == "greedy":
            ra.ra_tree_verify_greedy(x, *tree, path, acc, nxt, max_draft_len=T, device_error=err)
        else:
            ra.ra_tree_verify(target, draft if mode == "drawn" else None, *tree, uu, uuf, path, acc, nxt, max_draft_len=T,
                              device_error=err)
        assert np.array_equal(path.cpu().numpy(), want_path)
        assert np.array_equal(acc.cpu().numpy(), want_acc) and np.array_equal(nxt.cpu().numpy(), want_next)
    assert int(err) == ra.DEVERR_LENGTH
