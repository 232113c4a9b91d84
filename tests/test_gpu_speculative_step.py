"""Steps of speculative decoding as a user runs them, all lengths on the GPU: slots for the drafted trees, norm + rotation +
store, tree attention, verification, the accepted path committed, then single tokens and a further chunk with changed
scores over the same table.  Captured once and replayed, against the same steps in 64 bits on the host."""
import numpy as np
import pytest
import torch

import kv8_ref
import mod_ref as M
import prefix_shared_kv_ra_gb300 as ra
import step_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
HQ, HKV, D, VOCAB, T, B = 8, 2, 64, 1009, 7, 5


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Inputs:
    """One step's inputs: a new draw of everything."""

    def __init__(self, rng):
        n = B * T
        self.parents = np.concatenate([R.tree(rng, T) for _ in range(B)])
        self.tokens = rng.integers(0, VOCAB, n)
        logits = rng.normal(size=(n, VOCAB)) * 3
        self.target, self.draft = softmax(logits), softmax(logits + 0.3 * rng.normal(size=logits.shape))
        for b in range(B):
            for i in range(1, T):
                q = self.draft[b * T + self.parents[b * T + i]].astype(np.float64)
                self.tokens[b * T + i] = rng.choice(VOCAB, p=q / q.sum())
        self.u, self.uf = rng.random(n, np.float32), rng.random(B, np.float32)
        self.qkv = rng.normal(size=(n, HQ + 2 * HKV, D)).astype(np.float32)
        self.q1 = rng.normal(size=(B, HQ, D)).astype(np.float32)
        seen = np.zeros((n, 32), bool)
        for b in range(B):
            for i in range(T):
                j = i
                while j >= 0:
                    seen[b * T + i, j] = True
                    j = self.parents[b * T + j]
        self.seen = seen.reshape(B, T, 32)[:, :, :T]
        self.mask = np.packbits(seen, axis=1, bitorder="little").view(np.int32)


def test_steps_captured_and_replayed():
    rng = np.random.default_rng(21)
    n, width, slots = B * T, 220, 900
    first = Inputs(rng)
    # what the step reads and writes, at fixed addresses
    prefix = np.array([0, 3, 40, 64, 17])
    table = np.full((B + 1, width), -1, np.int32)
    ids = rng.permutation(slots - 1) + 1
    at = 0
    for b in range(B):
        table[b, :prefix[b]] = ids[at:at + prefix[b]]
        at += prefix[b]
    g = dict(table=i32(table), rpi=i32(np.arange(B)), seq=i32(prefix), new=i32([T] * B), free=i32(ids[at:]),
             count=i32([len(ids) - at]), loc=i32(np.zeros(n)), pos=i32(np.zeros(n)), qo=i32(np.zeros(B + 1)),
             ends=i32(np.zeros(B)), path=i32(np.zeros((B, T))), acc=i32(np.zeros(B)), next=i32(np.zeros(B)),
             err=torch.zeros(1, dtype=torch.int32, device=DEV))
    k0, v0 = rng.normal(size=(slots, HKV, D)), rng.normal(size=(slots, HKV, D))
    g["k"], g["v"] = (torch.from_numpy(x.astype(np.float32)).to(DEV).to(BF) for x in (k0, v0))
    x = {k: torch.from_numpy(getattr(first, k)).to(DEV) for k in ("target", "draft", "u", "uf")}
    x["tokens"], x["parents"], x["mask"] = i32(first.tokens), i32(first.parents), torch.from_numpy(first.mask).to(DEV)
    x["qkv"], x["q1"] = (torch.from_numpy(getattr(first, k)).to(DEV).to(BF) for k in ("qkv", "q1"))
    w = torch.ones(D, dtype=BF, device=DEV)
    angle = np.arange(width)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    rot = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(DEV)
    q, o = torch.empty(n, HQ, D, dtype=BF, device=DEV), torch.empty(n, HQ, D, dtype=BF, device=DEV)
    o1, oe = torch.empty(B, HQ, D, dtype=BF, device=DEV), torch.empty(n, HQ, D, dtype=BF, device=DEV)
    slopes = torch.from_numpy((2.0 ** -np.arange(1, HQ + 1)).astype(np.float32)).to(DEV)
    scale = D ** -0.5
    tws = torch.empty(ra.ra_tree_workspace_bytes(B, n, HQ, HKV, D, T), dtype=torch.uint8, device=DEV)
    dws = torch.empty(ra.ra_decode_workspace_bytes(B, HQ, HKV, D, width), dtype=torch.uint8, device=DEV)
    ews = torch.empty(ra.ra_extend_mod_workspace_bytes(B, n, HQ, HKV), dtype=torch.uint8, device=DEV)

    def step():
        e = dict(device_error=g["err"])
        ra.ra_step_slots(g["table"], g["rpi"], g["seq"], g["new"], g["free"], g["count"], g["loc"], g["pos"], g["qo"],
                         g["ends"], **e)
        qs, ks, vs = x["qkv"].split([HQ, HKV, HKV], 1)
        ra.ra_qk_norm_rope_store(qs, ks, vs, w, w, g["pos"], rot, q, g["k"], g["v"], g["loc"], **e)
        ra.ra_tree_attention(g["k"], g["v"], q, o, g["table"], g["rpi"], g["seq"], g["new"], g["qo"], x["mask"],
                             max_draft_len=T, max_prefix_len=width - T, sm_scale=scale, workspace=tws, **e)
        # the drafted tokens as a plain chunk, in a layer with capped scores and a window
        ra.ra_extend_attention_mod(g["k"], g["v"], q, oe, g["table"], g["rpi"], g["seq"], g["new"], g["qo"], max_extend_len=T,
                                   max_prefix_len=width - T, sm_scale=scale, workspace=ews, score_cap=20.0, window=30, **e)
        ra.ra_tree_verify(x["target"], x["draft"], x["tokens"], x["parents"], g["new"], g["qo"], x["u"], x["uf"], g["path"],
                          g["acc"], g["next"], max_draft_len=T, **e)
        ra.ra_tree_commit(g["table"], g["rpi"], g["seq"], g["new"], g["qo"], g["loc"], g["path"], g["acc"], g["seq"],
                          g["free"], g["count"], **e)
        # single tokens over what was committed, right behind the lengths that it reads
        ra.ra_decode_attention_mod(g["k"], g["v"], x["q1"], o1, g["table"], g["rpi"], g["seq"], max_seq_len=width,
                                   sm_scale=scale, workspace=dws, score_cap=20.0, window=50, slopes=slopes, **e)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.synchronize()
    ht, hf, hc, hl = table, g["free"].cpu().numpy(), len(ids) - at, prefix
    for k in range(4):
        s = Inputs(rng)
        with torch.cuda.stream(stream):
            for name in ("target", "draft", "u", "uf"):
                x[name].copy_(torch.from_numpy(getattr(s, name)))
            x["tokens"].copy_(i32(s.tokens))
            x["parents"].copy_(i32(s.parents))
            x["mask"].copy_(torch.from_numpy(s.mask))
            x["qkv"].copy_(torch.from_numpy(s.qkv))
            x["q1"].copy_(torch.from_numpy(s.q1))
            graph.replay()
        torch.cuda.synchronize()
        assert int(g["err"]) == 0
        # the step on the host
        ht, loc, pos, qo, ends, hc = R.step_slots(ht, np.arange(B), hl, [T] * B, hf, hc, 1, n)
        assert np.array_equal(g["loc"].cpu(), loc) and np.array_equal(g["pos"].cpu(), pos) and np.array_equal(g["ends"].cpu(), ends)
        kk, vv, qq = f64(g["k"]), f64(g["v"]), f64(q)
        assert torch.equal(g["v"][torch.from_numpy(loc).to(DEV)], x["qkv"][:, HQ + HKV:])
        path, acc, nxt = np.full((B, T), -1), np.zeros(B, int), np.zeros(B, int)
        for b in range(B):
            rows, sl = slice(b * T, b * T + T), ht[b, :ends[b]]
            seen = np.concatenate([np.ones((T, hl[b]), bool), s.seen[b]], 1)
            ref, a, mag = kv8_ref.attend(qq[rows], kk[sl], vv[sl], scale, seen)
            assert (np.abs(f64(o[rows]) - ref) <= kv8_ref.attention_bound(ref, a, mag, D, kv8_ref.EPS_BF16)).all(), (k, b)
            ref, bound = M.attend(qq[rows], kk[sl], vv[sl], scale, hl[b] + np.arange(T), 20.0, None, 30)
            assert (np.abs(f64(oe[rows]) - ref) <= bound).all(), (k, b)
            p, nxt[b] = R.verify(s.target, s.draft, s.tokens, s.parents, T, b * T, s.u, s.uf[b])
            path[b, :len(p)], acc[b] = p, len(p)
        assert np.array_equal(g["path"].cpu(), path) and np.array_equal(g["acc"].cpu(), acc)
        assert np.array_equal(g["next"].cpu(), nxt)
        ht, hf, hc, hl = R.commit(ht, np.arange(B), hl, [T] * B, qo, loc, path, acc, hf, hc)
        assert np.array_equal(g["table"].cpu(), ht) and np.array_equal(g["free"].cpu(), hf) and int(g["count"]) == hc
        assert np.array_equal(g["seq"].cpu(), hl)
        for b in range(B):
            sl = ht[b, :hl[b]]
            ref, bound = M.attend(f64(x["q1"][b:b + 1]), kk[sl], vv[sl], scale, hl[b:b + 1] - 1, 20.0,
                                  slopes.cpu().numpy().astype(np.float64), 50)
            assert (np.abs(f64(o1[b:b + 1]) - ref) <= bound).all(), (k, b)
    assert sorted(set(hf[:hc]) | set(ht[ht >= 0])) == sorted(ids)       # no slot lost or doubled


def test_lengths_read_by_the_next_call_at_once():
    """Planning kernels read lengths before they wait for the kernel in front: a call that wrote them must be over.  Many
    rounds of new lengths, each followed at once by the calls that read them."""
    rng = np.random.default_rng(2)
    batch, width = 90, 400                                    # above what plans in its own warps
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    free = i32(rng.permutation(batch * width) + 1)
    count, left = i32([batch * width]), i32([0])
    k, v = (torch.randn(batch * width + 1, 1, 64, device=DEV).to(BF) for _ in range(2))
    q = torch.randn(batch, 4, 64, device=DEV).to(BF)
    loc, pos = i32(np.zeros(batch * width)), i32(np.zeros(batch * width))
    qo, ends, zero, rpi = i32(np.zeros(batch + 1)), i32(np.ones(batch)), i32(np.zeros(batch)), i32(np.arange(batch))
    news = [i32(rng.integers(1, width, batch)) for _ in range(20)]
    ws = [torch.empty(ra.ra_decode_workspace_bytes(batch, 4, 1, 64, width), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for new in news:
        a, b = torch.empty_like(q), torch.empty_like(q)
        ra.ra_step_slots(table, rpi, zero, new, free, count, loc, pos, qo, ends, free_count_out=left)
        ra.ra_decode_attention(k, v, q, a, table, rpi, ends, max_seq_len=width, sm_scale=0.125, workspace=ws[0])
        ra.ra_decode_attention_mod(k, v, q, b, table, rpi, ends, max_seq_len=width, sm_scale=0.125, workspace=ws[1],
                                   score_cap=50.0)
        outs.append((a, b, table.clone()))
    torch.cuda.synchronize()
    for new, (a, b, t) in zip(news, outs):
        for r in rng.integers(0, batch, 6):
            sl = t[r, :int(new[r])].cpu().numpy()
            for out, cap in ((a, 0.0), (b, 50.0)):
                ref, bound = M.attend(f64(q[r:r + 1]), f64(k)[sl], f64(v)[sl], 0.125, np.array([len(sl) - 1]), cap)
                assert (np.abs(f64(out[r:r + 1]) - ref) <= bound).all()
