"""The operators beside attention where offsets pass 32 bits, on two streams at once, and on padded batches."""
import numpy as np
import pytest
import torch

import kv8_ref as R
import prefix_shared_kv_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def randn(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


def kv8_decode(pool, q, table, lens, hkv, scale, ws=None, rpi=None, **kw):
    o = torch.full_like(q, 7.0)
    n, hq, d = q.shape
    if ws is None:
        ws = torch.empty(ra.ra_decode_workspace_bytes(n, hq, hkv, d, table.shape[1]), dtype=torch.uint8, device=DEV)
    ra.ra_kv8_decode_attention(pool, q, o, table, i32(np.arange(n)) if rpi is None else rpi, lens, num_kv_heads=hkv,
                               max_seq_len=table.shape[1], sm_scale=scale, workspace=ws, **kw)
    return o


def test_pools_past_32_bits():
    """Records and rows at the end of pools of more than 4 GiB."""
    hq, hkv, d, n = 16, 8, 128, 90
    S = 2_200_000                                     # x 2080 bytes, x 2048 bytes a bf16 pool
    rng = np.random.default_rng(0)
    loc = S - 1 - rng.permutation(400)[:n]
    loc[3] = 1
    pool = torch.empty(S, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
    k, v = randn(1, n, hkv, d), randn(2, n, hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_kv8_store(pool, k, v, i32(loc), device_error=err)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    ra.ra_kv8_load(pool, i32(loc), kb, vb, device_error=err)
    rk, rv = R.unpack(R.pack(f64(k), f64(v)), hkv, d)
    assert np.array_equal(f64(kb), rk) and np.array_equal(f64(vb), rv)
    q = randn(3, 1, hq, d)
    o = kv8_decode(pool, q, i32(loc[None]), i32([n]), hkv, d ** -0.5, device_error=err)
    ref, a, x = R.attend(f64(q), rk, rv, d ** -0.5)
    assert (np.abs(f64(o) - ref) <= R.attention_bound(ref, a, x, d, R.EPS_F16) + n * 2.0 ** -24 * np.abs(rv).max()).all()
    del pool
    kp, vp = (torch.empty(S, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    rot = torch.zeros(4, d, device=DEV)
    rot[:, :d // 2] = 1.0                             # no turn: K as it is
    qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
    qq = randn(4, n, hq, d)
    ra.ra_qk_norm_rope_store(qq, k, v, None, None, i32(np.zeros(n)), rot, qo, kp, vp, i32(loc), device_error=err)
    assert torch.equal(kp[torch.from_numpy(loc).to(DEV)], k) and torch.equal(qo, qq)
    for T in (2, 40):                                 # narrow and wide
        P = n - T
        seen = np.tril(np.ones((T, T), bool))
        bits = np.zeros((T, 64), bool)
        bits[:, :T] = seen
        mask = np.packbits(bits.reshape(T, 2, 32), axis=-1, bitorder="little").view(np.int32).reshape(T, 2)
        q = randn(5, T, hq, d)
        o = torch.empty_like(q)
        ws = torch.empty(ra.ra_tree_workspace_bytes(1, T, hq, hkv, d, T), dtype=torch.uint8, device=DEV)
        ra.ra_tree_attention(kp, vp, q, o, i32(loc[None]), i32([0]), i32([P]), i32([T]), i32([0, T]),
                             torch.from_numpy(mask).to(DEV), max_draft_len=T, max_prefix_len=P, sm_scale=d ** -0.5,
                             workspace=ws, device_error=err)
        full = np.concatenate([np.ones((T, P), bool), seen], 1)
        ref, a, x = R.attend(f64(q), f64(k), f64(v), d ** -0.5, full)
        assert (np.abs(f64(o) - ref) <= R.attention_bound(ref, a, x, d, R.EPS_BF16)).all()
    assert int(err.item()) == 0


def test_token_strides_past_32_bits():
    """Rows of a projection whose tokens lie more than 2^31 elements apart in all."""
    n, hq, hkv, d = 3, 4, 2, 64
    stride = 800_000_000
    buf = torch.empty(2 * stride + (hq + 2 * hkv) * d, dtype=BF, device=DEV)
    x = randn(6, n, hq + 2 * hkv, d)
    qkv = buf.as_strided((n, hq + 2 * hkv, d), (stride, d, 1))
    qkv.copy_(x)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    rot = torch.zeros(4, d, device=DEV)
    rot[:, :d // 2] = 1.0
    kp, vp = (torch.zeros(5, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    ra.ra_qk_norm_rope_store(q, k, v, None, None, i32([0, 1, 2]), rot, q, kp, vp, i32([4, 2, 3]))   # in place
    assert torch.equal(qkv, x)
    assert torch.equal(kp[[4, 2, 3]], x[:, hq:hq + hkv]) and torch.equal(vp[[4, 2, 3]], x[:, hq + hkv:])


@pytest.mark.parametrize("batch", [6, 50])
def test_two_streams_at_once(batch):
    """Calls on two streams with workspaces of their own give what they give alone."""
    rng = np.random.default_rng(batch)
    hq, hkv, d = 32, 8, 128
    lens = rng.integers(1, 900, batch)
    S = int(lens.sum()) + 1
    table = np.zeros((batch, 900), np.int32)
    at = 1
    for b, m in enumerate(lens):
        table[b, :m] = np.arange(at, at + m)
        at += m
    k, v = randn(7, S, hkv, d), randn(8, S, hkv, d)
    pool = torch.empty(S, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
    ra.ra_kv8_store(pool, k, v, i32(np.arange(S)))
    T = np.minimum(lens, 6)
    qo = np.concatenate([[0], np.cumsum(T)])
    mask = torch.full((int(qo[-1]), 1), -1, dtype=torch.int32, device=DEV)
    tab, ln, rp = i32(table), i32(lens), i32(np.arange(batch))
    tree_args = (i32(lens - T), i32(T), i32(qo), mask)
    q, qt = randn(9, batch, hq, d), randn(10, int(qo[-1]), hq, d)

    def decode(ws):
        return kv8_decode(pool, q, tab, ln, hkv, 0.09, ws, rp)

    def tree(ws):
        o = torch.empty_like(qt)
        ra.ra_tree_attention(k, v, qt, o, tab, rp, *tree_args, max_draft_len=6, max_prefix_len=900, sm_scale=0.09,
                             workspace=ws)
        return o
    def spaces(n):
        return [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    wd = spaces(ra.ra_decode_workspace_bytes(batch, hq, hkv, d, 900))
    wt = spaces(ra.ra_tree_workspace_bytes(batch, int(qo[-1]), hq, hkv, d, 6))
    alone = decode(wd[0]), tree(wt[0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((decode(wd[i]), tree(wt[i])) if i == 0 else (tree(wt[i]), decode(wd[i]))[::-1])
    torch.cuda.synchronize()
    for outs in got:
        for o in outs:
            assert torch.equal(o[0], alone[0]) and torch.equal(o[1], alone[1])


def test_padded_batch_reads_slot_zero():
    """Padding rows of a captured batch (slot 0, length 1) leave the real rows as they are."""
    hq, hkv, d = 16, 4, 128
    rng = np.random.default_rng(3)
    lens = np.array([70, 300, 1, 45])
    S = int(lens.sum()) + 1
    k, v = randn(11, S, hkv, d), randn(12, S, hkv, d)
    pool = torch.zeros(S, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
    ra.ra_kv8_store(pool, k[1:].contiguous(), v[1:].contiguous(), i32(np.arange(1, S)))
    table = np.zeros((5, 300), np.int32)
    at = 1
    for b, m in enumerate(lens):
        table[b, :m] = np.arange(at, at + m)
        at += m
    q = randn(13, 8, hq, d)
    real = kv8_decode(pool, q[:4].contiguous(), i32(table), i32(lens), hkv, 0.09)
    rows = np.array([0, 1, 2, 3, 4, 4, 4, 4])
    o = kv8_decode(pool, q, i32(table), i32(np.concatenate([lens, [1] * 4])), hkv, 0.09, rpi=i32(rows))
    assert rng is not None and torch.isfinite(o.float()).all()
    assert (o[:4].float() - real.float()).abs().max() <= 2.0 ** -7 * real.float().abs().max()   # (another split)
    assert not o[4:].any()                            # slot 0 holds zeros
