"""ra_qk_norm_rope_store and its quantised-pool form against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import kv8_ref as R
import prefix_shared_kv_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def setup(seed, n, hq, hkv, d, rot, extra=0, max_pos=300):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n, hq + 2 * hkv + extra, d)) * 2.0 ** rng.integers(-5, 6, (n, hq + 2 * hkv + extra, 1))
    qkv = torch.from_numpy(x.astype(np.float32)).to(DEV).to(BF)
    q, k, v, _ = qkv.split([hq, hkv, hkv, extra], 1)
    w = [torch.from_numpy((1 + 0.3 * rng.normal(size=d)).astype(np.float32)).to(DEV).to(BF) for _ in range(2)]
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(DEV)
    pos = rng.integers(0, max_pos, n)
    if n > 1:
        pos[0], pos[-1] = 0, max_pos - 1
    slots = n + 11
    loc = rng.permutation(slots)[:n]
    return rng, q, k, v, w, cs, pos, slots, loc


def check_rows(got, x, w, eps, ang, rot, inter):
    """fp32: the mean (d + 2 roundings and the square root's) and six products and sums, 2^-16 of the
    magnitudes is over twice their sum at d = 128; then one rounding to bf16."""
    ref, mag = R.norm_rope(f64(x), None if w is None else f64(w), eps, ang, rot, inter)
    bad = np.abs(f64(got) - ref) > R.EPS_BF16 * np.abs(ref) + 2.0 ** -16 * mag
    assert not bad.any(), np.argwhere(bad)[:3]
    return ref, mag


CASES = [
    # n, hq, hkv, d, rot, interleaved
    (1, 32, 8, 128, 128, False), (64, 32, 8, 128, 128, False), (700, 64, 8, 128, 128, False),
    (5, 8, 2, 64, 64, False), (33, 8, 2, 64, 32, True), (1000, 8, 2, 64, 64, True), (17, 12, 3, 128, 64, False),
    (9, 5, 5, 64, 48, False), (9, 5, 5, 128, 96, False), (31, 16, 16, 128, 16, True), (31, 16, 16, 128, 128, True),
    (3, 20, 20, 64, 16, False), (2, 11, 11, 128, 112, True), (600, 40, 20, 64, 32, False), (50, 7, 1, 128, 32, False),
    # many tokens of few heads: rows of several tokens and blocks share a warp
    (1301, 8, 2, 64, 64, False), (1303, 5, 5, 64, 48, True), (1217, 3, 3, 128, 128, False), (1299, 7, 1, 64, 32, True),
    (1217, 7, 1, 128, 64, False), (437, 5, 11, 64, 16, False), (1219, 9, 3, 64, 64, False), (2433, 1, 1, 128, 128, True),
]


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", CASES)
def test_norm_rope_store_bf16(n, hq, hkv, d, rot, inter):
    rng, q, k, v, w, cs, pos, S, loc = setup(n + hq + rot, n, hq, hkv, d, rot, extra=1)
    kp = torch.full((S, hkv, d), 9.0, dtype=BF, device=DEV)
    vp = torch.full_like(kp, 9.0)
    qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_qk_norm_rope_store(q, k, v, *w, i32(pos), cs, qo, kp, vp, i32(loc), eps=1e-5, interleaved=inter,
                             device_error=err)
    assert int(err.item()) == 0
    ang = cs.double().cpu().numpy()[pos]
    check_rows(qo, q, w[0], 1e-5, ang, rot, inter)
    at = torch.from_numpy(loc).to(DEV)
    check_rows(kp[at], k, w[1], 1e-5, ang, rot, inter)
    assert torch.equal(vp[at], v)
    rest = np.setdiff1d(np.arange(S), loc)
    assert (kp[rest] == 9.0).all() and (vp[rest] == 9.0).all()


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", CASES)
def test_norm_rope_store_kv8(n, hq, hkv, d, rot, inter):
    rng, q, k, v, w, cs, pos, S, loc = setup(2 * n + hq + rot, n, hq, hkv, d, rot)
    pool = torch.full((S, ra.ra_kv8_slot_bytes(hkv, d)), 0xAB, dtype=torch.uint8, device=DEV)
    qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
    ra.ra_qk_norm_rope_kv8_store(q, k, v, *w, i32(pos), cs, qo, pool, i32(loc), interleaved=inter)
    ang = cs.double().cpu().numpy()[pos]
    check_rows(qo, q, w[0], 1e-6, ang, rot, inter)
    rec = pool.cpu().numpy()
    assert np.all(rec[np.setdiff1d(np.arange(S), loc)] == 0xAB)
    rec = rec[loc]
    # V is quantised from bf16: its codes and exponents, and all padding, as ra_kv8_store writes them
    exact = R.pack(f64(v), f64(v))
    hpc = R.hpc_of(hkv)
    is_k = np.zeros(rec.shape[1], bool)
    for h in range(hkv):
        at = h // hpc * (hpc * 2 * d + 16)
        is_k[at + (h % hpc) * 2 * d:at + (h % hpc) * 2 * d + d] = True
        is_k[at + hpc * 2 * d + 2 * (h % hpc)] = True
    assert np.array_equal(rec[:, ~is_k], exact[:, ~is_k])
    # K: a half step of e4m3 (2^-4 relative, 2^-10 of the scale below its normal range) beyond the fp32 value
    ref, mag = R.norm_rope(f64(k), f64(w[1]), 1e-6, ang, rot, inter)
    got, _ = R.unpack(rec, hkv, d)
    e = R.row_exponent(ref)[..., None]
    fp32 = 2.0 ** -16 * mag
    top = np.abs(ref).max(-1, keepdims=True)
    e = np.where(np.abs(np.log2(top / 448) - np.round(np.log2(top / 448))) < 1e-4, e + 1, e)   # either exponent
    bad = np.abs(got - ref) > np.maximum(2.0 ** -4 * (np.abs(ref) + fp32), 2.0 ** -10 * 2.0 ** e) + fp32
    assert not bad.any(), np.argwhere(bad)[:3]


def test_without_weights_in_place_and_other_strides():
    """No norm; q rotated in place inside the projection; k and v from tensors of their own."""
    n, hq, hkv, d, rot = 40, 16, 4, 128, 128
    rng, q, k, v, w, cs, pos, S, loc = setup(5, n, hq, hkv, d, rot)
    before = q.clone()
    k, v = k.contiguous(), v.contiguous()
    kp, vp = (torch.zeros(S, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    ra.ra_qk_norm_rope_store(q, k, v, None, None, i32(pos), cs, q, kp, vp, i32(loc))
    ang = cs.double().cpu().numpy()[pos]
    check_rows(q, before, None, 0.0, ang, rot, False)
    check_rows(kp[torch.from_numpy(loc).to(DEV)], k, None, 0.0, ang, rot, False)


def test_rows_of_zeros_infinities_and_nan():
    """A zero row stays zero (eps > 0); a row's infinity or NaN stays in that row."""
    n, hq, hkv, d = 6, 8, 2, 128
    rng, q, k, v, w, cs, pos, S, loc = setup(8, n, hq, hkv, d, d)
    q[0, 0], q[1, 1, 3], q[2, 2, 70] = 0, float("inf"), float("nan")
    k[3, 1, 0] = float("nan")
    qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
    kp, vp = (torch.zeros(S, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    ra.ra_qk_norm_rope_store(q, k, v, *w, i32(pos), cs, qo, kp, vp, i32(loc))
    assert not qo[0, 0].any()
    assert torch.isnan(qo[2, 2]).all() and torch.isnan(kp[int(loc[3]), 1]).all()
    fine = torch.isfinite(qo.float()).all(-1).cpu().numpy()
    assert not fine[1, 1] and not fine[2, 2] and fine.sum() == n * hq - 2
    assert torch.isfinite(kp.float()).all(-1).sum() == S * hkv - 1


@pytest.mark.parametrize("kv8", [False, True])
def test_bad_positions_and_slots_are_flagged(kv8):
    n, hq, hkv, d = 9, 8, 2, 64
    rng, q, k, v, w, cs, pos, S, loc = setup(11, n, hq, hkv, d, d)
    pos[2], pos[4] = -1, 300
    loc = loc.copy()
    loc[5], loc[6] = -1, S
    qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if kv8:
        pool = torch.zeros(S, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
        ra.ra_qk_norm_rope_kv8_store(q, k, v, *w, i32(pos), cs, qo, pool, i32(loc), device_error=err)
        written = pool.any(1)
    else:
        kp, vp = (torch.zeros(S, hkv, d, dtype=BF, device=DEV) for _ in range(2))
        ra.ra_qk_norm_rope_store(q, k, v, *w, i32(pos), cs, qo, kp, vp, i32(loc), device_error=err)
        written = vp.flatten(1).any(1)
    assert int(err.item()) == ra.DEVERR_POSITION | ra.DEVERR_SLOT
    pos = np.where((pos < 0) | (pos >= 300), 0, pos)
    check_rows(qo, q, w[0], 1e-6, cs.double().cpu().numpy()[pos], d, False)
    assert sorted(np.flatnonzero(written.cpu().numpy())) == sorted(loc[(loc >= 0) & (loc < S)])


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (5, 1, 64), (3, 3, 128), (5, 11, 64)])
@pytest.mark.parametrize("kv8", [False, True])
def test_bad_positions_and_slots_among_many_tokens(kv8, hq, hkv, d):
    """Tokens that share a warp with a bad one are stored as alone; the bad ones' pool rows stay."""
    n = 1217
    rng, q, k, v, w, cs, pos, S, loc = setup(12, n, hq, hkv, d, d)
    loc = loc.copy()
    bad = rng.permutation(n)[:200]
    bad.sort()
    loc_bad = loc.copy()
    loc_bad[bad] = np.where(np.arange(200) % 2, -1, S)
    pools = []
    for at in (loc, loc_bad):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        qo = torch.empty(n, hq, d, dtype=BF, device=DEV)
        if kv8:
            pool = torch.full((S, ra.ra_kv8_slot_bytes(hkv, d)), 0xAB, dtype=torch.uint8, device=DEV)
            ra.ra_qk_norm_rope_kv8_store(q, k, v, *w, i32(pos), cs, qo, pool, i32(at), device_error=err)
        else:
            kp, vp = (torch.full((S, hkv, d), 9.0, dtype=BF, device=DEV) for _ in range(2))
            ra.ra_qk_norm_rope_store(q, k, v, *w, i32(pos), cs, qo, kp, vp, i32(at), device_error=err)
            pool = torch.cat([kp, vp], 1)
        pools.append((pool, qo, int(err.item())))
    assert pools[0][2] == 0 and pools[1][2] == ra.DEVERR_SLOT
    assert torch.equal(pools[0][1], pools[1][1])
    kept = np.setdiff1d(np.arange(S), loc[bad])
    assert torch.equal(pools[0][0][kept], pools[1][0][kept])
    assert (pools[1][0][loc[bad]] == (0xAB if kv8 else 9.0)).all()


def test_layer_steps_together_over_a_quantised_pool():
    """Prefill of three requests (norm, rotation, store, then the prefix read back for the extend call's bf16
    pool), then a decode step: each output against 64-bit attention over the values the pool holds."""
    hq, hkv, d, scale = 16, 4, 128, 128 ** -0.5
    lens = [70, 33, 129]
    n = sum(lens)
    rng, q, k, v, w, cs, pos, S, loc = setup(13, n + 3, hq, hkv, d, d)
    pos = np.concatenate([np.arange(m) for m in lens] + [np.array(lens)])
    pool = torch.zeros(S, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
    qo = torch.empty(n + 3, hq, d, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    starts = np.concatenate([[0], np.cumsum(lens)])
    table = np.full((3, 140), -1, np.int32)
    for b, m in enumerate(lens):
        table[b, :m] = loc[starts[b]:starts[b + 1]]
        table[b, m] = loc[n + b]
    rpi = i32([0, 1, 2])
    p = slice(0, n)
    ra.ra_qk_norm_rope_kv8_store(q[p], k[p], v[p], *w, i32(pos[p]), cs, qo[p], pool, i32(loc[p]), device_error=err)
    # extend over a bf16 pool of the call: row i of it holds token i's values
    kb, vb = (torch.empty(n, hkv, d, dtype=BF, device=DEV) for _ in range(2))
    ra.ra_kv8_load(pool, i32(loc[p]), kb, vb, device_error=err)
    local = np.zeros((3, 140), np.int32)
    for b, m in enumerate(lens):
        local[b, :m] = np.arange(starts[b], starts[b + 1])
    oe = torch.empty(n, hq, d, dtype=BF, device=DEV)
    ws = torch.empty(ra.ra_extend_workspace_bytes(3, n, hq, hkv), dtype=torch.uint8, device=DEV)
    ra.ra_extend_attention(kb, vb, qo[p], oe, i32(local), rpi, i32([0, 0, 0]), i32(lens), i32(starts),
                           max_extend_len=max(lens), max_prefix_len=0, sm_scale=scale, workspace=ws, device_error=err)
    s = slice(n, n + 3)
    ra.ra_qk_norm_rope_kv8_store(q[s], k[s], v[s], *w, i32(pos[s]), cs, qo[s], pool, i32(loc[s]), device_error=err)
    od = torch.empty(3, hq, d, dtype=BF, device=DEV)
    ws2 = torch.empty(ra.ra_decode_workspace_bytes(3, hq, hkv, d, 140), dtype=torch.uint8, device=DEV)
    ra.ra_kv8_decode_attention(pool, qo[s], od, i32(table), rpi, i32([m + 1 for m in lens]), num_kv_heads=hkv,
                               max_seq_len=140, sm_scale=scale, workspace=ws2, device_error=err)
    assert int(err.item()) == 0
    rec = pool.cpu().numpy()
    for b, m in enumerate(lens):
        kk, vv = R.unpack(rec[table[b, :m + 1]], hkv, d)
        rows = slice(starts[b], starts[b + 1])
        ref, a, x = R.attend(f64(qo[rows]), kk[:m], vv[:m], scale, np.tril(np.ones((m, m), bool)))
        assert (np.abs(f64(oe[rows]) - ref) <= R.attention_bound(ref, a, x, d, R.EPS_BF16)).all()
        ref, a, x = R.attend(f64(qo[n + b:n + b + 1]), kk, vv, scale)
        assert (np.abs(f64(od[b:b + 1]) - ref) <= R.attention_bound(ref, a, x, d, R.EPS_F16) + 2.0 ** -24 * m *
                np.abs(vv).max()).all()
