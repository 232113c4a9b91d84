"""Quantised pools on the GPU: the store bit for bit against the record's definition, the read-back exactly,
decode attention against 64-bit softmax over the values the records stand for."""
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


def rows(rng, *shape, lo=-6, hi=6):
    x = rng.normal(size=shape) * 2.0 ** rng.integers(lo, hi, shape[:-1] + (1,))
    return gpu(x.astype(np.float32)).to(BF)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


SHAPES = [(1, 64), (1, 128), (2, 64), (3, 128), (5, 64), (8, 128), (8, 64), (12, 128), (16, 128), (20, 64), (11, 128)]


@pytest.mark.parametrize("hkv,d", SHAPES)
@pytest.mark.parametrize("n", [1, 7, 300])
def test_store_writes_the_record_and_load_reads_it(hkv, d, n):
    rng = np.random.default_rng(n * 1000 + hkv * 10 + d)
    k, v = rows(rng, n, hkv, d), rows(rng, n, hkv, d)
    k[0, 0] = 0                                              # a zero row: exponent -118, codes 0
    v[-1, -1, :3] = torch.tensor([1e-30, -2e-30, 0.0]).to(BF)
    S = n + 9
    pool = torch.full((S, ra.ra_kv8_slot_bytes(hkv, d)), 0xAB, dtype=torch.uint8, device=DEV)
    loc = rng.permutation(S)[:n]
    err = err_word()
    ra.ra_kv8_store(pool, k, v, i32(loc), device_error=err)
    got = pool.cpu().numpy()
    exp = R.pack(f64(k), f64(v))
    assert np.array_equal(got[loc], exp)
    assert np.all(got[np.setdiff1d(np.arange(S), loc)] == 0xAB)   # other records untouched
    k2, v2 = torch.full_like(k, 7), torch.full_like(v, 7)
    ra.ra_kv8_load(pool, i32(loc), k2, v2, device_error=err)
    rk, rv = R.unpack(exp, hkv, d)
    assert np.array_equal(f64(k2), rk) and np.array_equal(f64(v2), rv)
    assert int(err.item()) == 0


def test_store_special_values():
    """Infinities saturate to +-448 at the exponent of the row's finite values, NaN stays NaN, values at the
    largest and smallest magnitudes keep finite values."""
    d, big = 64, float(torch.finfo(BF).max)
    k = torch.zeros(1, 8, d, dtype=BF)
    k[0, 0, :4] = torch.tensor([float("inf"), 1.0, float("-inf"), 0.5]).to(BF)
    k[0, 1, :3] = torch.tensor([float("nan"), 3.0, -1.0]).to(BF)
    k[0, 2, :3] = torch.tensor([big, -big, 2.0 ** 120]).to(BF)
    k[0, 3, :3] = torch.tensor([2.0 ** -133, -2.0 ** -126, 2.0 ** -120]).to(BF)
    k[0, 4] = float("inf")
    k[0, 5, :2] = torch.tensor([448.0, 1.75 * 2 ** 8]).to(BF)
    k[0, 6, :2] = torch.tensor([450.0, 1.0]).to(BF)
    k[0, 7, :2] = torch.tensor([-0.0, 0.0]).to(BF)
    k = k.to(DEV)
    pool = torch.zeros(2, ra.ra_kv8_slot_bytes(8, d), dtype=torch.uint8, device=DEV)
    ra.ra_kv8_store(pool, k, k, i32([1]))
    exp = R.pack(f64(k), f64(k))
    assert np.array_equal(pool.cpu().numpy()[1:], exp)
    k2, v2 = torch.empty_like(k), torch.empty_like(k)
    ra.ra_kv8_load(pool, i32([1]), k2, v2)
    assert torch.isfinite(k2[0, [0, 2, 3, 4, 5, 6, 7]].float()).all() and torch.isnan(k2[0, 1, 0])
    rk, _ = R.unpack(exp, 8, d)
    assert np.array_equal(f64(k2), rk, equal_nan=True)


def test_bad_slots_are_flagged_and_skipped():
    hkv, d = 2, 64
    rng = np.random.default_rng(5)
    k, v = rows(rng, 4, hkv, d), rows(rng, 4, hkv, d)
    pool = torch.zeros(6, ra.ra_kv8_slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
    err = err_word()
    ra.ra_kv8_store(pool, k, v, i32([3, 6, -1, 5]), device_error=err)
    assert int(err.item()) == ra.DEVERR_SLOT
    exp = R.pack(f64(k), f64(v))
    got = pool.cpu().numpy()
    assert np.array_equal(got[[3, 5]], exp[[0, 3]]) and not got[[0, 1, 2, 4]].any()
    err.zero_()
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    ra.ra_kv8_load(pool, i32([3, 9, 3, -2]), k2, v2, device_error=err)       # a slot twice, two bad ones
    assert int(err.item()) == ra.DEVERR_SLOT
    rk, _ = R.unpack(exp, hkv, d)
    assert np.array_equal(f64(k2)[[0, 2]], rk[[0, 0]]) and not f64(k2)[[1, 3]].any()


@pytest.mark.parametrize("hkv,d", SHAPES + [(4, 128), (6, 128), (7, 64)])
def test_many_tokens_with_special_values_and_bad_slots(hkv, d):
    """Enough tokens that a warp takes whole blocks, or several of them, at once; the last ones leave it part empty."""
    n = 2501
    rng = np.random.default_rng(hkv + d)
    k, v = rows(rng, n, hkv, d), rows(rng, n, hkv, d)
    k[3, 0, :3] = torch.tensor([float("inf"), 1.0, float("nan")]).to(BF)
    v[n - 1, hkv - 1, :2] = torch.tensor([float("-inf"), 0.25]).to(BF)
    k[7], v[8, 0] = 0, float("inf")
    S = n + 5
    loc = rng.permutation(S)[:n]
    bad = np.sort(rng.permutation(n)[:150])
    at = loc.copy()
    at[bad] = np.where(np.arange(150) % 2, -1, S)
    good = np.setdiff1d(np.arange(n), bad)
    pool = torch.full((S, ra.ra_kv8_slot_bytes(hkv, d)), 0xAB, dtype=torch.uint8, device=DEV)
    err = err_word()
    ra.ra_kv8_store(pool, k, v, i32(at), device_error=err)
    assert int(err.item()) == ra.DEVERR_SLOT
    got = pool.cpu().numpy()
    exp = R.pack(f64(k), f64(v))
    assert np.array_equal(got[loc[good]], exp[good])
    assert np.all(got[np.setdiff1d(np.arange(S), loc[good])] == 0xAB)
    pool = gpu(np.where(np.isin(np.arange(S), loc[good])[:, None], got, 0))
    err.zero_()
    k2, v2 = torch.full_like(k, 7), torch.full_like(v, 7)
    ra.ra_kv8_load(pool, i32(loc[good]), k2[:len(good)], v2[:len(good)], device_error=err)
    rk, rv = R.unpack(exp[good], hkv, d)
    assert int(err.item()) == 0
    assert np.array_equal(f64(k2)[:len(good)], rk, equal_nan=True)
    assert np.array_equal(f64(v2)[:len(good)], rv, equal_nan=True)
    assert (k2[len(good):] == 7).all() and (v2[len(good):] == 7).all()


def decode_case(rng, lens, hq, hkv, d, spread=6, share=0):
    """A pool of quantised rows, a table over shuffled slots (the first `share` positions common to all
    requests), queries; records outside the contexts hold NaN codes."""
    lens = np.asarray(lens)
    total = share + int(np.maximum(lens - share, 0).sum())
    S = total + 5
    perm = rng.permutation(S)
    k = rng.normal(size=(S, hkv, d)) * 2.0 ** rng.integers(-spread, spread + 1, (S, hkv, 1)) * 0.3
    v = rng.normal(size=(S, hkv, d)) * 2.0 ** rng.integers(-spread, spread + 1, (S, hkv, 1))
    rec = R.pack(k, v)
    rec[perm[total:]] = 0x7f                                # unused slots: NaN codes, exponent 0
    table = np.full((len(lens) + 2, max(lens.max(), 1) + 3), -1, np.int32)
    rpi = rng.permutation(len(lens) + 2)[:len(lens)]
    at = share
    for b, n in enumerate(lens):
        own = max(n - share, 0)
        table[rpi[b], :n] = np.concatenate([perm[:min(n, share)], perm[at:at + own]])
        at += own
    q = gpu(rng.normal(size=(len(lens), hq, d)).astype(np.float32)).to(BF)
    return rec, table, rpi.astype(np.int32), lens.astype(np.int32), q


def decode(rec, table, rpi, lens, q, hkv, scale, **kw):
    o = torch.full_like(q, 7.0)
    ws = torch.empty(ra.ra_decode_workspace_bytes(len(lens), q.shape[1], hkv, q.shape[2], table.shape[1]),
                     dtype=torch.uint8, device=DEV)
    ra.ra_kv8_decode_attention(gpu(rec), q, o, i32(table), i32(rpi), i32(lens), num_kv_heads=hkv,
                               max_seq_len=kw.pop("max_seq_len", table.shape[1]), sm_scale=scale, workspace=ws, **kw)
    return o


def check_decode(o, rec, table, rpi, lens, q, hkv, scale):
    d = q.shape[2]
    for b, n in enumerate(lens):
        k, v = R.unpack(rec[table[rpi[b], :n]], hkv, d)
        ref, a, x = R.attend(f64(q[b:b + 1]), k, v, scale)
        # f16 weights: 2^-11 relative, or 2^-25 of the largest weight times a code of at most 448
        bound = R.attention_bound(ref, a, x, d, R.EPS_F16)
        p_v = n * 2.0 ** -25 * 448 / 224 * np.abs(v).max() * 2.0
        bad = np.abs(f64(o[b:b + 1]) - ref) > bound + p_v
        assert not bad.any(), (b, n, np.argwhere(bad)[:3], np.abs(f64(o[b:b + 1]) - ref).max())


DECODE = [
    ([1], 8, 2, 64), ([1, 2, 3], 32, 8, 128), ([15, 16, 17, 31, 32, 33], 32, 8, 128), ([129, 128, 127], 64, 8, 128),
    ([1500], 32, 8, 128), ([700, 1, 2049, 64, 333], 16, 16, 128), ([513, 90], 12, 3, 128), ([260, 77], 5, 5, 64),
    ([100, 1000], 40, 20, 64), ([37, 512], 8, 1, 128), ([250], 11, 11, 64), ([640, 3], 24, 12, 128),
    ([1, 63, 64, 65, 1000, 5], 12, 3, 128), ([127, 128, 129, 2500], 32, 4, 128), (list(range(5, 900, 20)), 12, 3, 128),
    (list(range(1, 1300, 29)), 16, 4, 128), (list(range(5, 900, 20)), 4, 2, 128),
]


@pytest.mark.parametrize("lens,hq,hkv,d", DECODE)
def test_decode_matches_64_bit_attention(lens, hq, hkv, d):
    rng = np.random.default_rng(len(lens) * 100 + hq + d)
    rec, table, rpi, lens, q = decode_case(rng, lens, hq, hkv, d, spread=1)
    err = err_word()
    o = decode(rec, table, rpi, lens, q, hkv, d ** -0.5, device_error=err)
    assert int(err.item()) == 0
    check_decode(o, rec, table, rpi, lens, q, hkv, d ** -0.5)


@pytest.mark.parametrize("batch,longest,bound", [(32, 300, None), (33, 300, None), (32, 1500, 1 << 20), (5, 2500, 1 << 20),
                                                 (1, 6000, None), (100, 90, None)])
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (8, 2, 64)])
def test_decode_planned_by_the_warps_and_by_the_kernel(batch, longest, bound, hq, hkv, d):
    """Both sides of the small-call rule (the number of requests; the bound of their keys), the same requests under a loose
    bound, requests of one key among long ones."""
    rng = np.random.default_rng(batch + longest)
    lens = rng.integers(1, longest + 1, batch)
    lens[-1] = 1
    lens[0] = longest
    rec, table, rpi, lens, q = decode_case(rng, lens, hq, hkv, d, spread=1)
    if bound:
        wide = np.full((table.shape[0], bound), -1, np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    err = err_word()
    o = decode(rec, table, rpi, lens, q, hkv, d ** -0.5, device_error=err)
    assert int(err.item()) == 0
    check_decode(o, rec, table, rpi, lens, q, hkv, d ** -0.5)


@pytest.mark.parametrize("batch", [33, 50, 64, 65])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (12, 3, 128), (8, 2, 64), (16, 16, 64)])
def test_decode_of_more_requests_than_lanes(batch, hq, hkv, d):
    """33 to 64 requests (two per lane of a small call) and one more, two of them invalid, split and unsplit ones."""
    rng = np.random.default_rng(batch + hq)
    lens = rng.integers(1, 120, batch)
    lens[[0, 31, 32, batch - 1]] = [500, 90, 431, 333]
    rec, table, rpi, lens, q = decode_case(rng, lens, hq, hkv, d, spread=1)
    r2, l2 = rpi.copy(), lens.copy()
    r2[batch - 2], l2[3] = -1, 0
    err = err_word()
    o = decode(rec, table, r2, l2, q, hkv, d ** -0.5, device_error=err)
    assert int(err.item()) == ra.DEVERR_TABLE | ra.DEVERR_LENGTH
    assert (o[[3, batch - 2]] == 7.0).all()
    ok = np.setdiff1d(np.arange(batch), [3, batch - 2])
    check_decode(o[torch.from_numpy(ok).to(DEV)], rec, table, rpi[ok], lens[ok], q[torch.from_numpy(ok).to(DEV)], hkv,
                 d ** -0.5)


def test_decode_shared_prefix_and_many_splits():
    rng = np.random.default_rng(9)
    rec, table, rpi, lens, q = decode_case(rng, rng.integers(400, 3000, 24), 32, 8, 128, spread=1, share=400)
    o = decode(rec, table, rpi, lens, q, 8, 128 ** -0.5)
    check_decode(o, rec, table, rpi, lens, q, 8, 128 ** -0.5)


@pytest.mark.parametrize("spread", [5, 12])
def test_decode_scales_far_apart(spread):
    """K and V rows whose exponents differ by up to 2 * spread: scores that move both references, weights far
    below the largest V's."""
    rng = np.random.default_rng(spread)
    rec, table, rpi, lens, q = decode_case(rng, [400, 65, 1000], 16, 4, 128, spread=spread)
    o = decode(rec, table, rpi, lens, q, 4, 0.02)
    check_decode(o, rec, table, rpi, lens, q, 4, 0.02)


def test_decode_extreme_scales():
    """All V rows at 2^118 or 2^-105, queries at 2^100 against keys at 2^-100: finite, and within bounds."""
    rng = np.random.default_rng(77)
    hq, hkv, d = 8, 2, 64
    for vs in (2.0 ** 118, 2.0 ** -105):
        n = 200
        k = rng.normal(size=(n, hkv, d)) * 2.0 ** -100
        v = rng.normal(size=(n, hkv, d)) * vs
        rec = R.pack(k, v)
        table = rng.permutation(n)[None].astype(np.int32)
        q = gpu((rng.normal(size=(1, hq, d)) * 2.0 ** 100).astype(np.float32)).to(BF)
        rpi, lens = np.zeros(1, np.int32), np.array([n], np.int32)
        check_decode(decode(rec, table, rpi, lens, q, hkv, 0.125), rec, table, rpi, lens, q, hkv, 0.125)


def test_decode_zero_rows_and_equal_scores():
    """q = 0 gives the mean of the values; zero K and V records count as keys of score 0 and value 0."""
    hq, hkv, d, n = 8, 2, 128, 100
    rng = np.random.default_rng(3)
    v = rng.normal(size=(n, hkv, d))
    v[::2] = 0
    rec = R.pack(np.zeros((n, hkv, d)), v)
    table, rpi, lens = np.arange(n, dtype=np.int32)[None], np.zeros(1, np.int32), np.array([n], np.int32)
    q = torch.zeros(1, hq, d, dtype=BF, device=DEV)
    check_decode(decode(rec, table, rpi, lens, q, hkv, 1.0), rec, table, rpi, lens, q, hkv, 1.0)


def test_decode_nan_stays_in_its_request():
    """A NaN value in one request's context reaches that head's output only; other requests are unaffected."""
    rng = np.random.default_rng(21)
    rec, table, rpi, lens, q = decode_case(rng, [90, 200], 8, 2, 64, spread=1)
    rec[table[rpi[0], 89], 64 + 5] = 0x7f                   # V of head 0, d = 5, of request 0's last key
    o = decode(rec, table, rpi, lens, q, 2, 0.125)
    x = f64(o[0])
    assert np.isnan(x[:4, 5]).all() and np.isfinite(np.delete(x[:4], 5, 1)).all() and np.isfinite(x[4:]).all()
    check_decode(o[1:], rec, table, rpi[1:], lens[1:], q[1:], 2, 0.125)


def test_decode_bad_requests_are_flagged_and_left_alone():
    rng = np.random.default_rng(4)
    rec, table, rpi, lens, q = decode_case(rng, [40, 50, 60, 70], 8, 2, 64, spread=1)
    good = decode(rec, table, rpi, lens, q, 2, 0.125)
    for rp, ln, bit in ((table.shape[0], 50, ra.DEVERR_TABLE), (rpi[1], 0, ra.DEVERR_LENGTH),
                        (rpi[1], -3, ra.DEVERR_LENGTH)):
        r2, l2 = rpi.copy(), lens.copy()
        r2[1], l2[1] = rp, ln
        err = err_word()
        o = decode(rec, table, r2, l2, q, 2, 0.125, device_error=err)
        assert int(err.item()) == bit
        assert torch.equal(o[[0, 2, 3]], good[[0, 2, 3]]) and (o[1] == 7.0).all()
    t2 = table.copy()
    t2[rpi[2], 7] = len(rec)                                # a slot past the pool: read as slot 0
    err = err_word()
    o = decode(rec, t2, rpi, lens, q, 2, 0.125, device_error=err)
    assert int(err.item()) == ra.DEVERR_SLOT and torch.equal(o[[0, 1, 3]], good[[0, 1, 3]])


def test_decode_is_deterministic_and_replays_from_a_graph():
    rng = np.random.default_rng(31)
    rec, table, rpi, lens, q = decode_case(rng, rng.integers(1, 1200, 9), 32, 8, 128, spread=1)
    hkv, n = 8, len(lens)
    pool, tab, rp, ln = gpu(rec), i32(table), i32(rpi), i32(lens)
    o = torch.empty_like(q)
    ws = torch.empty(ra.ra_decode_workspace_bytes(n, 32, hkv, 128, table.shape[1]), dtype=torch.uint8, device=DEV)
    kn, vn = rows(rng, n, hkv, 128, lo=-1, hi=1), rows(rng, n, hkv, 128, lo=-1, hi=1)
    loc = i32([table[r, m - 1] for r, m in zip(rpi, lens)])

    def step():
        ra.ra_kv8_store(pool, kn, vn, loc)
        ra.ra_kv8_decode_attention(pool, q, o, tab, rp, ln, num_kv_heads=hkv, max_seq_len=table.shape[1],
                                   sm_scale=0.09, workspace=ws)
    step()
    first = o.clone()
    step()
    assert torch.equal(o, first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        kn.copy_(rows(rng, n, hkv, 128, lo=-1, hi=1))
        q.copy_(rows(rng, n, 32, 128, lo=-1, hi=1))
        ln.copy_(i32(np.maximum(lens - rng.integers(0, 3, n), 1)))
        g.replay()
        torch.cuda.synchronize()
        got, l2 = o.clone(), ln.cpu().numpy()
        step()
        assert torch.equal(got, o)
    check_decode(got, pool.cpu().numpy(), table, rpi, l2, q, hkv, 0.09)
