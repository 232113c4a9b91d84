"""Quantised pools and the norm + rotation + store call on the CPU: the record layout, the reference itself
and every refusal that needs no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_ref as R
import prefix_shared_kv_ra_gb300 as ra
from prefix_shared_kv_ra_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ra.load()


FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)


def test_slot_bytes_follow_the_layout(lib):
    for hkv in (1, 2, 3, 5, 7, 8, 11, 12, 16, 20, 32, 40):
        for d in (64, 128):
            assert ra.ra_kv8_slot_bytes(hkv, d) == R.slot_bytes(hkv, d)
    assert ra.ra_kv8_slot_bytes(8, 128) == 2080
    for hkv, d in ((0, 128), (8, 96), (2048, 64)):
        assert lib.ra_kv8_slot_bytes(hkv, d) == 0
        with pytest.raises(ra.RAError):
            ra.ra_kv8_slot_bytes(hkv, d)


def test_reference_codes_agree_with_torch():
    """The reference's rounding is torch's e4m3 cast within range, and pack / unpack invert each other."""
    x = np.concatenate([np.linspace(-448, 448, 20001), R.CODES[~np.isnan(R.CODES)],
                        (R._POS[1:] + R._POS[:-1]) / 2]).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x.astype(np.float64)), got)
    rng = np.random.default_rng(0)
    k = rng.normal(size=(3, 12, 64)) * 2.0 ** rng.integers(-20, 20, (3, 12, 1))
    k[0, 0] = 0
    kk, vv = R.unpack(R.pack(k, -k), 12, 64)
    e = R.row_exponent(k)[..., None]
    assert np.all(np.abs(kk - k) <= np.maximum(2.0 ** -4 * np.abs(k), 2.0 ** -10 * 2.0 ** e))
    assert np.array_equal(kk, -vv)
    k2, _ = R.unpack(R.pack(kk, vv), 12, 64)
    assert np.array_equal(k2, kk)


def test_kv8_store_and_load_validation(lib):
    for f, args in ((lib.ra_kv8_store, lambda p, k, v, s: (p, 16, 8, 128, k, v, s)),
                    (lib.ra_kv8_load, lambda p, k, v, s: (p, 16, 8, 128, s, k, v))):
        ok = args(FAKE, FAKE, FAKE, FAKE)
        assert f(*ok, 0, None, None) == 0                                   # no tokens: no-op
        assert f(*ok, -1, None, None) == 1
        assert f(*args(None, FAKE, FAKE, FAKE), 3, None, None) == 1
        assert f(*args(FAKE, FAKE, None, FAKE), 3, None, None) == 1
        assert f(*args(ODD, FAKE, FAKE, FAKE), 3, None, None) == 1
        assert f(*args(FAKE, ODD, FAKE, FAKE), 3, None, None) == 1
        assert f(*args(FAKE, FAKE, FAKE, ctypes.c_void_p((1 << 20) + 2)), 3, None, None) == 1
        assert f(ok[0], 0, *ok[2:], 3, None, None) == 1                     # no slots
        assert f(ok[0], 16, 8, 96, *ok[4:], 3, None, None) == 2             # head_dim
        assert f(ok[0], 16, 0, 128, *ok[4:], 3, None, None) == 1
    assert b"num_kv_heads" in lib.ra_last_error_message()


def _decode(lib, **over):
    a = dict(pool=FAKE, S=1024, hkv=8, d=128, q=FAKE, o=FAKE, hq=32, scale=0.088, table=FAKE, stride=4096, rows=64,
             rpi=FAKE, lens=FAKE, batch=4, max_len=4096, ws=FAKE, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lib.ra_kv8_decode_attention(*a.values())


def test_kv8_decode_validation(lib):
    assert _decode(lib, batch=0) == 0
    assert _decode(lib, batch=-1) == 1
    assert _decode(lib, hq=30) == 1
    assert _decode(lib, hq=128) == 2                # group 16
    assert _decode(lib, d=96) == 2
    assert _decode(lib, scale=float("inf")) == 1
    assert _decode(lib, scale=0.0) == 1
    assert _decode(lib, max_len=0) == 1
    assert _decode(lib, stride=100) == 1
    assert _decode(lib, rows=0) == 1
    assert _decode(lib, pool=None) == 1
    assert _decode(lib, q=ODD) == 1
    assert _decode(lib, wsb=16) == 3
    assert _decode(lib, ws=ODD) == 1
    assert _decode(lib, wsb=ra.ra_decode_workspace_bytes(4, 32, 8, 128, 4096) - 1) == 3


def _rope(lib, kv8=False, **over):
    a = dict(q=FAKE, qs=6144, k=FAKE, ks=6144, v=FAKE, vs=6144, hq=32, hkv=8, d=128, qw=FAKE, kw=FAKE, eps=1e-6,
             pos=FAKE, cs=FAKE, maxp=4096, rot=128, inter=0, qo=FAKE, qos=4096)
    a.update(pool=FAKE, S=64, loc=FAKE, n=3, err=None, stream=None) if kv8 else \
        a.update(kp=FAKE, vp=FAKE, S=64, loc=FAKE, n=3, err=None, stream=None)
    a.update(over)
    return (lib.ra_qk_norm_rope_kv8_store if kv8 else lib.ra_qk_norm_rope_store)(*a.values())


@pytest.mark.parametrize("kv8", [False, True])
def test_norm_rope_validation(lib, kv8):
    assert _rope(lib, kv8, n=0) == 0
    assert _rope(lib, kv8, n=-1) == 1
    assert _rope(lib, kv8, d=96) == 2
    assert _rope(lib, kv8, hkv=0) == 1
    assert _rope(lib, kv8, rot=0) == 2
    assert _rope(lib, kv8, rot=24) == 2
    assert _rope(lib, kv8, rot=144) == 1
    assert _rope(lib, kv8, eps=-1.0) == 1
    assert _rope(lib, kv8, eps=float("nan")) == 1
    assert _rope(lib, kv8, maxp=0) == 1
    assert _rope(lib, kv8, qw=None) == 1             # weights go together
    assert _rope(lib, kv8, inter=2) == 1
    assert _rope(lib, kv8, pos=None) == 1
    assert _rope(lib, kv8, qs=4088) == 1             # narrower than a token
    assert _rope(lib, kv8, ks=6146) == 1             # not a multiple of 16 bytes
    assert _rope(lib, kv8, q=ODD) == 1
    assert _rope(lib, kv8, cs=ODD) == 1
    assert _rope(lib, kv8, loc=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert _rope(lib, kv8, **({"pool": None} if kv8 else {"vp": None})) == 1


def test_bindings_check_before_the_call():
    """Shapes, types and devices are checked in Python (CPU tensors: nothing reaches a GPU)."""
    bf = torch.bfloat16
    pool = torch.zeros(16, ra.ra_kv8_slot_bytes(2, 64), dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=bf)
    idx = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ra.ra_kv8_store(pool, k, k[:2], idx)
    with pytest.raises(ValueError):
        ra.ra_kv8_store(pool[:, :-16].contiguous(), k, k, idx)
    with pytest.raises(ValueError):
        ra.ra_kv8_store(pool[:, :256], k, k, idx)
    with pytest.raises(TypeError):
        ra.ra_kv8_load(pool, idx.long(), k, k)
    with pytest.raises(TypeError):
        ra.ra_kv8_load(pool, idx, k.float(), k.float())
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_kv8_load(pool, idx, k, k.clone())
    q = torch.zeros(3, 8, 64, dtype=bf)
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ra.ra_kv8_decode_attention(pool, q, q, idx[None], idx[:2], idx, num_kv_heads=2, max_seq_len=3, sm_scale=1.0,
                                   workspace=ws)
    kp = torch.zeros(16, 2, 64, dtype=bf)
    cs = torch.zeros(32, 64)
    w = torch.ones(64, dtype=bf)
    args = dict(device_error=None)
    with pytest.raises(ValueError):                       # heads of k and the pool differ
        ra.ra_qk_norm_rope_store(q, k[:, :1], k[:, :1], w, w, idx, cs, q, kp, kp, idx, **args)
    with pytest.raises(ValueError):                       # a row of heads that is not contiguous
        ra.ra_qk_norm_rope_store(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, w, w, idx, cs, q, kp, kp, idx)
    with pytest.raises(TypeError):
        ra.ra_qk_norm_rope_store(q, k, k, w.float(), w, idx, cs, q, kp, kp, idx)
    with pytest.raises(TypeError):
        ra.ra_qk_norm_rope_kv8_store(q, k, k, w, w, idx, cs.double(), q, pool, idx)
    with pytest.raises(ValueError):
        ra.ra_qk_norm_rope_kv8_store(q, k, k, w[:32], w, idx, cs, q, pool, idx)


def test_replay_refuses_an_unknown_cache_type():
    from prefix_shared_kv_ra_gb300.serving import ServingReplay
    with pytest.raises(ValueError):
        ServingReplay(num_slots=64, num_q_heads=2, num_kv_heads=1, head_dim=64, max_len=8, max_running=1,
                      device="cuda:0", kv_dtype="int8")


def test_bindings_take_tensors_only():
    t = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(16, ra.ra_kv8_slot_bytes(2, 64), dtype=torch.uint8)
    for bad in (None, 3, [1, 2], np.zeros(3, np.int32)):
        with pytest.raises(TypeError):
            ra.ra_kv8_store(pool, t, t, bad)
