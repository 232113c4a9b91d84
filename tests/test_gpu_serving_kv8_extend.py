"""The extend calls of a replay over a quantised pool against 64-bit attention over the pool's records: suffixes behind
cached prefixes that the step's requests share, read back into rows of the step."""
import numpy as np
import pytest
import torch

import kv8_ref as R
from prefix_shared_kv_ra_gb300 import serving

pytestmark = pytest.mark.gpu


def test_extend_over_a_quantised_pool(monkeypatch):
    hq, hkv, d = 16, 4, 128
    rp = serving.ServingReplay(num_slots=1 << 11, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, max_len=512,
                               max_running=16, device="cuda:0", seed=5, use_graphs=False, kv_dtype="e4m3")
    calls = []
    extend = serving.ra_extend_attention

    def spy(k, v, q, o, table, rows, pre, ext, indptr, **kw):
        extend(k, v, q, o, table, rows, pre, ext, indptr, **kw)
        calls.append((k.shape[0], q, o, pre, ext, indptr))

    monkeypatch.setattr(serving, "ra_extend_attention", spy)
    rng = np.random.default_rng(0)
    system = rng.integers(1, 1 << 20, 130, dtype=np.int32)

    def prompt(n):
        return np.concatenate([system, rng.integers(1, 1 << 20, n, dtype=np.int32)])

    rp.step([(0, prompt(7), 1)])                            # then decoded and retired: the system prompt is cached
    rp.step([])
    assert len(rp.finished) == 1
    suffixes = [20, 1, 64, 5]
    rp.step([(10 + i, prompt(n), 3) for i, n in enumerate(suffixes)])
    torch.cuda.synchronize()
    assert int(rp.err.item()) == 0
    rows, q, o, pre, ext, indptr = calls[-1]
    assert rows == 130 + sum(suffixes) and pre.tolist() == [130] * 4 and ext.tolist() == suffixes
    for i, n in enumerate(suffixes):
        slots = torch.from_numpy(rp.running[10 + i].slots[:130 + n].astype(np.int64)).to(rp.dev)
        k, v = R.unpack(rp.kv8_pool[slots].cpu().numpy(), hkv, d)
        a0 = int(indptr[i])
        qi, oi = (t[a0:a0 + n].float().cpu().numpy().astype(np.float64) for t in (q, o))
        seen = np.arange(130 + n)[None, :] <= 130 + np.arange(n)[:, None]
        ref, a, x = R.attend(qi, k, v, rp.scale, seen)
        assert (np.abs(oi - ref) <= R.attention_bound(ref, a, x, d, R.EPS_BF16)).all()
