"""The extend call's rows of a quantised replay on the CPU: what is read back, and where the call's table finds it."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from prefix_shared_kv_ra_gb300 import serving


@pytest.fixture
def loads(monkeypatch):
    """Calls of ra_kv8_load, each as its slots; row i of k_out is filled with its slot's number."""
    calls = []

    def load(pool, slots, k_out, v_out, device_error=None, stream=None):
        calls.append(slots.numpy().copy())
        k_out.copy_(slots[:, None, None].expand_as(k_out))
        v_out.copy_(-slots[:, None, None].expand_as(v_out))

    monkeypatch.setattr(serving, "ra_kv8_load", load)
    return calls


def replay(num_slots):
    return serving.ServingReplay(num_slots=num_slots, num_q_heads=4, num_kv_heads=2, head_dim=64, max_len=64,
                                 max_running=8, device="cpu", kv_dtype="e4m3", use_graphs=False)


@pytest.mark.parametrize("shared,own", [(40, [3, 1, 7, 2, 5]), (0, [4, 9]), (12, [6])])
def test_a_shared_prefix_is_read_back_once(loads, shared, own):
    rng = np.random.default_rng(shared)
    r = replay(200)
    slots = (1 + rng.permutation(199)).astype(np.int32)
    prefix, at, admitted = slots[:shared], shared, []
    for n in own:
        admitted.append(SimpleNamespace(slots=np.concatenate([prefix, slots[at:at + n]])))
        at += n
    k, v, table, rows = r._extend_pool(admitted, None)
    assert len(loads) == 1
    assert loads[0].size == np.unique(loads[0]).size == shared + sum(own) == k.shape[0] == v.shape[0]
    for i, a in zip(rows.tolist(), admitted):
        at = table[i, :a.slots.size].long()
        assert k[at, 0, 0].tolist() == a.slots.tolist() and v[at, 1, 63].tolist() == (-a.slots).tolist()
    assert table.dtype == torch.int32 and table.shape[1] == max(a.slots.size for a in admitted)
    assert int(table.min()) >= 0 and int(table.max()) < k.shape[0]
