"""Tensors on the CPU are refused by every call, with the same error."""
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
from prefix_shared_kv_ra_gb300 import _build

BF, I = torch.bfloat16, torch.int32


def calls():
    pool, q = torch.zeros(8, 2, 64, dtype=BF), torch.zeros(3, 4, 64, dtype=BF)
    new, idx, table = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, dtype=I), torch.zeros(3, 8, dtype=I)
    ws, kv8 = torch.zeros(64, dtype=torch.uint8), torch.zeros(8, ra.ra_kv8_slot_bytes(2, 64), dtype=torch.uint8)
    one = dict(max_seq_len=8, sm_scale=1.0, workspace=ws)
    qo, cs = torch.zeros(4, dtype=I), torch.zeros(8, 64)
    return {
        "kv_store": lambda: ra.ra_kv_store(pool, pool, new, new, idx),
        "extend": lambda: ra.ra_extend_attention(pool, pool, q, q.clone(), table, idx, idx, idx, qo, max_extend_len=1,
                                                 max_prefix_len=4, sm_scale=1.0, workspace=ws),
        "decode": lambda: ra.ra_decode_attention(pool, pool, q, q.clone(), table, idx, idx, **one),
        "decode_store": lambda: ra.ra_decode_attention_store(pool, pool, new, new, idx, q, q.clone(), table, idx, idx, **one),
        "selftest": lambda: ra.ra_selftest_bounded_wait(10, idx[:1]),
        "kv8_store": lambda: ra.ra_kv8_store(kv8, new, new, idx),
        "kv8_decode": lambda: ra.ra_kv8_decode_attention(kv8, q, q.clone(), table, idx, idx, num_kv_heads=2, **one),
        "norm_rope": lambda: ra.ra_qk_norm_rope_store(q, new, new, None, None, idx, cs, q, pool, pool, idx),
        "tree": lambda: ra.ra_tree_attention(pool, pool, q, q.clone(), table, idx, idx, idx, qo, torch.zeros(3, 1, dtype=I),
                                             max_draft_len=1, max_prefix_len=4, sm_scale=1.0, workspace=ws),
    }


@pytest.mark.parametrize("name", ["kv_store", "extend", "decode", "decode_store", "selftest", "kv8_store", "kv8_decode",
                                  "norm_rope", "tree"])
def test_cpu_tensors_are_refused(name):
    _build.build()
    with pytest.raises(ValueError, match="CUDA tensors"):
        calls()[name]()
