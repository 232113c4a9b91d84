"""The serving replay with its slot maps made on the GPU (ra_step_slots, in the captured decode step too): the same slots,
tables, caches and outputs as with the host's."""
import pytest
import torch

from prefix_shared_kv_ra_gb300.serving import ServingReplay, multiturn_chat, run_chat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_dtype,use_graphs", [("bf16", True), ("bf16", False), ("e4m3", True)])
def test_replays_agree(kv_dtype, use_graphs):
    replays = []
    for device_slots in (False, True):
        rp = ServingReplay(num_slots=1 << 12, num_q_heads=8, num_kv_heads=2, head_dim=64, max_len=512, max_running=16,
                           device="cuda:0", seed=5, graph_sizes=(4, 8, 16), use_graphs=use_graphs, kv_dtype=kv_dtype,
                           device_slots=device_slots)
        convs = multiturn_chat(10, 3, seed=2, system_prompts=2, system_len=64, user_len=(4, 24), out_len=(2, 9))
        st = run_chat(rp, convs, max_steps=200, arrivals_per_step=3)
        torch.cuda.synchronize()
        assert int(rp.err.item()) == 0 and len(rp.finished) == 30 and not rp.running
        replays.append((rp, st))
    (a, sa), (b, sb) = replays
    assert sa["decode_tokens"] == sb["decode_tokens"] and sa["evicted"] == sb["evicted"] and sa["hit_ratio"] == sb["hit_ratio"]
    assert [r.rid for r in a.finished] == [r.rid for r in b.finished]
    for x, y in zip(a.finished, b.finished):
        assert (x.slots == y.slots).all()
    assert torch.equal(a.table, b.table)
    if kv_dtype == "bf16":
        assert torch.equal(a.k_pool[1:], b.k_pool[1:]) and torch.equal(a.v_pool[1:], b.v_pool[1:])  # (slot 0: padding rows)
    else:
        assert torch.equal(a.kv8_pool[1:], b.kv8_pool[1:])
    assert sorted(a._graphs) == sorted(b._graphs)
    for size, (_, buf, _) in a._graphs.items():
        other = b._graphs[size][1]
        # (padding rows attend to slot 0, which they all write)
        live = buf["rpi"] != a.pad_row
        assert torch.equal(buf["rpi"], other["rpi"]) and torch.equal(buf["lens"], other["lens"])
        assert torch.equal(buf["loc"], other["loc"]) and torch.equal(buf["o"][live], other["o"][live])
