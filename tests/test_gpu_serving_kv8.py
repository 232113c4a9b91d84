"""The serving replay over a quantised pool: the same chats admitted, prefilled, decoded from graphs and retired;
slot accounting as over a bf16 pool, and one decode step against 64-bit attention over the records."""
import gc
import weakref

import numpy as np
import pytest
import torch

import kv8_ref as R
from prefix_shared_kv_ra_gb300.serving import ServingReplay, multiturn_chat, run_chat

pytestmark = pytest.mark.gpu


def test_chat_replay_over_a_quantised_pool():
    kw = dict(num_slots=1 << 15, num_q_heads=16, num_kv_heads=4, head_dim=128, max_len=2048, max_running=32,
              device="cuda:0", seed=3, graph_sizes=(8, 16, 32))
    convs = multiturn_chat(10, 2, seed=1, system_prompts=2, system_len=128, user_len=(16, 64), out_len=(4, 10))
    replays = [ServingReplay(kv_dtype=t, **kw) for t in ("bf16", "e4m3")]
    stats = [run_chat(r, convs, max_steps=300, arrivals_per_step=5) for r in replays]
    rp = replays[1]
    torch.cuda.synchronize()
    assert int(rp.err.item()) == 0 and len(rp.finished) == 20 and not rp.running
    for key in ("extend_tokens", "decode_tokens", "cached_tokens", "prompt_tokens", "evicted"):
        assert stats[0][key] == stats[1][key], key
    assert rp.pool.available() + rp.cache.total_tokens() == rp.pool.num_slots - 1
    # admit and prefill more, decode once, and check that step on the device pool's records
    run_chat(rp, multiturn_chat(5, 1, seed=9, system_prompts=2, system_len=96, user_len=(8, 16), out_len=(3, 3)),
             max_steps=2, arrivals_per_step=5, rid0=10_000)
    n = len(rp.prefilled)
    assert n > 0 and int(rp.err.item()) == 0
    g, buf, run = rp._graph(next(s for s in rp.graph_sizes if s >= n))
    torch.cuda.synchronize()
    rows, lens, table = buf["rpi"][:n].cpu().numpy(), buf["lens"][:n].cpu().numpy(), rp.table.cpu().numpy()
    for b in range(n):
        slots = torch.from_numpy(table[rows[b], :lens[b]].astype(np.int64)).to(rp.dev)
        k, v = R.unpack(rp.kv8_pool[slots].cpu().numpy(), 4, 128)
        q, o = (buf[x][b:b + 1].float().cpu().numpy().astype(np.float64) for x in ("q", "o"))
        ref, a, x = R.attend(q, k, v, rp.scale)
        bound = R.attention_bound(ref, a, x, 128, R.EPS_F16) + lens[b] * 2.0 ** -24 * np.abs(v).max()
        assert (np.abs(o - ref) <= bound).all()



@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_replay_and_its_graphs_are_freed_without_the_collector(kv_dtype):
    """A graph destroyed while another is captured invalidates the capture: a replay is in no reference cycle, and
    the collector does not run during its captures (a graph that is garbage in a cycle outlives them)."""
    kw = dict(num_slots=1 << 10, num_q_heads=8, num_kv_heads=2, head_dim=64, max_len=256, max_running=8,
              device="cuda:0", seed=3, graph_sizes=(2, 4, 8), kv_dtype=kv_dtype)
    gc.collect()
    gc.disable()
    try:
        rp = ServingReplay(**kw)
        g = weakref.ref(rp._graph(2)[2])
        whole = weakref.ref(rp)
        del rp
        assert whole() is None and g() is None
    finally:
        gc.enable()
    rp = ServingReplay(**kw)
    cycle = [torch.cuda.CUDAGraph()]
    x = torch.zeros(8, device="cuda:0")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(cycle[0], stream=stream):
        x.add_(1)
    torch.cuda.synchronize()
    cycle.append(cycle)
    before = gc.get_threshold()
    gc.disable()
    try:
        del cycle
        gc.set_threshold(1, 1, 1)
        gc.enable()
        graph, buf, run = rp._graph(4)
    finally:
        gc.set_threshold(*before)
        gc.collect()  # (not during a capture of a later test)
    graph.replay()
    torch.cuda.synchronize()
    assert gc.isenabled() and int(rp.err.item()) == 0
