"""Scores with a constant offset: the weights are those without it, and so is the time, also of rows whose keys begin behind the
first columns of a key tile (windows, documents)."""
import numpy as np
import pytest
import torch

import test_gpu_attention_mod as A

pytestmark = pytest.mark.gpu


def shift(c, by):
    """Adds `by` to every score: K's first dimension is 8, q's what that takes (exact in bf16 for heads of 64)."""
    c.k[:, :, 0] = torch.where(c.k[:, :, 0].isnan(), c.k[:, :, 0], torch.full_like(c.k[:, :, 0], 8.0))
    c.q[:, :, 0] = by / c.scale / 8.0


@pytest.mark.parametrize("by", [-300, -100, -64, 100])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=150), dict(window=300, cap=2000.0), dict(doc=57),
                                dict(doc=130, slopes=True), dict(window=77, slopes=True), dict(full=[40, 300], window=90)])
def test_values(by, kw):
    kw = dict(kw)
    c = A.Case(np.random.default_rng(4), [700, 31], [200, 257], 8, 2, 64, **kw)
    shift(c, by)
    c.check(c.extend())
    assert int(c.err) == 0


@pytest.mark.parametrize("kw", [dict(window=500), dict(window=500, cap=2000.0), dict(doc=210)])
def test_time(kw):
    """(Rows computed again key by key took a hundred times as long.)"""
    def us(by):
        c = A.Case(np.random.default_rng(4), [1200] * 6, [300] * 6, 32, 8, 64, **kw)
        shift(c, by)
        import prefix_shared_kv_ra_gb300 as ra
        ws = torch.empty(ra.ra_extend_mod_workspace_bytes(c.B, c.total, c.hq, c.hkv), dtype=torch.uint8, device=A.DEV)
        o = torch.empty_like(c.q)
        args = (c.k, c.v, c.q, o, A.i32(c.table), A.i32(c.rpi), A.i32(c.P), A.i32(c.E), A.i32(c.qo))
        kws = dict(c.kw(), max_extend_len=300, max_prefix_len=1200, workspace=ws)
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ra.ra_extend_attention_mod(*args, **kws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return min(times)

    assert us(-100.0) < 4 * us(0.0)
