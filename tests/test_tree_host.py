"""ra_tree_attention's refusals and workspace size on the CPU (nothing is launched)."""
import ctypes

import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
from prefix_shared_kv_ra_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ra.load()


FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


def _tree(lib, **over):
    a = dict(k=FAKE, v=FAKE, S=1024, hkv=8, d=128, q=FAKE, o=FAKE, hq=32, scale=0.088, table=FAKE, stride=4096, rows=64,
             rpi=FAKE, plen=FAKE, dlen=FAKE, qo=FAKE, mask=FAKE, words=2, batch=4, total_q=100, max_d=40, max_p=4000,
             ws=FAKE, wsb=1 << 40, err=None, stream=None)
    a.update(over)
    return lib.ra_tree_attention(*a.values())


def test_tree_validation(lib):
    need = ra.ra_tree_workspace_bytes(4, 100, 32, 8, 128, 40)
    assert need > 0
    assert _tree(lib, wsb=need - 1) == 3 and b"workspace" in lib.ra_last_error_message()
    assert _tree(lib, ws=None, wsb=need) == 3
    assert _tree(lib, ws=ODD) == 1
    assert _tree(lib, batch=0, ws=None, wsb=0) == 0
    assert _tree(lib, total_q=0, ws=None, wsb=0) == 0
    assert _tree(lib, batch=-1) == 1
    assert _tree(lib, hq=30) == 1
    assert _tree(lib, hq=24) == 2            # group 3 does not divide 128
    assert _tree(lib, d=96) == 2
    assert _tree(lib, scale=0.0) == 1
    assert _tree(lib, max_d=0) == 1
    assert _tree(lib, max_d=1025, words=40) == 2
    assert _tree(lib, max_d=65) == 1         # 65 drafted tokens in 64 mask bits
    assert _tree(lib, max_p=-1) == 1
    assert _tree(lib, max_p=5000) == 1       # table narrower than the prefix bound
    assert _tree(lib, mask=None) == 1
    assert _tree(lib, q=ODD) == 1
    assert _tree(lib, mask=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert _tree(lib, rows=0) == 1


def test_tree_workspace_is_bounded(lib):
    small = ra.ra_tree_workspace_bytes(4, 32, 32, 8, 128, 8)
    wide = ra.ra_tree_workspace_bytes(4, 256, 32, 8, 128, 64)
    assert 0 < small < wide < 100 << 20                    # 608 partial tiles of at most 256 rows
    assert ra.ra_tree_workspace_bytes(64, 4096, 32, 8, 128, 64, max_prefix_len=1 << 20) < 100 << 20
    assert ra.ra_tree_workspace_bytes(4, 32, 30, 8, 128, 8) == 0
    assert ra.ra_tree_workspace_bytes(4, 32, 32, 8, 128, 0) == 0


def test_tree_binding_checks_before_the_call():
    bf, i = torch.bfloat16, torch.int32
    pool = torch.zeros(16, 2, 64, dtype=bf)
    q = torch.zeros(5, 8, 64, dtype=bf)
    table, b2, qo, mask = torch.zeros(2, 9, dtype=i), torch.zeros(2, dtype=i), torch.zeros(3, dtype=i), \
        torch.zeros(5, 1, dtype=i)
    kw = dict(max_draft_len=3, max_prefix_len=4, sm_scale=1.0, workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ra.ra_tree_attention(pool, pool, q, q, table, b2, b2, b2, qo[:2], mask, **kw)
    with pytest.raises(ValueError):
        ra.ra_tree_attention(pool, pool, q, q, table, b2, b2, b2, qo, mask[:4], **kw)
    with pytest.raises(ValueError):
        ra.ra_tree_attention(pool, pool[:8], q, q, table, b2, b2, b2, qo, mask, **kw)
    with pytest.raises(TypeError):
        ra.ra_tree_attention(pool, pool, q, q, table, b2, b2, b2, qo, mask.long(), **kw)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_tree_attention(pool, pool, q, q.clone(), table, b2, b2, b2, qo, mask, **kw)
