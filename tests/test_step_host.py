"""Refusals of ra_step_slots, ra_tree_verify, ra_tree_verify_greedy and ra_tree_commit on the CPU (nothing is
launched), and the verification's definition itself."""
import ctypes

import numpy as np
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra
import step_ref as R
from prefix_shared_kv_ra_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ra.load()


FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


def _step(lib, **over):
    a = dict(table=FAKE, stride=100, rows=4, rpi=FAKE, lens=FAKE, new=FAKE, batch=3, pages=FAKE, cap=10, count=FAKE, out=FAKE,
             page=16, loc=FAKE, pos=FAKE, n=9, qo=FAKE, seq=FAKE, err=None, stream=None)
    a.update(over)
    return lib.ra_step_slots(*a.values())


def test_step_slots_validation(lib):
    for wrong in (dict(batch=-1), dict(batch=65536), dict(n=-1), dict(n=1 << 31), dict(page=0), dict(page=1 << 21), dict(cap=-1),
                  dict(rows=0), dict(stride=0), dict(table=None), dict(count=None), dict(out=None), dict(qo=None),
                  dict(rpi=None), dict(lens=None), dict(new=None), dict(seq=None), dict(loc=None), dict(pos=None),
                  dict(pages=None), dict(loc=ODD), dict(qo=ODD), dict(pages=ODD), dict(lens=ODD)):
        assert _step(lib, **wrong) == 1, wrong
    assert b"4-byte" in lib.ra_last_error_message()


def _commit(lib, **over):
    a = dict(table=FAKE, stride=100, rows=4, rpi=FAKE, prefix=FAKE, drafts=FAKE, qo=FAKE, batch=3, loc=FAKE, total=9, path=FAKE,
             width=8, acc=FAKE, seq=FAKE, free=FAKE, cap=10, count=FAKE, out=FAKE, err=None, stream=None)
    a.update(over)
    return lib.ra_tree_commit(*a.values())


def test_tree_commit_validation(lib):
    for wrong in (dict(batch=-1), dict(total=-1), dict(cap=-1), dict(rows=0), dict(stride=0), dict(width=0), dict(table=None),
                  dict(rpi=None), dict(prefix=None), dict(drafts=None), dict(qo=None), dict(loc=None), dict(path=None),
                  dict(acc=None), dict(seq=None), dict(free=None), dict(count=None), dict(out=None), dict(path=ODD),
                  dict(free=ODD)):
        assert _commit(lib, **wrong) == 1, wrong
    assert _commit(lib, width=1025) == 2


def _verify(lib, **over):
    a = dict(p=FAKE, ps=100, q=FAKE, qs=100, vocab=100, tok=FAKE, par=FAKE, T=FAKE, qo=FAKE, u=FAKE, uf=FAKE, batch=3, total=9,
             widest=8, path=FAKE, acc=FAKE, nxt=FAKE, err=None, stream=None)
    a.update(over)
    return lib.ra_tree_verify(*a.values())


def _greedy(lib, **over):
    a = dict(x=FAKE, fp32=0, xs=100, vocab=100, tok=FAKE, par=FAKE, T=FAKE, qo=FAKE, batch=3, total=9, widest=8, path=FAKE,
             acc=FAKE, nxt=FAKE, err=None, stream=None)
    a.update(over)
    return lib.ra_tree_verify_greedy(*a.values())


def test_verify_validation(lib):
    common = (dict(batch=-1), dict(batch=65536), dict(total=-1), dict(vocab=0), dict(vocab=(1 << 28) + 1), dict(widest=0),
              dict(tok=None), dict(par=None), dict(T=None), dict(qo=None), dict(path=None), dict(acc=None), dict(nxt=None),
              dict(tok=ODD), dict(path=ODD))
    for wrong in common + (dict(ps=99), dict(qs=99), dict(p=None), dict(u=None), dict(uf=None), dict(p=ODD), dict(q=ODD)):
        assert _verify(lib, **wrong) == 1, wrong
    for wrong in common + (dict(xs=99), dict(x=None), dict(fp32=2), dict(x=ctypes.c_void_p((1 << 20) + 1)),
                           dict(x=ODD, fp32=1)):
        assert _greedy(lib, **wrong) == 1, wrong
    assert _verify(lib, widest=1025) == 2 and _greedy(lib, widest=1025) == 2
    assert _verify(lib, batch=0, p=None, q=None) == 0 and _greedy(lib, batch=0, x=None) == 0


I = torch.int32


def test_bindings_check_before_the_call():
    i = lambda *s: torch.zeros(*s, dtype=I)
    p = torch.zeros(9, 50)
    tree = (i(9), i(9), i(3), i(4))
    out = (i(3, 8), i(3), i(3))
    good = [p, p.clone(), *tree, torch.zeros(9), torch.zeros(3), *out]

    def verify(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        ra.ra_tree_verify(*a, max_draft_len=8)

    with pytest.raises(ValueError, match="CUDA"):
        verify()
    for wrong in (dict(a1=torch.zeros(9, 51)), dict(a2=i(8)), dict(a3=i(10)), dict(a5=i(3)), dict(a6=torch.zeros(8)),
                  dict(a7=torch.zeros(4)), dict(a8=i(3, 7)), dict(a9=i(2)), dict(a0=torch.zeros(50, 9).t()),
                  dict(a0=torch.zeros(1, 50).expand(9, 50)), dict(a0=torch.zeros(50))):
        with pytest.raises(ValueError):
            verify(**wrong)
    for wrong in (dict(a0=p.double(), a1=None), dict(a1=p.half()), dict(a2=torch.zeros(9)), dict(a6=i(9)),
                  dict(a9=torch.zeros(3))):
        with pytest.raises(TypeError):
            verify(**wrong)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_tree_verify_greedy(p.bfloat16(), *tree, *out, max_draft_len=8)
    with pytest.raises(TypeError):
        ra.ra_tree_verify_greedy(p.half(), *tree, *out, max_draft_len=8)
    with pytest.raises(ValueError, match="32 bits"):
        ra.ra_tree_verify_greedy(p, *tree, *out, max_draft_len=1 << 40)
    step = [i(4, 30), i(3), i(3), i(3), i(10), i(1), i(9), i(9), i(4), i(3)]
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_step_slots(*step)
    for k, bad in ((2, i(2)), (3, i(4)), (5, i(2)), (7, i(8)), (8, i(3)), (9, i(4)), (0, i(30))):
        with pytest.raises(ValueError):
            ra.ra_step_slots(*[bad if j == k else x for j, x in enumerate(step)])
    with pytest.raises(TypeError):
        ra.ra_step_slots(*[x.long() if j == 4 else x for j, x in enumerate(step)])
    done = [i(4, 30), i(3), i(3), i(3), i(4), i(9), i(3, 8), i(3), i(3), i(10), i(1)]
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_tree_commit(*done)
    for k, bad in ((2, i(2)), (4, i(3)), (6, i(2, 8)), (7, i(4)), (8, i(2)), (10, i(3))):
        with pytest.raises(ValueError):
            ra.ra_tree_commit(*[bad if j == k else x for j, x in enumerate(done)])


def test_the_definition_keeps_the_targets_distribution():
    """By enumeration: over all draws of two drafts from q and a fine grid of numbers, what comes out first has the
    distribution p, by the definition the kernels are tested against."""
    p, q = np.array([[0.5, 0.125, 0.25, 0.125]] * 3), np.array([[0.125, 0.25, 0.25, 0.375]] * 3)
    out = np.zeros(4)
    n = 32
    grid = (np.arange(n) + 0.5) / n
    for x in range(4):
        for y in range(4):
            for u in grid:
                for v in grid:
                    # the draw integrated over its number: its residual's distribution
                    path, _ = R.verify(p, q, [0, x, y], [-1, 0, 0], 3, 0, [0, u, v], 0.0)
                    weight = q[0, x] * q[0, y] / n ** 2
                    if len(path) > 1:
                        out[x if path[1] == 1 else y] += weight
                    else:
                        r = np.maximum(p[0] - q[0], 0)
                        r = np.maximum(r - r.sum() * q[0], 0)
                        out += weight * r / r.sum()
    assert np.abs(out - p[0]).max() < 1.5 / n, out


def _extend_mod(lib, **over):
    a = dict(k=FAKE, v=FAKE, S=1024, hkv=8, d=128, q=FAKE, o=FAKE, hq=32, scale=0.088, cap=30.0, window=100, slopes=FAKE,
             first=FAKE, full=FAKE, table=FAKE, stride=4096, rows=64, rpi=FAKE, plen=FAKE, elen=FAKE, qo=FAKE, batch=4,
             total=100, max_e=40, max_p=4000, ws=FAKE, wsb=1 << 30, err=None, stream=None)
    a.update(over)
    return lib.ra_extend_attention_mod(*a.values())


def _decode_mod(lib, **over):
    a = dict(k=FAKE, v=FAKE, S=1024, hkv=8, d=128, q=FAKE, o=FAKE, hq=32, scale=0.088, cap=30.0, window=100, slopes=FAKE,
             first=FAKE, table=FAKE, stride=4096, rows=64, rpi=FAKE, lens=FAKE, batch=4, longest=4096, ws=FAKE, wsb=1 << 30,
             err=None, stream=None)
    a.update(over)
    return lib.ra_decode_attention_mod(*a.values())


def test_attention_mod_validation(lib):
    nan, inf = float("nan"), float("inf")
    for call in (_extend_mod, _decode_mod):
        for wrong in (dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(cap=1e-7), dict(cap=2e12), dict(window=-1),
                      dict(scale=0.0), dict(scale=nan), dict(scale=3e38, cap=1e-3), dict(slopes=ODD), dict(first=ODD),
                      dict(hq=30), dict(S=0), dict(batch=-1), dict(k=None), dict(q=ODD), dict(table=None), dict(rows=0),
                      dict(stride=39), dict(ws=ctypes.c_void_p((1 << 20) + 8))):
            assert call(lib, **wrong) == 1, (call, wrong)
        assert call(lib, d=96) == 2
        assert call(lib, wsb=15) == 3
        assert call(lib, batch=0, k=None) == 0
    assert _extend_mod(lib, hq=24) == 2                     # group 3 does not divide 128
    assert _decode_mod(lib, hq=128) == 2                    # groups of up to 8
    assert _extend_mod(lib, total=0, k=None) == 0
    need = ra.ra_extend_mod_workspace_bytes(4, 100, 32, 8)
    assert _extend_mod(lib, wsb=need - 1) == 3 and ra.ra_extend_mod_workspace_bytes(4, 100, 30, 8) == 0
    assert ra.ra_extend_mod_workspace_bytes(4, 100, 24, 8) == 0


def test_attention_mod_bindings_check_before_the_call():
    bf = torch.bfloat16
    i = lambda *s: torch.zeros(*s, dtype=I)
    pool, q = torch.zeros(16, 2, 64, dtype=bf), torch.zeros(5, 8, 64, dtype=bf)
    kw = dict(sm_scale=1.0, workspace=torch.zeros(64, dtype=torch.uint8))
    ext = dict(kw, max_extend_len=3, max_prefix_len=4)
    args = [pool, pool, q, q.clone(), i(2, 9), i(2), i(2), i(2), i(3)]
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_extend_attention_mod(*args, **ext)
    for bad in (dict(slopes=torch.zeros(7)), dict(first_key=i(4)), dict(full_lens=i(3)), dict(window=1 << 40)):
        with pytest.raises(ValueError):
            ra.ra_extend_attention_mod(*args, **dict(ext, **bad))
    for bad in (dict(slopes=torch.zeros(8, dtype=bf)), dict(first_key=torch.zeros(5)), dict(full_lens=i(2).long())):
        with pytest.raises(TypeError):
            ra.ra_extend_attention_mod(*args, **dict(ext, **bad))
    for k, x in ((1, pool[:8]), (3, q[:4]), (6, i(3)), (7, i(1)), (8, i(2)), (4, i(9))):
        with pytest.raises(ValueError):
            ra.ra_extend_attention_mod(*[x if j == k else y for j, y in enumerate(args)], **ext)
    dec = dict(kw, max_seq_len=9)
    one = [pool, pool, q[:2], q[:2].clone(), i(2, 9), i(2), i(2)]
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_decode_attention_mod(*one, **dec)
    for bad in (dict(slopes=torch.zeros(7)), dict(first_key=i(5))):
        with pytest.raises(ValueError):
            ra.ra_decode_attention_mod(*one, **dict(dec, **bad))
    with pytest.raises(ValueError):
        ra.ra_decode_attention_mod(pool, pool, q, q.clone(), i(2, 9), i(2), i(2), **dec)
