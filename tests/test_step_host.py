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
