"""ra_step_slots with as many tokens as its arrays may hold, 2^31 - 1, in two rounds of requests: the last run of four tokens
begins at the last token, so its end is behind 2^31."""
import pytest
import torch

import prefix_shared_kv_ra_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_the_last_tokens_of_2_to_the_31():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    B, page, n = 514, 1 << 20, (1 << 31) - 1
    lens = torch.full((B,), n // B, dtype=torch.int64)
    lens[0] += n - int(lens.sum())
    # the second round's first token is at 2 mod 4, as is the last token
    lens[0] += (2 - int(lens[:512].sum())) % 4
    lens[B - 1] -= int(lens.sum()) - n
    assert int(lens.sum()) == n and int(lens[:512].sum()) % 4 == 2 and (n - 1) % 4 == 2
    width = int(lens.max())
    new = lens.int().to(DEV)
    # table rows 1 .. B between two that stay
    table = torch.full((B + 2, width), -1, dtype=torch.int32, device=DEV)
    need = int(((lens + page - 1) // page).sum())
    free = torch.arange(need, device=DEV, dtype=torch.int32).remainder(1900) + 1   # (slots of 2,000 pages fit 32 bits)
    count = torch.full((1,), need, dtype=torch.int32, device=DEV)
    loc, positions = (torch.full((n,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    qo, seq = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (B + 1, B))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ra.ra_step_slots(table, torch.arange(1, B + 1, dtype=torch.int32, device=DEV), torch.zeros_like(new), new, free, count,
                     loc, positions, qo, seq, page_size=page, device_error=err)
    assert int(err) == 0 and int(count) == 0 and torch.equal(seq, new)
    ends = lens.cumsum(0)
    assert torch.equal(qo.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.int64), ends]))
    assert (table[0] == -1).all() and (table[B + 1] == -1).all()
    first = torch.cat([torch.zeros(1, dtype=torch.int64), ((lens + page - 1) // page).cumsum(0)])
    for b in (0, 1, 510, 511, 512, B - 1):
        m, q0 = int(lens[b]), int(qo[b])
        at = torch.arange(m, device=DEV)
        nth = int(first[b]) + at // page
        want = (free[need - 1 - nth].long() * page + at % page).int()
        assert torch.equal(positions[q0:q0 + m], at.int()) and torch.equal(loc[q0:q0 + m], want)
        assert torch.equal(table[b + 1, :m], want) and (table[b + 1, m:] == -1).all()
