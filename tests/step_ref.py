"""The step's bookkeeping and the verification of drafted trees by their definitions, in Python and 64 bits."""
import numpy as np


def step_slots(table, rpi, cur, new, free, count, page, n):
    """(table, loc, positions, qo, seq, left) of requests that all fit."""
    table = table.copy()
    loc, pos, qo = np.zeros(n, np.int64), np.zeros(n, np.int64), [0]
    left, t = int(count), 0
    for r, c, m in zip(rpi, cur, new):
        for p in range(c, c + m):
            if p % page == 0:
                left -= 1
                slot = free[left] * page
            else:
                slot = table[r, p - 1] + 1
            table[r, p] = slot
            loc[t], pos[t] = slot, p
            t += 1
        qo.append(t)
    return table, loc, pos, np.array(qo), np.asarray(cur) + np.asarray(new), left


def commit(table, rpi, prefix, drafts, qo, loc, path, accepted, free, count):
    table, free, left = table.copy(), free.copy(), int(count)
    for b, r in enumerate(rpi):
        P, T, n, q0 = prefix[b], drafts[b], accepted[b], qo[b]
        kept = list(path[b, :n])
        table[r, P:P + T] = [loc[q0 + i] for i in kept] + [-1] * (T - n)
        for i in range(T):
            if i not in kept:
                free[left] = loc[q0 + i]
                left += 1
    return table, free, left, np.asarray(prefix) + np.asarray(accepted)


def verify(target, draft, tokens, parents, T, q0, u, u_final):
    """(path, next token) of one tree; rows in 64 bits; draft None: drafts taken as given."""
    path, vocab = [0], target.shape[1]
    while True:
        node = path[-1]
        p = np.maximum(np.nan_to_num(target[q0 + node].astype(np.float64), nan=0.0, posinf=np.inf), 0.0)
        r, mass, went = p.copy(), 1.0, False
        for i in range(node + 1, T):
            if parents[q0 + i] != node:
                continue
            x = tokens[q0 + i]
            known = 0 <= x < vocab
            rx = r[x] if known else 0.0
            qx = 1.0 if draft is None else (float(draft[q0 + node, x]) if known else 0.0)
            if float(u[q0 + i]) * qx * mass < rx:
                path.append(i)
                went = True
                break
            if draft is None:
                mass -= rx
                if known:
                    r[x] = 0
            else:
                r = np.maximum(r - mass * draft[q0 + node].astype(np.float64), 0.0)
                mass = r.sum()
        if went:
            continue
        if not r.sum() > 0:
            r = p
        c = np.cumsum(r)
        if not (c[-1] > 0 and np.isfinite(c[-1])):
            return path, 0
        over = np.flatnonzero(c > float(u_final) * c[-1])
        return path, int(over[0]) if over.size else int(np.flatnonzero(r > 0)[-1])


def greedy(logits, tokens, parents, T, q0):
    path = [0]
    while True:
        row = logits[q0 + path[-1]].astype(np.float64)
        if np.isnan(row).all():
            return path, 0
        top = int(np.flatnonzero(row == np.nanmax(row))[0])
        kids = [i for i in range(path[-1] + 1, T) if parents[q0 + i] == path[-1] and tokens[q0 + i] == top]
        if not kids:
            return path, top
        path.append(kids[0])


def tree(rng, T):
    """Parents of T nodes: -1, then an earlier node (mostly the one before)."""
    return np.array([-1] + [i - 1 if rng.random() < 0.5 else int(rng.integers(0, i)) for i in range(1, T)])
