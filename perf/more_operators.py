"""Measured cases of the operators that change a step's attention scores and that keep its bookkeeping on the GPU.

Four operators, each in a plain form (elementary torch operations, `own` false) and as the calls a user
makes of this package (`own` true):

* extend: attention of a chunk of new tokens over the cache with changed scores and masks: scores capped by a
  tanh, a bias linear in the distance, a sliding window, packed documents, a prefix that every row sees
  (`ra_extend_attention_mod`);
* decode: the same for single tokens (`ra_decode_attention_mod`);
* verify: drafted tokens of a tree accepted or refused against the target's probabilities from given random
  numbers (`ra_tree_verify`), or against its largest logit (`ra_tree_verify_greedy`);
* slots: a step's slots, table entries, positions and row starts made from the requests' lengths
  (`ra_step_slots`), and the accepted path of each draft tree committed to the table, its refused slots
  returned to the free list (`ra_tree_commit`).

Attention.  Query row at position p of a request, key at position j, h the q head:
  s = sm_scale <q, k_j>;  with a cap c: s <- c tanh(s / c);  with slopes: s <- s - slopes[h] |p - j|;
  j is seen when max(first_key, p - window + 1) <= j (no window: window 0) and (j <= p or j < full_len).
A row that sees nothing gives 0.

Verification.  Node 0 of a tree is the token decided before; its row of the target's probabilities is the
distribution of the next token.  Rows p are taken as normalised.  At a node, its children are tried in index
order against the residual r = p, S = 1:
  drafts drawn from q (one row per node): child with token x is accepted when u q(x) S < r(x); on a refusal
    t <- t + S, r = max(p - t q, 0), S = sum r  (t = 0 before the first);
  drafts taken as given: accepted when u S < r(x); on a refusal S <- S - r(x), r(x) <- 0.
From the last accepted node the next token is drawn from r: the first v with sum_{j <= v} r(j) > u_final sum r.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one user's short turn over a cached conversation, capped scores: latency and the split of few rows
        dict(name="extend_one", op="extend", batch=1, hq=32, hkv=8, d=128, prefix_lo=1500, prefix_hi=1500, new_lo=33,
             new_hi=33, cap=50.0, window=0, slopes=False, doc=0, full=0),
        # the few-shot batch in a layer with a sliding window and capped scores
        dict(name="extend_window", op="extend", batch=16, hq=32, hkv=8, d=128, prefix_lo=3000, prefix_hi=3000,
             new_lo=200, new_hi=400, cap=30.0, window=1024, slopes=False, doc=0, full=0),
        # fresh prompts of several packed documents, a bias by distance, heads of 64
        dict(name="extend_docs", op="extend", batch=4, hq=16, hkv=16, d=64, prefix_lo=0, prefix_hi=0, new_lo=2000,
             new_hi=4095, cap=0.0, window=0, slopes=True, doc=611, full=0),
        # long prompts whose first part all rows see, capped, 70B-shape heads: the largest
        dict(name="extend_prefix", op="extend", batch=8, hq=64, hkv=8, d=128, prefix_lo=0, prefix_hi=2000, new_lo=700,
             new_hi=1500, cap=50.0, window=0, slopes=False, doc=0, full=512),
        # one user alone, capped
        dict(name="decode_one", op="decode", batch=1, hq=32, hkv=8, d=128, min_len=1500, max_len=1500, skewed=False,
             cap=50.0, window=0, slopes=False, first=False),
        # the 8B-shape decode batch in a layer with a sliding window
        dict(name="decode_window", op="decode", batch=64, hq=32, hkv=8, d=128, min_len=512, max_len=4096,
             skewed=False, cap=30.0, window=1024, slopes=False, first=False),
        # a large ragged multi-turn batch, 70B-shape heads, capped scores and a bias: HBM-bound
        dict(name="decode_mix", op="decode", batch=224, hq=64, hkv=8, d=128, min_len=65, max_len=13700, skewed=True,
             cap=50.0, window=0, slopes=True, first=False),
        # a few requests' short drafts that are taken as given: latency
        dict(name="verify_given", op="verify", mode="given", batch=4, draft=8, vocab=32003),
        # a full batch whose drafts were drawn from a draft model
        dict(name="verify_drawn", op="verify", mode="drawn", batch=64, draft=16, vocab=128000),
        # wide trees against the largest logit
        dict(name="verify_greedy", op="verify", mode="greedy", batch=64, draft=64, vocab=128000),
        # a prefill step's pages and slots
        dict(name="slots_prefill", op="slots", mode="step", batch=32, new_lo=64, new_hi=4001, cur_hi=5000, page=16,
             pad=37),
        # the trees of a full batch committed
        dict(name="slots_commit", op="slots", mode="commit", batch=224, draft=64, cur_hi=8000),
    ]


HEADS = [(32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 4, 128), (8, 8, 64), (16, 16, 64), (32, 32, 128), (8, 1, 128)]
# bounds of the drawn cases, from the largest listed ones: flops of an extend call without masks, bytes of a decode call
LARGEST_EXTEND, LARGEST_DECODE = 5.5e11, 2.9e9


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["extend", "extend", "decode", "decode", "verify", "slots"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "extend":
        lo, hi = sorted((log(1, 4001) - 1, log(1, 4001) - 1))
        n0, n1 = sorted((log(1, 4095), log(1, 4095)))
        c = dict(op=op, batch=log(1, 16), hq=hq, hkv=hkv, d=d, prefix_lo=lo, prefix_hi=hi, new_lo=n0, new_hi=n1,
                 cap=rng.choice([0.0, 20.0, 30.0, 50.0]), window=rng.choice([0, 0, log(1, 4096)]),
                 slopes=rng.random() < 0.4, doc=rng.choice([0, 0, log(5, 2000)]),
                 full=rng.choice([0, 0, log(1, 2000)]))
        while c["batch"] > 1 and dense(c) > LARGEST_EXTEND:
            c["batch"] //= 2
        while dense(c) > LARGEST_EXTEND:
            c["new_hi"] = max(1, c["new_hi"] // 2)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        return c
    if op == "decode":
        lo, hi = sorted((log(1, 13700), log(1, 13700)))
        c = dict(op=op, batch=log(1, 224), hq=hq, hkv=hkv, d=d, min_len=lo, max_len=hi, skewed=rng.random() < 0.5,
                 cap=rng.choice([0.0, 20.0, 30.0, 50.0]), window=rng.choice([0, 0, log(1, 4096)]),
                 slopes=rng.random() < 0.4, first=rng.random() < 0.3)
        while sum(context_lengths(c)) * hkv * d * 4 > LARGEST_DECODE:
            c["batch"] //= 2
        return c
    if op == "verify":
        mode = rng.choice(["given", "drawn", "greedy"])
        c = dict(op=op, mode=mode, batch=log(1, 64), draft=log(1, 64), vocab=log(500, 200000))
        while c["batch"] * c["draft"] * c["vocab"] > (64 * 64 if mode == "greedy" else 64 * 16) * 128000:
            c["batch"] = max(1, c["batch"] // 2)
        return c
    if rng.random() < 0.5:
        n0, n1 = sorted((log(1, 4001), log(1, 4001)))
        c = dict(op=op, mode="step", batch=log(1, 256), new_lo=n0 - 1, new_hi=n1, cur_hi=log(1, 8000),
                 page=rng.choice([1, 1, 16, 32, 64]), pad=rng.choice([0, rng.randrange(1, 100)]))
        while sum(new_lengths(c)) > 65000:
            c["batch"] = max(1, c["batch"] // 2)
        return c
    return dict(op=op, mode="commit", batch=log(1, 224), draft=log(1, 64), cur_hi=log(1, 8000))


# ------------------------------------------------------------------ lengths, from the case alone
def spread(batch, lo, hi, skewed=False):
    """`batch` lengths between lo and hi: evenly spread, or (skewed) evenly in their logarithm."""
    at = [(i + 0.5) / batch for i in range(batch)]
    if skewed:
        return [min(hi, int((lo + 1) * ((hi + 2) / (lo + 1)) ** u) - 1) for u in at]
    return [lo + int(u * (hi - lo + 1)) for u in at]


def new_lengths(c):
    return spread(c["batch"], c["new_lo"], c["new_hi"])


def prefix_lengths(c):
    return spread(c["batch"], c["prefix_lo"], c["prefix_hi"])[::-1]


def draft_lengths(c):
    return spread(c["batch"], max(1, c["draft"] // 2), c["draft"])


def context_lengths(c):
    return spread(c["batch"], c["min_len"], c["max_len"], c["skewed"])


def dense(c):
    return sum(e * (p + e) for p, e in zip(prefix_lengths(c), new_lengths(c))) * c["hq"] * c["d"] * 4


def full_length(c, b, length):
    """Keys of request b that every row sees."""
    return min(length, c["full"] + 17 * b) if c["full"] else 0


def first_of(c, p):
    """First key of the document of position p (documents of `doc` tokens)."""
    return p // c["doc"] * c["doc"] if c["doc"] else 0


# ------------------------------------------------------------------ inputs
def rows(gen, *shape):
    """K/V-like rows: normal values with a scale of their own per row."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    x *= torch.exp2(torch.rand(*shape[:-1], 1, generator=gen, device=DEV) * 2 - 1)
    return x.to(torch.bfloat16)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def slot_table(gen, lens, width, capacity):
    """A table whose row of request b lists lens[b] of `capacity` slots in random order (-1 behind them)."""
    slots = (torch.randperm(capacity - 1, generator=gen, device=DEV) + 1).int()  # slot 0 is the padding slot
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(len(lens), generator=gen, device=DEV).tolist()
    at = 0
    for b, n in enumerate(lens):
        table[order[b], :n] = slots[at:at + n]
        at += n
    return table, ints(order)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"extend": prepare_extend, "decode": prepare_decode, "verify": prepare_verify, "slots": prepare_slots}[
        c["op"]](c, gen)


def slopes_of(hq):
    return torch.exp2(-8.0 * (torch.arange(hq, device=DEV) + 1) / hq).float()


def prepare_extend(c, gen):
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    c["P"], c["E"] = prefix_lengths(c), new_lengths(c)
    lens = [p + e for p, e in zip(c["P"], c["E"])]
    capacity = sum(lens) + 17
    c["table"], c["rpi"] = slot_table(gen, lens, max(lens) + 3, capacity)
    c["rows"] = c["rpi"].tolist()
    c["k"], c["v"] = rows(gen, capacity, hkv, d), rows(gen, capacity, hkv, d)
    total = sum(c["E"])
    c["q"] = (3 * torch.randn(total, hq, d, generator=gen, device=DEV)).to(torch.bfloat16)
    c["o"] = torch.empty_like(c["q"])
    c["starts"] = [sum(c["E"][:b]) for b in range(c["batch"])]
    c["prefix"], c["new"], c["qo"] = ints(c["P"]), ints(c["E"]), ints(c["starts"] + [total])
    c["total"], c["scale"] = total, d ** -0.5
    c["bounds"] = dict(max_extend_len=max(c["E"]), max_prefix_len=max(c["P"]))
    c["slope"] = slopes_of(hq) if c["slopes"] else None
    c["first_key"] = c["full_lens"] = None
    if c["doc"]:
        c["first_key"] = ints([first_of(c, p) for b in range(c["batch"]) for p in range(c["P"][b], lens[b])])
    if c["full"]:
        c["full_lens"] = ints([full_length(c, b, n) for b, n in enumerate(lens)])
    return c


def prepare_decode(c, gen):
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    lens = context_lengths(c)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=gen, device=DEV).tolist()]
    capacity = sum(lens) + 17
    c["table"], c["rpi"] = slot_table(gen, lens, max(lens), capacity)
    c["k"], c["v"] = rows(gen, capacity, hkv, d), rows(gen, capacity, hkv, d)
    c["lens"] = ints(lens)
    c["L"], c["rows"] = lens, c["rpi"].tolist()
    c["q"] = (3 * torch.randn(c["batch"], hq, d, generator=gen, device=DEV)).to(torch.bfloat16)
    c["o"] = torch.empty_like(c["q"])
    c["scale"], c["slope"] = d ** -0.5, slopes_of(hq) if c["slopes"] else None
    c["F"] = [n // 3 for n in lens] if c["first"] else [0] * len(lens)
    c["first_key"] = ints(c["F"]) if c["first"] else None
    return c


def random_trees(c, gen):
    """draft lengths, row starts and parents (-1 at node 0; a node's parent is a node before it)."""
    c["T"] = draft_lengths(c)
    c["widest"] = max(c["T"])
    c["starts"] = [sum(c["T"][:b]) for b in range(c["batch"])]
    c["total"] = sum(c["T"])
    c["drafts"], c["qo"] = ints(c["T"]), ints(c["starts"] + [c["total"]])
    i = torch.cat([torch.arange(t, device=DEV) for t in c["T"]])
    # half of the nodes extend the node before them (chains), the others any earlier one
    back = torch.floor(torch.rand(c["total"], generator=gen, device=DEV) * i).long()
    chain = torch.rand(c["total"], generator=gen, device=DEV) < 0.5
    c["parents"] = torch.where(i > 0, torch.where(chain, i - 1, back), -1).int()
    c["base"] = (torch.arange(c["total"], device=DEV) - i)     # row of the request's node 0
    c["path"] = torch.empty(c["batch"], c["widest"], dtype=torch.int32, device=DEV)
    c["accepted"] = torch.empty(c["batch"], dtype=torch.int32, device=DEV)


def pick(gen, probs):
    """One token per row, drawn from its probabilities."""
    u = torch.rand(probs.shape[0], 1, generator=gen, device=DEV, dtype=torch.float64)
    cdf = probs.double().cumsum(1)
    return (cdf <= u * cdf[:, -1:]).sum(1).clamp(max=probs.shape[1] - 1)


def prepare_verify(c, gen):
    random_trees(c, gen)
    n, vocab = c["total"], c["vocab"]
    parent = (c["base"] + c["parents"].clamp(min=0)).long()
    c["next"] = torch.empty(c["batch"], dtype=torch.int32, device=DEV)
    # a long tail with a few likely tokens
    logits = torch.randn(n, vocab, generator=gen, device=DEV) * 2
    likely = torch.randint(0, vocab, (n, 8), generator=gen, device=DEV)
    logits.scatter_add_(1, likely, 8 + 10 * torch.rand(n, 8, generator=gen, device=DEV))
    if c["mode"] == "greedy":
        c["logits"] = logits.to(torch.bfloat16)
        del logits
        top = first_largest(c["logits"])[parent]
        other = torch.randint(0, vocab, (n,), generator=gen, device=DEV)
        c["tokens"] = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.7, top, other).int()
        return c
    c["target"] = torch.softmax(logits, -1)
    logits += torch.randn(n, vocab, generator=gen, device=DEV) * 0.5
    draft = torch.softmax(logits, -1)
    del logits
    c["tokens"] = torch.cat([pick(gen, draft[parent[i:i + 128]]) for i in range(0, n, 128)]).int()
    c["draft_probs"] = draft if c["mode"] == "drawn" else None
    c["u"] = torch.rand(n, generator=gen, device=DEV)
    c["u_final"] = torch.rand(c["batch"], generator=gen, device=DEV)
    return c


def prepare_slots(c, gen):
    batch = c["batch"]
    cur = torch.randint(0, c["cur_hi"] + 1, (batch,), generator=gen, device=DEV).tolist()
    if c["mode"] == "commit":
        random_trees(c, gen)
        new = c["T"]
        page, spare = 1, 0
    else:
        new = new_lengths(c)
        page, spare = c["page"], c["pad"]
    width = c["cur_hi"] + max(new) + 5
    pages = [-(-a // page) for a in cur]
    need = [-(-(a + b) // page) - n for a, b, n in zip(cur, new, pages)]
    count = sum(pages) + sum(need) + 50
    ids = (torch.randperm(count, generator=gen, device=DEV) + 1).int()
    table = torch.full((batch + 1, width), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(batch + 1, generator=gen, device=DEV)[:batch].tolist()
    at, off = 0, torch.arange(page, device=DEV)
    for b in range(batch):
        table[order[b], :cur[b]] = (ids[at:at + pages[b], None] * page + off).flatten()[:cur[b]].int()
        at += pages[b]
    c["table"], c["rpi"], c["cur"] = table, ints(order), ints(cur)
    total = sum(new)
    c["left"] = torch.empty(1, dtype=torch.int32, device=DEV)
    c["seq"] = torch.empty(batch, dtype=torch.int32, device=DEV)
    if c["mode"] == "step":
        c["free"], c["count"] = ids[at:].contiguous(), ints([count - at])
        c["new"] = ints(new)
        c["loc"] = torch.empty(total + spare, dtype=torch.int32, device=DEV)
        c["positions"] = torch.empty_like(c["loc"])
        c["qo"] = torch.empty(batch + 1, dtype=torch.int32, device=DEV)
        return c
    # the step's drafted slots and an accepted path per tree: from node 0, a random child at each step
    c["loc"] = ids[at:at + total].contiguous()
    free = ids[at + total:]
    c["free"] = torch.cat([free, torch.zeros(total + 3, dtype=torch.int32, device=DEV)])
    c["count"] = ints([count - at - total])
    parents, score = c["parents"].tolist(), torch.rand(total, generator=gen, device=DEV).tolist()
    path, accepted = [], []
    for b in range(batch):
        q0, kids = c["starts"][b], {}
        for i in range(1, c["T"][b]):
            kids.setdefault(parents[q0 + i], []).append(i)
        walk = [0]
        while walk[-1] in kids and score[q0 + walk[-1]] < 0.8:
            choice = kids[walk[-1]]
            walk.append(choice[int(score[q0 + walk[-1]] * len(choice))])
        path.append(walk + [-1] * (c["widest"] - len(walk)))
        accepted.append(len(walk))
    c["path"], c["accepted"] = ints(path), ints(accepted)
    return c


# ------------------------------------------------------------------ one pass
def run(s):
    return {"extend": run_extend, "decode": run_decode, "verify": run_verify,
            "slots": run_commit if s.get("mode") == "commit" else run_step}[s["op"]](s)


def attend32(q, k, v, s, p, first, full):
    """q [t, hq, d] at positions p [t] over k, v [l, hkv, d] in 32 bits; first [t] or None, full a length."""
    hkv = k.shape[1]
    q = q.float().unflatten(1, (hkv, -1))
    x = torch.einsum("thgd,lhd->hgtl", q, k.float()) * s["scale"]
    if s["cap"]:
        x = torch.tanh(x / s["cap"]) * s["cap"]
    j = torch.arange(k.shape[0], device=DEV)
    dist = p[:, None] - j[None, :]
    if s["slope"] is not None:
        x = x - s["slope"].reshape(hkv, -1, 1, 1) * dist.abs().float()
    hidden = (dist < 0) & (j[None, :] >= full)
    if s["window"]:
        hidden |= dist >= s["window"]
    if first is not None:
        hidden |= j[None, :] < first[:, None]
    x = x.masked_fill(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    y = torch.einsum("hgtl,lhd->thgd", e, v.float())
    total = e.sum(-1).permute(2, 0, 1)[..., None]
    return torch.where(total > 0, y / total, torch.zeros_like(y)).flatten(1, 2)


def run_extend(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        if "ws" not in s:
            s["ws"] = torch.empty(ra.ra_extend_mod_workspace_bytes(s["batch"], s["total"], s["hq"], s["hkv"]),
                                  dtype=torch.uint8, device=DEV)
        ra.ra_extend_attention_mod(s["k"], s["v"], s["q"], s["o"], s["table"], s["rpi"], s["prefix"], s["new"], s["qo"],
                                   sm_scale=s["scale"], score_cap=s["cap"], window=s["window"], slopes=s["slope"],
                                   first_key=s["first_key"], full_lens=s["full_lens"], workspace=s["ws"], **s["bounds"])
        return s["o"]
    for b in range(s["batch"]):
        P, E, q0 = s["P"][b], s["E"][b], s["starts"][b]
        at = s["table"][s["rows"][b], :P + E].long()
        k, v = s["k"][at], s["v"][at]
        full = full_length(s, b, P + E)
        for i in range(0, E, 512):
            n = min(512, E - i)
            rows_ = slice(q0 + i, q0 + i + n)
            first = s["first_key"][rows_] if s["doc"] else None
            s["o"][rows_] = attend32(s["q"][rows_], k, v, s, P + i + torch.arange(n, device=DEV), first, full).to(
                torch.bfloat16)
    return s["o"]


def run_decode(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        if "ws" not in s:
            s["ws"] = torch.empty(ra.ra_decode_workspace_bytes(s["batch"], s["hq"], s["hkv"], s["d"],
                                                               s["table"].shape[1]), dtype=torch.uint8, device=DEV)
        ra.ra_decode_attention_mod(s["k"], s["v"], s["q"], s["o"], s["table"], s["rpi"], s["lens"],
                                   max_seq_len=s["table"].shape[1], sm_scale=s["scale"], score_cap=s["cap"],
                                   window=s["window"], slopes=s["slope"], first_key=s["first_key"], workspace=s["ws"])
        return s["o"]
    for b in range(s["batch"]):
        at = s["table"][s["rows"][b], :s["L"][b]].long()
        p = torch.full((1,), s["L"][b] - 1, device=DEV)
        s["o"][b] = attend32(s["q"][b:b + 1], s["k"][at], s["v"][at], s, p,
                             s["first_key"][b:b + 1] if s["first"] else None, 0)[0].to(torch.bfloat16)
    return s["o"]


def first_largest(x):
    """Index of each row's largest value, the lowest of equal ones."""
    out = []
    for part in x.split(256):
        top = part.amax(1, keepdim=True)
        i = torch.arange(x.shape[1], device=DEV)
        out.append(torch.where(part == top, i, x.shape[1]).amin(1))
    return torch.cat(out)


def run_verify(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        tree = (s["tokens"], s["parents"], s["drafts"], s["qo"])
        out = (s["path"], s["accepted"], s["next"])
        if s["mode"] == "greedy":
            ra.ra_tree_verify_greedy(s["logits"], *tree, *out, max_draft_len=s["widest"])
        else:
            ra.ra_tree_verify(s["target"], s["draft_probs"], *tree, s["u"], s["u_final"], *out,
                              max_draft_len=s["widest"])
        return out
    batch, vocab = s["batch"], s["vocab"]
    start, drafts = s["qo"][:-1].long(), s["drafts"].long()
    cur = torch.zeros(batch, dtype=torch.long, device=DEV)
    count = torch.ones_like(cur)
    path = torch.full((batch, s["widest"] + 1), -1, dtype=torch.long, device=DEV)  # (a spare column for no entry)
    path[:, 0] = 0
    greedy, drawn = s["mode"] == "greedy", s["mode"] == "drawn"
    if greedy:
        top = first_largest(s["logits"])
    else:
        t = torch.zeros(batch, 1, dtype=torch.float64, device=DEV)
        total = torch.ones_like(t)
        gone = torch.zeros(batch, vocab, dtype=torch.bool, device=DEV)
    for i in range(1, s["widest"]):
        row = (start + i).clamp(max=s["total"] - 1)
        here = (i < drafts) & (s["parents"][row] == cur)
        token = s["tokens"][row].long()
        if greedy:
            take = here & (top[start + cur] == token)
        else:
            at = start + cur
            u = s["u"][row].double()[:, None]
            x = token[:, None]
            r = s["target"][at, token].double()[:, None]
            if drawn:
                qx = s["draft_probs"][at, token].double()[:, None]
                take = (u * qx * total < (r - t * qx).clamp(min=0))[:, 0] & here
            else:
                r = torch.where(gone.gather(1, x), torch.zeros_like(r), r)
                take = (u * total < r)[:, 0] & here
            refuse = (here & ~take)[:, None]
            if drawn:
                t2 = t + total
                rest = (s["target"][at].double() - t2 * s["draft_probs"][at].double()).clamp(min=0).sum(1, keepdim=True)
                t, total = torch.where(refuse, t2, t), torch.where(refuse, rest, total)
            else:
                total = torch.where(refuse, total - r, total)
                gone.scatter_(1, x, gone.gather(1, x) | refuse)
            t = torch.where(take[:, None], torch.zeros_like(t), t)
            total = torch.where(take[:, None], torch.ones_like(total), total)
            gone &= ~take[:, None]
        cur = torch.where(take, i, cur)
        path.scatter_(1, torch.where(take, count, s["widest"])[:, None], i)
        count = count + take
    path[:, -1] = -1
    s["path"].copy_(path[:, :-1])
    s["accepted"].copy_(count)
    if greedy:
        s["next"].copy_(top[start + cur])
        return s["path"], s["accepted"], s["next"]
    p = s["target"][start + cur].double()
    r = p.masked_fill(gone, 0)
    if drawn:
        r = (r - t * s["draft_probs"][start + cur].double()).clamp(min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    cdf = r.cumsum(1)
    # rounding may leave no sum above the bound: the last token with any weight, then
    at = torch.where(cdf > s["u_final"].double()[:, None] * cdf[:, -1:], torch.arange(vocab, device=DEV), vocab).amin(1)
    last = torch.where(r > 0, torch.arange(vocab, device=DEV), 0).amax(1)
    s["next"].copy_(torch.where(at < vocab, at, last))
    return s["path"], s["accepted"], s["next"]


def run_step(s):
    out = (s["table"], s["loc"], s["positions"], s["qo"], s["seq"], s["left"])
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        ra.ra_step_slots(s["table"], s["rpi"], s["cur"], s["new"], s["free"], s["count"], s["loc"], s["positions"],
                         s["qo"], s["seq"], page_size=s["page"], free_count_out=s["left"])
        return out
    cur, new, page = s["cur"].long(), s["new"].long(), s["page"]
    have = (cur + page - 1) // page
    need = (cur + new + page - 1) // page - have
    ends = new.cumsum(0)
    t = torch.arange(s["loc"].shape[0], device=DEV)
    live = t < ends[-1]
    b = torch.searchsorted(ends, t, right=True).clamp(max=cur.shape[0] - 1)
    i = t - (ends - new)[b]
    pos = cur[b] + i
    fresh = pos >= have[b] * page
    nth = (need.cumsum(0) - need)[b] + pos // page - have[b]
    taken = s["free"][(s["count"].long() - 1 - nth).clamp(0, s["free"].shape[0] - 1)].long() * page + pos % page
    row = s["rpi"].long()[b]
    before = s["table"][row, (cur[b] - 1).clamp(min=0)].long() + i + 1
    slot = torch.where(fresh, taken, before)
    s["loc"].copy_(torch.where(live, slot, 0))
    s["positions"].copy_(torch.where(live, pos, 0))
    # (entries behind the last token repeat token 0's)
    one = torch.where(live, t, 0)
    s["table"][row[one], pos[one]] = slot[one].int()
    s["qo"][0] = 0
    s["qo"][1:] = ends
    s["seq"].copy_(cur + new)
    s["left"].copy_(s["count"] - need.sum())
    return out


def run_commit(s):
    out = (s["table"], s["seq"], s["free"], s["left"])
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        ra.ra_tree_commit(s["table"], s["rpi"], s["cur"], s["drafts"], s["qo"], s["loc"], s["path"], s["accepted"],
                          s["seq"], s["free"], s["count"], free_count_out=s["left"])
        return out
    batch, widest, total = s["batch"], s["widest"], s["total"]
    cur, drafts, n = s["cur"].long(), s["drafts"].long(), s["accepted"].long()
    i = torch.arange(widest, device=DEV)
    start = s["qo"][:-1].long()[:, None]
    kept = i < n[:, None]
    node = torch.where(kept, s["path"].long(), 0)
    slot = torch.where(kept, s["loc"][(start + node).clamp(max=total - 1)], -1)
    inside = i < drafts[:, None]
    at = (cur[:, None] + torch.minimum(i, drafts[:, None] - 1))
    s["table"][s["rpi"].long()[:, None], at] = torch.where(inside, slot, slot.gather(1, drafts[:, None] - 1))
    dead = torch.ones(total, dtype=torch.int32, device=DEV)
    dead[torch.where(kept, start + node, start)] = 0
    nth = dead.cumsum(0) - 1 + s["count"].long()
    s["free"].scatter_(0, torch.where(dead > 0, nth, s["free"].shape[0] - 1), torch.where(dead > 0, s["loc"], 0))
    s["seq"].copy_(cur + n)
    s["left"].copy_(s["count"] + dead.sum())
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(c):
    if c["op"] == "extend":
        keys = pairs = 0
        for b, (P, E) in enumerate(zip(prefix_lengths(c), new_lengths(c))):
            full, lowest = full_length(c, b, P + E), P + E
            for p in range(P, P + E):
                lo = max(first_of(c, p), p - c["window"] + 1 if c["window"] else 0)
                lowest = min(lowest, lo)
                pairs += max(p + 1, full) - lo
            keys += P + E - lowest
        n = sum(new_lengths(c))
        return dict(bytes=keys * (c["hkv"] * c["d"] * 4 + 4) + n * c["hq"] * c["d"] * 4,
                    flops=pairs * c["hq"] * c["d"] * 4)
    if c["op"] == "decode":
        seen = 0
        for n in context_lengths(c):
            lo = max(n // 3 if c["first"] else 0, n - c["window"] if c["window"] else 0)
            seen += n - lo
        return dict(bytes=seen * (c["hkv"] * c["d"] * 4 + 4) + c["batch"] * c["hq"] * c["d"] * 4,
                    flops=seen * c["hq"] * c["d"] * 4)
    if c["op"] == "verify":
        n = sum(draft_lengths(c))
        # one row of the target per tree at least (and one of the drafts where there were refusals)
        per = {"given": 4, "drawn": 8, "greedy": 2}[c["mode"]] * c["vocab"]
        return dict(bytes=c["batch"] * per + n * 12, flops=c["batch"] * c["vocab"] * 2)
    if c["mode"] == "step":
        n = sum(new_lengths(c))
        return dict(bytes=n * 12 + n // c["page"] * 4 + c["pad"] * 8 + c["batch"] * 24, flops=n * 2)
    n = sum(draft_lengths(c))
    return dict(bytes=n * 12 + c["batch"] * 24, flops=n * 2)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": exact_extend, "decode": exact_decode, "verify": exact_verify,
            "slots": exact_commit if s.get("mode") == "commit" else exact_step}[s["op"]](s)


def seen_softmax(q, k, v, s, p, first, full):
    """Rows q [t, hq, d] at positions p (a list) over k, v [l, hkv, d], head by head, all in 64 bits."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    group = q.shape[1] // k.shape[1]
    j = torch.arange(k.shape[0], device=DEV)
    low = torch.tensor([max(f, a - s["window"] + 1 if s["window"] else 0) for a, f in zip(p, first)], device=DEV)
    high = torch.tensor([max(a + 1, full) for a in p], device=DEV)
    seen = (j >= low[:, None]) & (j < high[:, None])
    far = (torch.tensor(p, device=DEV)[:, None] - j).abs().double()
    some = seen.any(1)
    for h in range(q.shape[1]):
        x = q[:, h].double() @ k[:, h // group].double().T * s["scale"]
        if s["cap"]:
            x = s["cap"] * torch.tanh(x / s["cap"])
        if s["slope"] is not None:
            x = x - float(s["slope"][h]) * far
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        x[~some] = 0.0
        y = torch.softmax(x, -1) @ v[:, h // group].double()
        out[:, h] = torch.where(some[:, None], y, torch.zeros_like(y))
    return out


def exact_extend(s):
    out = []
    for b in range(s["batch"]):
        P, E, q0 = s["P"][b], s["E"][b], s["starts"][b]
        at = s["table"][s["rows"][b], :P + E].long()
        p = list(range(P, P + E))
        out.append(seen_softmax(s["q"][q0:q0 + E], s["k"][at], s["v"][at], s, p, [first_of(s, a) for a in p],
                                full_length(s, b, P + E)))
    return torch.cat(out)


def exact_decode(s):
    out = []
    for b in range(s["batch"]):
        at = s["table"][s["rows"][b], :s["L"][b]].long()
        out.append(seen_softmax(s["q"][b:b + 1], s["k"][at], s["v"][at], s, [s["L"][b] - 1], [s["F"][b]], 0))
    return torch.cat(out)


def exact_verify(s):
    paths, accepted, nexts = [], [], []
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    for b in range(s["batch"]):
        q0, T = s["starts"][b], s["T"][b]
        walk, done, pick_ = [0], False, None
        while not done:
            node = walk[-1]
            kids = [i for i in range(node + 1, T) if parents[q0 + i] == node]
            done = True
            if s["mode"] == "greedy":
                x = s["logits"][q0 + node].double()
                pick_ = int((x == x.max()).nonzero()[0])
                for i in kids:
                    if tokens[q0 + i] == pick_:
                        walk.append(i)
                        done = False
                        break
                continue
            p = s["target"][q0 + node].double()
            r, mass = p.clone(), 1.0          # the residual, not normalised, and its sum
            q = s["draft_probs"][q0 + node].double() if s["mode"] == "drawn" else None
            for i in kids:
                x, u = tokens[q0 + i], float(s["u"][q0 + i])
                chance = float(r[x]) / mass if mass else 0.0
                if u * (float(q[x]) if q is not None else 1.0) < chance:
                    walk.append(i)
                    done = False
                    break
                if q is not None:
                    r = torch.clamp(r - mass * q, min=0)   # (r / mass - q, times mass)
                    mass = float(r.sum())
                else:
                    mass -= float(r[x])
                    r[x] = 0
            if done:
                if not float(r.sum()) > 0:
                    r = p
                sums = torch.cumsum(r, 0)
                above = (sums > float(s["u_final"][b]) * sums[-1]).nonzero()
                pick_ = int(above[0]) if len(above) else int((r > 0).nonzero()[-1])
        paths.append(walk + [-1] * (s["widest"] - len(walk)))
        accepted.append(len(walk))
        nexts.append(pick_)
    return ints(paths), ints(accepted), ints(nexts)


def exact_step(s):
    table, free = s["table"].tolist(), s["free"].tolist()
    left, page = int(s["count"]), s["page"]
    loc, positions, qo, seq = [], [], [0], []
    for row, cur, new in zip(s["rpi"].tolist(), s["cur"].tolist(), s["new"].tolist()):
        for p in range(cur, cur + new):
            if p % page == 0:
                left -= 1
                slot = free[left] * page
            else:
                slot = table[row][p - 1] + 1
            table[row][p] = slot
            loc.append(slot)
            positions.append(p)
        qo.append(len(loc))
        seq.append(cur + new)
    spare = [0] * (s["loc"].shape[0] - len(loc))
    return ints(table), ints(loc + spare), ints(positions + spare), ints(qo), ints(seq), ints([left])


def exact_commit(s):
    table, loc, free = s["table"].tolist(), s["loc"].tolist(), s["free"].tolist()
    left, seq = int(s["count"]), []
    for b, (row, cur) in enumerate(zip(s["rpi"].tolist(), s["cur"].tolist())):
        q0, T, n = s["starts"][b], s["T"][b], int(s["accepted"][b])
        nodes = s["path"][b, :n].tolist()
        table[row][cur:cur + T] = [loc[q0 + i] for i in nodes] + [-1] * (T - n)
        for i in range(T):
            if i not in nodes:
                free[left] = loc[q0 + i]
                left += 1
        seq.append(cur + n)
    return ints(table), ints(seq), ints(free), ints([left])
