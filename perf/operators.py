"""Measured cases of the serving operators around the attention calls.

Four operators, each in a plain form (elementary torch operations in 32 bits, `own` false) and as the
calls a user makes of this package (`own` true):

* norm_rope: per-head RMS norm of q and k, the position rotation, and the store of k and v into their
  pool slots, in one pass over a fused qkv projection (`ra_qk_norm_rope_store`, or
  `ra_qk_norm_rope_kv8_store` for a quantised pool);
* kv8_store: new K/V rows quantised into pool slots and read back (`ra_kv8_store`, `ra_kv8_load`);
* kv8_load: cached rows read back from a quantised pool (`ra_kv8_load`);
* kv8_decode: decode attention over a quantised pool (`ra_kv8_decode_attention`);
* tree: attention of a tree of drafted tokens over a cached prefix (`ra_tree_attention`).

A quantised pool holds one record per token slot, made of blocks of `hpc` kv heads (the largest divisor
of the number of kv heads that is at most 8).  A block is, per head, the D codes of K then the D codes of
V (e4m3), followed by 16 bytes of scales: byte 2h is head h's K exponent and byte 2h + 1 its V exponent,
both biased by 127 (the value is code x 2^(byte - 127)), the rest zero.  A record is padded to a multiple
of 32 bytes.  The exponent of a row is the smallest e with max|x| <= 448 x 2^e, clamped to [-118, 119].
"""
import math

import torch

own = False

DEV = "cuda"
ROPE_BASE = 500000.0
MAX_POS = 32768


def listed():
    return [
        # one decode step of 64 requests, 8B-shape heads: launch latency counts
        dict(name="norm_rope_decode", op="norm_rope", tokens=64, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             kv="bf16"),
        # the prefill tokens of a large multi-turn step, 70B-shape heads: HBM-bound
        dict(name="norm_rope_prefill", op="norm_rope", tokens=9437, hq=64, hkv=8, d=128, rot=128, interleaved=False,
             kv="bf16"),
        # a small model's heads, half of each head rotated in adjacent pairs, into a quantised pool
        dict(name="norm_rope_kv8_partial", op="norm_rope", tokens=4777, hq=8, hkv=2, d=64, rot=32, interleaved=True,
             kv="e4m3"),
        # one decode step's new rows of 224 requests quantised and read back
        dict(name="kv8_store_decode", op="kv8_store", tokens=224, hkv=8, d=128),
        # a long prefill's rows: HBM-bound
        dict(name="kv8_store_prefill", op="kv8_store", tokens=65521, hkv=8, d=128),
        # a few-shot prefix read back for an extend call
        dict(name="kv8_load_prefix", op="kv8_load", tokens=3000, hkv=8, d=128),
        # the distinct tokens of a whole multi-turn batch read back
        dict(name="kv8_load_batch", op="kv8_load", tokens=239251, hkv=8, d=128),
        # one user alone: latency
        dict(name="kv8_decode_one", op="kv8_decode", batch=1, hq=32, hkv=8, d=128, min_len=1500, max_len=1500,
             skewed=False),
        # the 8B-shape decode batch
        dict(name="kv8_decode_8b", op="kv8_decode", batch=64, hq=32, hkv=8, d=128, min_len=512, max_len=4096,
             skewed=False),
        # a large ragged multi-turn batch, 70B-shape heads
        dict(name="kv8_decode_mix", op="kv8_decode", batch=224, hq=64, hkv=8, d=128, min_len=65, max_len=13700,
             skewed=True),
        # a few requests with short drafts: latency and the split of the prefix
        dict(name="tree_small", op="tree", batch=4, hq=32, hkv=8, d=128, min_len=512, max_len=4096,
             skewed=False, draft=8),
        # a full batch with wide trees, 70B-shape heads: tensor-core bound
        dict(name="tree_large", op="tree", batch=64, hq=64, hkv=8, d=128, min_len=512, max_len=4096,
             skewed=False, draft=64),
    ]


HEADS = [(32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 4, 128), (8, 8, 64), (16, 16, 128), (12, 3, 128), (5, 5, 64)]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_rope", "kv8_store", "kv8_load", "kv8_decode", "tree"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "norm_rope":
        return dict(op=op, tokens=log(1, 9437), hq=hq, hkv=hkv, d=d, rot=rng.choice([16, 32, 64, d]),
                    interleaved=rng.random() < 0.5, kv=rng.choice(["bf16", "e4m3"]))
    if op in ("kv8_store", "kv8_load"):
        return dict(op=op, tokens=log(1, 65521), hkv=hkv, d=d)
    if op == "kv8_decode":
        lo, hi = sorted((log(1, 13700), log(1, 13700)))
        return dict(op=op, batch=log(1, 224), hq=hq, hkv=hkv, d=d, min_len=lo, max_len=hi,
                    skewed=rng.random() < 0.5)
    lo, hi = sorted((log(1, 4096) - 1, log(1, 4096)))
    return dict(op=op, batch=log(1, 64), hq=hq, hkv=hkv, d=d, min_len=lo, max_len=hi, skewed=rng.random() < 0.5,
                draft=log(1, 64))


# ------------------------------------------------------------------ quantised records, in torch
def heads_per_block(hkv):
    return next(h for h in range(8, 0, -1) if hkv % h == 0)


def slot_bytes(hkv, d):
    hpc = heads_per_block(hkv)
    return (hkv // hpc * (hpc * 2 * d + 16) + 31) // 32 * 32


def row_exponents(x):
    """Smallest e with max|x| <= 448 * 2^e over the last axis, clamped to [-118, 119] (fp32 rows)."""
    m, ex = torch.frexp(x.abs().amax(-1))
    e = ex.to(torch.int32) - torch.where(m <= 0.875, 9, 8).to(torch.int32)
    return torch.where(m == 0, -118, e).clamp(-118, 119)


def pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def quantise(x):
    """fp32 rows -> (e4m3 codes, int32 exponents)."""
    e = row_exponents(x)
    return (x * pow2(-e)[..., None]).to(torch.float8_e4m3fn), e


def pack(k, v):
    """fp32 K and V rows [n, hkv, d] -> records [n, slot_bytes]."""
    n, hkv, d = k.shape
    hpc = heads_per_block(hkv)
    ck, ek = quantise(k)
    cv, ev = quantise(v)
    codes = torch.stack([ck.view(torch.uint8), cv.view(torch.uint8)], 2).reshape(n, hkv // hpc, hpc * 2 * d)
    scales = torch.zeros(n, hkv // hpc, 16, dtype=torch.uint8, device=k.device)
    scales[:, :, :2 * hpc] = (torch.stack([ek, ev], 2) + 127).to(torch.uint8).reshape(n, hkv // hpc, 2 * hpc)
    rec = torch.cat([codes, scales], 2).reshape(n, -1)
    return torch.nn.functional.pad(rec, (0, slot_bytes(hkv, d) - rec.shape[1]))


def unpack(rec, hkv, d):
    """Records [..., slot_bytes] -> fp32 K and V rows [..., hkv, d]."""
    hpc = heads_per_block(hkv)
    blocks = hkv // hpc
    size = hpc * 2 * d + 16
    rec = rec[..., :blocks * size].reshape(*rec.shape[:-1], blocks, size)
    codes = rec[..., :hpc * 2 * d].contiguous().view(torch.float8_e4m3fn).float()
    codes = codes.reshape(*rec.shape[:-2], hkv, 2, d)
    e = rec[..., hpc * 2 * d:hpc * 2 * d + 2 * hpc].reshape(*rec.shape[:-2], hkv, 2).int() - 127
    kv = codes * pow2(e)[..., None]
    return kv[..., 0, :], kv[..., 1, :]


# ------------------------------------------------------------------ inputs
def rows(gen, *shape):
    """K/V-like rows: normal values with a scale of their own per row."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    x *= torch.exp2(torch.rand(*shape[:-1], 1, generator=gen, device=DEV) * 4 - 2)
    return x.to(torch.bfloat16)


def context(gen, lens, capacity):
    """A pool of `capacity` slots and a table whose row of request b lists lens[b] of them, in random order."""
    batch, longest = len(lens), int(lens.max())
    slots = torch.randperm(capacity - 1, generator=gen, device=DEV).int() + 1  # slot 0 is the padding slot
    start = torch.cumsum(lens, 0) - lens
    at = start[:, None] + torch.arange(longest, device=DEV)[None, :]
    table = torch.where(torch.arange(longest, device=DEV)[None, :] < lens[:, None],
                        slots[at.clamp(max=capacity - 2)], -1).int()
    order = torch.randperm(batch, generator=gen, device=DEV)
    out = torch.empty_like(table)
    out[order] = table
    return out.contiguous(), order.int()


def spread(batch, lo, hi, skewed):
    """`batch` lengths between lo and hi: evenly spread, or (skewed) evenly in their logarithm."""
    at = [(i + 0.5) / batch for i in range(batch)]
    if skewed:
        return [min(hi, int((lo + 1) * ((hi + 2) / (lo + 1)) ** u) - 1) for u in at]
    return [lo + int(u * (hi - lo + 1)) for u in at]


def context_lengths(c):
    return spread(c["batch"], c["min_len"], c["max_len"], c["skewed"])


def draft_lengths(c):
    return spread(c["batch"], max(1, c["draft"] // 2), c["draft"], False)


def shuffled(gen, lens):
    return torch.tensor(lens, device=DEV)[torch.randperm(len(lens), generator=gen, device=DEV)]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hkv, d = c["hkv"], c["d"]
    if c["op"] == "norm_rope":
        n, hq, rot = c["tokens"], c["hq"], c["rot"]
        c["qkv"] = rows(gen, n, hq + 2 * hkv, d)
        c["q"], c["k"], c["v"] = c["qkv"].split([hq, hkv, hkv], 1)
        c["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16)
        c["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16)
        c["eps"] = 1e-6
        c["positions"] = torch.randint(0, MAX_POS, (n,), generator=gen, device=DEV, dtype=torch.int32)
        freq = ROPE_BASE ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(MAX_POS, device=DEV, dtype=torch.float64)[:, None] * freq
        c["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        c["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        slots = n + n // 4 + 16
        c["loc"] = torch.randperm(slots - 1, generator=gen, device=DEV)[:n].int() + 1
        if c["kv"] == "bf16":
            c["k_pool"] = torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device=DEV)
            c["v_pool"] = torch.zeros_like(c["k_pool"])
        else:
            c["pool"] = torch.zeros(slots, slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
            c["k_back"] = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=DEV)
            c["v_back"] = torch.empty_like(c["k_back"])
        return c
    if c["op"] in ("kv8_store", "kv8_load"):
        n = c["tokens"]
        slots = n + n // 4 + 16
        c["loc"] = torch.randperm(slots - 1, generator=gen, device=DEV)[:n].int() + 1
        c["pool"] = torch.zeros(slots, slot_bytes(hkv, d), dtype=torch.uint8, device=DEV)
        c["k"], c["v"] = rows(gen, n, hkv, d), rows(gen, n, hkv, d)
        if c["op"] == "kv8_load":
            c["pool"][c["loc"].long()] = pack(c.pop("k").float(), c.pop("v").float())
        c["k_back"] = torch.empty(n, hkv, d, dtype=torch.bfloat16, device=DEV)
        c["v_back"] = torch.empty_like(c["k_back"])
        return c
    batch, hq = c["batch"], c["hq"]
    c["scale"] = d ** -0.5
    lens = shuffled(gen, context_lengths(c))
    if c["op"] == "kv8_decode":
        capacity = int(lens.sum()) + 17
        c["table"], c["rpi"] = context(gen, lens, capacity)
        c["pool"] = pack(rows(gen, capacity, hkv, d).float(), rows(gen, capacity, hkv, d).float())
        c["lens"] = lens.int()
        c["q"] = torch.randn(batch, hq, d, generator=gen, device=DEV).to(torch.bfloat16)
        c["o"] = torch.empty_like(c["q"])
        return c
    draft = shuffled(gen, draft_lengths(c))
    total, widest = int(draft.sum()), int(draft.max())
    c["bounds"] = dict(max_draft_len=widest, max_prefix_len=int(lens.max()))
    capacity = int((lens + draft).sum()) + 17
    c["table"], c["rpi"] = context(gen, lens + draft, capacity)
    c["k_pool"], c["v_pool"] = rows(gen, capacity, hkv, d), rows(gen, capacity, hkv, d)
    c["prefix"], c["drafts"] = lens.int(), draft.int()
    c["qo"] = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64), draft.cumsum(0)]).int()
    c["total"] = total
    c["q"] = torch.randn(total, hq, d, generator=gen, device=DEV).to(torch.bfloat16)
    c["o"] = torch.empty_like(c["q"])
    # random trees: token i's parent is a token before it, or the last prefix token; a token sees its
    # ancestors and itself
    parent = torch.floor(torch.rand(batch, widest, generator=gen, device=DEV)
                         * (torch.arange(widest, device=DEV) + 1)).long() - 1
    reach = torch.eye(widest, device=DEV).repeat(batch, 1, 1)
    reach.scatter_(2, parent.clamp(min=0)[..., None], (parent >= 0).float()[..., None])
    reach += torch.eye(widest, device=DEV)
    for _ in range(max(1, widest.bit_length())):
        reach = (reach @ reach > 0).float()
    words = (widest + 31) // 32
    bits = torch.nn.functional.pad(reach > 0, (0, words * 32 - widest)).reshape(batch, widest, words, 32).long()
    packed = (bits << torch.arange(32, device=DEV)).sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int()
    c["mask"] = packed[torch.arange(widest, device=DEV)[None, :] < draft[:, None]].contiguous()
    return c


# ------------------------------------------------------------------ one pass
def run(s):
    return {"norm_rope": run_norm_rope, "kv8_store": run_store, "kv8_load": run_load, "kv8_decode": run_decode,
            "tree": run_tree}[s["op"]](s)


def run_norm_rope(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        args = (s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"], s["q_out"])
        if s["kv"] == "bf16":
            ra.ra_qk_norm_rope_store(*args, s["k_pool"], s["v_pool"], s["loc"], eps=s["eps"],
                                     interleaved=s["interleaved"])
            return s["q_out"], s["k_pool"], s["v_pool"]
        ra.ra_qk_norm_rope_kv8_store(*args, s["pool"], s["loc"], eps=s["eps"], interleaved=s["interleaved"])
        ra.ra_kv8_load(s["pool"], s["loc"], s["k_back"], s["v_back"])
        return s["q_out"], s["k_back"], s["v_back"]
    rot = s["rot"]
    cos, sin = s["cos_sin"][s["positions"].long()][:, None].split(rot // 2, -1)

    def norm_rope(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    s["q_out"].copy_(norm_rope(s["q"], s["q_weight"]))
    k, loc = norm_rope(s["k"], s["k_weight"]), s["loc"].long()
    if s["kv"] == "bf16":
        s["k_pool"][loc] = k.to(torch.bfloat16)
        s["v_pool"][loc] = s["v"]
        return s["q_out"], s["k_pool"], s["v_pool"]
    s["pool"][loc] = pack(k, s["v"].float())
    kb, vb = unpack(s["pool"][loc], s["hkv"], s["d"])
    return s["q_out"], s["k_back"].copy_(kb), s["v_back"].copy_(vb)


def run_store(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        ra.ra_kv8_store(s["pool"], s["k"], s["v"], s["loc"])
        ra.ra_kv8_load(s["pool"], s["loc"], s["k_back"], s["v_back"])
        return s["k_back"], s["v_back"]
    loc = s["loc"].long()
    s["pool"][loc] = pack(s["k"].float(), s["v"].float())
    k, v = unpack(s["pool"][loc], s["hkv"], s["d"])
    return s["k_back"].copy_(k), s["v_back"].copy_(v)


def run_load(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        ra.ra_kv8_load(s["pool"], s["loc"], s["k_back"], s["v_back"])
        return s["k_back"], s["v_back"]
    k, v = unpack(s["pool"][s["loc"].long()], s["hkv"], s["d"])
    return s["k_back"].copy_(k), s["v_back"].copy_(v)


def run_decode(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        if "ws" not in s:
            s["ws"] = torch.empty(ra.ra_decode_workspace_bytes(s["batch"], s["hq"], s["hkv"], s["d"],
                                                               s["table"].shape[1]), dtype=torch.uint8, device=DEV)
        ra.ra_kv8_decode_attention(s["pool"], s["q"], s["o"], s["table"], s["rpi"], s["lens"], num_kv_heads=s["hkv"],
                                   max_seq_len=s["table"].shape[1], sm_scale=s["scale"], workspace=s["ws"])
        return s["o"]
    batch, hq, hkv, d = s["batch"], s["hq"], s["hkv"], s["d"]
    table = s["table"][s["rpi"].long()]
    k, v = unpack(s["pool"][table.clamp(min=0).long()], hkv, d)
    seen = torch.arange(table.shape[1], device=DEV)[None, :] < s["lens"][:, None]
    x = torch.einsum("bhgd,blhd->bhgl", s["q"].float().reshape(batch, hkv, hq // hkv, d), k) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    y = torch.einsum("bhgl,blhd->bhgd", p / p.sum(-1, keepdim=True), v)
    return s["o"].copy_(y.reshape(batch, hq, d))


def run_tree(s):
    if own:
        import prefix_shared_kv_ra_gb300 as ra
        if "ws" not in s:
            s["ws"] = torch.empty(ra.ra_tree_workspace_bytes(s["batch"], s["total"], s["hq"], s["hkv"], s["d"],
                                                             **s["bounds"]), dtype=torch.uint8, device=DEV)
        ra.ra_tree_attention(s["k_pool"], s["v_pool"], s["q"], s["o"], s["table"], s["rpi"], s["prefix"], s["drafts"],
                             s["qo"], s["mask"], sm_scale=s["scale"], workspace=s["ws"], **s["bounds"])
        return s["o"]
    batch, hq, hkv, d, widest = s["batch"], s["hq"], s["hkv"], s["d"], s["bounds"]["max_draft_len"]
    table = s["table"][s["rpi"].long()]
    longest = table.shape[1]
    at = table.clamp(min=0).long()
    k, v = s["k_pool"][at].float(), s["v_pool"][at].float()
    # query rows padded to [batch, widest]; row t of request b is row qo[b] + t
    live = torch.arange(widest, device=DEV)[None, :] < s["drafts"][:, None]
    row = (s["qo"][:-1, None] + torch.arange(widest, device=DEV)).clamp(max=s["total"] - 1).long()
    q = s["q"][row].float().reshape(batch, widest, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)
    x = torch.matmul(q.reshape(batch, hkv, -1, d), k.permute(0, 2, 3, 1)) * s["scale"]
    pos = torch.arange(longest, device=DEV)[None, :] - s["prefix"][:, None]
    j = pos.clamp(0, widest - 1)
    word = torch.gather(s["mask"][row], 2, (j >> 5)[:, None, :].expand(-1, widest, -1).long())
    seen = (pos < 0)[:, None] | (((word >> (j & 31)[:, None]) & 1 > 0) & (pos < s["drafts"][:, None])[:, None])
    x = x.reshape(batch, hkv, widest, hq // hkv, longest).masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    y = torch.matmul(p.reshape(batch, hkv, -1, longest), v.permute(0, 2, 1, 3))
    y = y.reshape(batch, hkv, widest, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(batch, widest, hq, d)
    return s["o"].copy_(y[live])


# ------------------------------------------------------------------ what a pass cannot do without
def work(c):
    hkv, d = c["hkv"], c["d"]
    record = slot_bytes(hkv, d)
    if c["op"] == "norm_rope":
        n, hq = c["tokens"], c["hq"]
        b = n * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + 4 * c["rot"] + 8)
        b += n * (hkv * d * 4 if c["kv"] == "bf16" else 2 * record + hkv * d * 4)
        return dict(bytes=b, flops=n * (hq + hkv) * d * 8)
    if c["op"] == "kv8_store":
        return dict(bytes=c["tokens"] * (2 * hkv * d * 4 + 2 * record + 8), flops=c["tokens"] * hkv * d * 8)
    if c["op"] == "kv8_load":
        return dict(bytes=c["tokens"] * (hkv * d * 4 + record + 4), flops=c["tokens"] * hkv * d * 4)
    lens = context_lengths(c)
    if c["op"] == "kv8_decode":
        return dict(bytes=sum(lens) * (record + 4) + c["batch"] * c["hq"] * d * 4, flops=sum(lens) * c["hq"] * d * 4)
    drafts = draft_lengths(c)
    keys = sum(lens) + sum(drafts)
    seen = sum(drafts) * (sum(lens) / len(lens) + sum(drafts) / len(drafts) / 2)
    return dict(bytes=keys * (hkv * d * 4 + 4) + sum(drafts) * c["hq"] * d * 4, flops=seen * c["hq"] * d * 4)


# ------------------------------------------------------------------ the definitions in 64 bits
def code_values():
    """The 256 e4m3 values by their definition: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = torch.arange(256, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).double() / 8
    x = torch.where(e == 0, m * 2.0 ** -6, (1 + m) * torch.exp2(e.double() - 7))
    x = torch.where((b & 127) == 127, torch.full_like(x, math.nan), x)
    return torch.where(b >= 128, -x, x)


def nearest_codes(x):
    """Each 64-bit row's values rounded to what its 8-bit form stands for (ties to the even mantissa)."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e, torch.full_like(e, -118)).clamp(-118, 119)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def record_rows(rec, hkv, d):
    """K and V rows of records in 64 bits, by the byte each value and each exponent is at."""
    hpc = heads_per_block(hkv)
    h = torch.arange(hkv, device=DEV)
    block = h // hpc * (hpc * 2 * d + 16)
    first, tail = block + h % hpc * 2 * d, block + hpc * 2 * d + h % hpc * 2
    table, at = code_values(), first[:, None] + torch.arange(d, device=DEV)
    k = table[rec[:, at].long()] * torch.exp2(rec[:, tail].double() - 127)[..., None]
    v = table[rec[:, at + d].long()] * torch.exp2(rec[:, tail + 1].double() - 127)[..., None]
    return k, v


def attend(q, k, v, scale, seen=None):
    """q [t, hq, d] over k, v [l, hkv, d], all in 64 bits; seen [t, l] or None."""
    x = torch.einsum("tkgd,lkd->tkgl", q.unflatten(1, (k.shape[1], -1)), k) * scale
    if seen is not None:
        x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
    return torch.einsum("tkgl,lkd->tkgd", torch.softmax(x, -1), v).flatten(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    hkv, d = s["hkv"], s["d"]
    if s["op"] == "norm_rope":
        rot = s["rot"]
        angle = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(angle[:, None, :rot // 2], angle[:, None, rot // 2:])

        def rotated(x, w):
            x = x.double()
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + s["eps"]) * w.double()
            pairs = x[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
            pairs = pairs if s["interleaved"] else pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z if s["interleaved"] else z.transpose(-1, -2)
            return torch.cat([z.flatten(-2), x[..., rot:]], -1)

        q, k, v = rotated(s["q"], s["q_weight"]), rotated(s["k"], s["k_weight"]), s["v"].double()
        if s["kv"] == "e4m3":
            return q, nearest_codes(k), nearest_codes(v)
        pools = []
        for x in (k, v):
            pools.append(torch.zeros(s["k_pool"].shape, dtype=torch.float64, device=DEV))
            pools[-1][s["loc"].long()] = x
        return q, *pools
    if s["op"] == "kv8_store":
        return nearest_codes(s["k"].double()), nearest_codes(s["v"].double())
    if s["op"] == "kv8_load":
        return record_rows(s["pool"][s["loc"].long()], hkv, d)
    out = []
    if s["op"] == "kv8_decode":
        for b in range(s["batch"]):
            slots = s["table"][int(s["rpi"][b]), :int(s["lens"][b])].long()
            k, v = record_rows(s["pool"][slots], hkv, d)
            out.append(attend(s["q"][b:b + 1].double(), k, v, s["scale"]))
        return torch.cat(out)
    for b in range(s["batch"]):
        p, t, q0 = int(s["prefix"][b]), int(s["drafts"][b]), int(s["qo"][b])
        slots = s["table"][int(s["rpi"][b]), :p + t].long()
        words = s["mask"][q0:q0 + t].long() & 0xFFFFFFFF
        tree = (words[:, :, None] >> torch.arange(32, device=DEV) & 1).flatten(1)[:, :t] > 0
        seen = torch.cat([torch.ones(t, p, dtype=torch.bool, device=DEV), tree], 1)
        out.append(attend(s["q"][q0:q0 + t].double(), s["k_pool"][slots].double(), s["v_pool"][slots].double(),
                          s["scale"], seen))
    return torch.cat(out)
