"""Plain 64-bit forms (numpy) of the quantised-cache, norm + rotation and attention operators, and the error
bounds the GPU tests hold the kernels to."""
from __future__ import annotations

import numpy as np

EPS_BF16 = 2.0 ** -8   # half a step, relative to the value
EPS_F16 = 2.0 ** -11
EPS_F32 = 2.0 ** -24


def code_table() -> np.ndarray:
    """Value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = np.nan if (b & 127) == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t[b] = -x if b & 128 else x
    return t


CODES = code_table()
_POS = CODES[:127]  # ascending


def hpc_of(hkv: int) -> int:
    return max(h for h in range(1, 9) if hkv % h == 0)


def slot_bytes(hkv: int, d: int) -> int:
    hpc = hpc_of(hkv)
    return -(-(hkv // hpc) * (hpc * 2 * d + 16) // 32) * 32


def row_exponent(x: np.ndarray) -> np.ndarray:
    """Smallest e in [-118, 119] with max|finite x| <= 448 * 2^e (last axis)."""
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -118)
    for k in range(-118, 119):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    return e


def encode(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code (ties to the even code), saturating; NaN -> 0x7f."""
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_POS, np.where(np.isnan(a), 0, a), side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(a == _POS[hi], hi, c)
    return np.where(np.isnan(y), 0x7f, c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def pack(k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """K, V rows [n, hkv, d] (64-bit) -> records [n, slot_bytes]."""
    n, hkv, d = k.shape
    hpc = hpc_of(hkv)
    rec = np.zeros((n, slot_bytes(hkv, d)), np.uint8)
    for h in range(hkv):
        at = h // hpc * (hpc * 2 * d + 16)
        for i, x in enumerate((k[:, h], v[:, h])):
            e = row_exponent(x)
            c0 = at + (h % hpc) * 2 * d + i * d
            with np.errstate(invalid="ignore"):
                rec[:, c0:c0 + d] = encode(x * 2.0 ** -e[:, None].astype(np.float64))
            rec[:, at + hpc * 2 * d + 2 * (h % hpc) + i] = e + 127
    return rec


def unpack(rec: np.ndarray, hkv: int, d: int):
    """Records [..., slot_bytes] -> K, V rows [..., hkv, d] in 64 bits."""
    hpc = hpc_of(hkv)
    k, v = [], []
    for h in range(hkv):
        at = h // hpc * (hpc * 2 * d + 16)
        for i, out in enumerate((k, v)):
            c0, s0 = at + (h % hpc) * 2 * d + i * d, at + hpc * 2 * d + 2 * (h % hpc) + i
            out.append(CODES[rec[..., c0:c0 + d]] * 2.0 ** (rec[..., s0:s0 + 1].astype(np.float64) - 127))
    return np.stack(k, -2), np.stack(v, -2)


def attend(q, k, v, scale, seen=None):
    """Softmax attention in 64 bits: q [t, hq, d] over k, v [l, hkv, d], seen [t, l] or None.  Returns the
    output and the sums the error bound needs: A = sum_j p_j |v_j|, and per (row, head) the score magnitude
    X = max_j sum_d |q_d k_jd| * scale over the visible keys.  A row that sees nothing gives 0."""
    t, hq, d = q.shape
    g = hq // k.shape[1]
    kk, vv = np.repeat(k, g, 1), np.repeat(v, g, 1)
    x = np.einsum("thd,lhd->thl", q, kk) * scale
    mag = np.einsum("thd,lhd->thl", np.abs(q), np.abs(kk)) * scale
    if seen is not None:
        x = np.where(seen[:, None], x, -np.inf)
        mag = np.where(seen[:, None], mag, 0.0)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    total = p.sum(-1, keepdims=True)
    p = p / np.where(total > 0, total, 1.0)
    return np.einsum("thl,lhd->thd", p, vv), np.einsum("thl,lhd->thd", p, np.abs(vv)), mag.max(-1)


def attention_bound(ref, a, x, d, p_eps):
    """|kernel - ref| of an attention whose scores are fp32 sums of d products, whose weights are rounded
    with relative error p_eps before the PV product, and whose output is rounded to bf16.
      scores: |dx| <= (d + 4) * 2^-24 * X (d products and their sums, the scale, the subtraction of the
        reference, whose size X bounds too), plus the exponential's 2^-22: a weight's relative error r <=
        2 * dx + 2^-22, the same for the sum that divides, so 2 r A with dx in e-units;
      weights: p_eps * A; PV sums in fp32: folded into 2^-14 A (well over (n + d) * 2^-24 for n <= 2^9 blocks
        of accumulation, the chains being at most 2^9 long per 128 keys);
      output: 2^-8 |ref| (1 + small)."""
    r = 2 * (d + 4) * EPS_F32 * x[..., None] + 2.0 ** -22
    return 1.001 * EPS_BF16 * np.abs(ref) + (2 * r + p_eps + 2.0 ** -14) * a + 1e-30


def norm_rope(x, w, eps, angles, rot, interleaved):
    """x [n, h, d] -> normalised and rotated rows, and the magnitude its rounding errors scale with."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    c, s = angles[:, None, :rot // 2], angles[:, None, rot // 2:]
    y, mag = x.copy(), np.abs(x)
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) * np.abs(c) + np.abs(b) * np.abs(s) + np.abs(b) * np.abs(c) + \
        np.abs(a) * np.abs(s)
    return y, mag
