"""Attention with changed scores by its definition in 64 bits, with the bound of the kernels' rounding."""
import numpy as np

EPS_F32, EPS_BF16 = 2.0 ** -24, 2.0 ** -8


def attend(q, k, v, scale, pos, cap=0.0, slopes=None, window=0, first=None, full=0):
    """q [t, hq, d] at positions pos [t] over k, v [l, hkv, d]; first [t] or None.  Returns the output and a bound of
    |kernel - output|:
      score of a key: d products and their sums in fp32, (d + 4) 2^-24 sum |q k| scale (tanh's slope is at most 1); the cap
        1e-6 of its value (the polynomial 7e-7; beyond it 2^-22 of the cap, where the value is over 0.84 of it); the bias,
        the sum and the subtracted reference, itself as large as the largest score: 4 roundings of |s| + |bias| + |m|;
      weight: e^(its error), 2^-22 of the exponential, 2^-8 of its rounding to bf16 (the sum that divides is unrounded);
        weights below 2^-126 of the largest vanish;
      product and sums in fp32: 2^-14 of sum p |v|;  output: half a step of bf16."""
    t, hq, d = q.shape
    g = hq // k.shape[1]
    j = np.arange(k.shape[0])
    far = np.abs(pos[:, None] - j).astype(np.float64)
    low = np.zeros(t, np.int64) if first is None else np.maximum(first, 0)
    if window:
        low = np.maximum(low, pos - window + 1)
    seen = (j >= low[:, None]) & ((j <= pos[:, None]) | (j < full))
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    some = seen.any(1)
    for h in range(hq):
        kk, vv = np.where(seen.any(0)[:, None], k[:, h // g], 0.0), np.where(seen.any(0)[:, None], v[:, h // g], 0.0)
        s = q[:, h] @ kk.T * scale
        mag = np.abs(q[:, h]) @ np.abs(kk).T * scale
        if cap:
            s = cap * np.tanh(s / cap)
        bias = slopes[h] * far if slopes is not None else np.zeros_like(s)
        x = np.where(seen, s - bias, -np.inf)
        m = np.where(some, x.max(1, initial=-np.inf), 0.0)[:, None]
        p = np.exp(x - m)
        p /= np.where(some[:, None], p.sum(1, keepdims=True), 1.0)
        err = (d + 4) * EPS_F32 * mag + (1e-6 * np.abs(s) if cap else 0) + 4 * EPS_F32 * (np.abs(s) + np.abs(bias) + np.abs(m))
        w = p * (1.05 * err + 2.0 ** -22)
        y, a = p @ vv, p @ np.abs(vv)
        out[:, h] = y
        bound[:, h] = (w @ np.abs(vv) + w.sum(1)[:, None] * np.abs(y) + (EPS_BF16 + 2.0 ** -14) * a +
                       1.001 * EPS_BF16 * np.abs(y) + 1e-30)
    return out, bound
