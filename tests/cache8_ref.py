"""Plain 64-bit forms of the 8-bit cache, of gathered attention weights and of the
eviction, and the error bounds of their tests."""
import numpy as np

from tests import keys_ref as ref

H, D, BLK = 64, 512, 8
FLOOR = 2.0 ** -60
BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127


def write(codes, scales, n_entries, x, start, n_new):
    """codes [B][cap][512] int8, scales [B][cap / 8] float32, x [B][T][512] in 64 bits: both after the call."""
    codes, scales = codes.copy(), scales.copy()
    x = np.where(np.isnan(x), 0.0, np.clip(x, -BF16_MAX, BF16_MAX))
    B, cap, _ = codes.shape
    for b in range(B):
        count = min(max(int(n_new[b]), 0), x.shape[1])
        lo, hi = max(int(start[b]), 0), min(int(start[b]) + count, cap)
        for r in range(lo // BLK, -(-hi // BLK)) if lo < hi else []:
            entries = range(BLK * r, BLK * r + BLK)
            fresh = [e for e in entries if lo <= e < hi]
            kept = [e for e in entries if e < lo or hi <= e < min(int(n_entries[b]), cap)]
            rows = x[b, [e - int(start[b]) for e in fresh]]
            s = np.float32(max(np.abs(rows).max() / 127.0, FLOOR))
            old = scales[b, r]
            if kept:
                s = max(s, old)
            codes[b, fresh] = np.rint(rows / np.float64(s))
            if kept:
                codes[b, kept] = np.rint(codes[b, kept] * np.float64(old) / np.float64(s))
            scales[b, r] = s
    return codes, scales


def entries(codes, scales):
    """Entries of one sequence [cap][512] in 64 bits."""
    return codes.astype(np.float64) * scales.astype(np.float64).repeat(BLK)[:, None]


def attend(q, keys, scale, most):
    """keys_ref.attend for f16 operands over keys of which some are codes times scales of `most` at the
    largest.  A weight goes to the second product as f16(P s): off by 2^-11 of itself, or by 2^-25 where f16 has
    fewer bits.  The key with the largest P s has 2^8 of it or more, so the sum of the P is at least 2^8 / s, and n
    weights of codes up to 127 (rows: s = 1, and their own size) add n 2^-25 127 s / 2^8 at most."""
    out, lse, b_out, b_lse = ref.attend(q, keys, scale, ref.U_F16)
    if keys.shape[0]:
        b_out = b_out + keys.shape[0] * 2.0 ** -33 * max(127 * most, np.abs(keys).max())
    return out, lse, b_out, b_lse


def gathered(q, keys, lse, scale):
    """What one query (q [64][512], lse [64]) adds to the entries it sees (keys [n][512]), and a bound.

    A weight is 2^(S f - l): S a sum of 512 exact products in binary32 (2^-24 each, taken 32 times for the adder's
    order and truncation) of q rounded to f16 (exact from 2^-14 on, 2^-25 below), f and l and their difference rounded
    to 24 bits (2^-21 of |logit| + |lse| for all of them), the exponential to 2^-22.  Sums: 20 additions for 64
    heads, 33 for splits, the rest compensated: 2^-18 of the sum."""
    with np.errstate(invalid="ignore"):
        live = lse > -np.inf
    q, lse = q[live], lse[live]
    logit = scale * (keys @ q.T)
    p = np.exp(logit - lse)
    rel = (32 * 2.0 ** -24 * abs(scale) * (np.abs(keys) @ np.abs(q).T) + 2.0 ** -21 * (np.abs(logit) + np.abs(lse) + 1)
           + 2.0 ** -25 * abs(scale) * np.abs(keys).sum(-1, keepdims=True))
    # p (e^rel - 1), written so that a weight of 0 with any rel has its bound
    return p.sum(-1), (np.exp(logit - lse + rel) - p).sum(-1) + 2.0 ** -18 * p.sum(-1) + 64 * 2.0 ** -126


def evicted(w, n, unit, budget, first, recent):
    """Numbers of the units of one sequence that stay (w: its weights, n entries), and the entries."""
    units, K = -(-n // unit), budget // unit
    worth = np.full(units, -np.inf)
    nan = np.zeros(units, bool)
    for u in range(units):
        part = w[u * unit:min(n, u * unit + unit)].astype(np.float64)
        nan[u] = np.all(np.isnan(part))
        worth[u] = -np.inf if nan[u] else np.nanmax(part)
    must = np.zeros(units, bool)
    must[:-(-first // unit)] = True
    if recent:
        must[max(0, n - recent) // unit:] = True
    order = np.lexsort((np.arange(units), -worth, nan, ~must))
    kept = np.sort(order[:K])
    entries = (kept[:, None] * unit + np.arange(unit)).ravel()
    return kept, entries[entries < n]
