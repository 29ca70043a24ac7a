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
