"""Plain 64-bit forms of the norm and rotation of queries and window keys and of
the attention over every visible key, and the error bounds of their tests."""
import math

import numpy as np

import oracle

H, D, ROT = 64, 512, 64
U_BF16, U_F16, U_E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -4      # half a step, relative


def bf16(bits):
    return (np.ascontiguousarray(bits).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def row_values(rows):
    """Stored window rows (bf16 bits, or E4M3 bytes) in 64 bits."""
    return oracle._E4M3[rows] if rows.dtype == np.uint8 else bf16(rows)


def norm_rope(x, weight, cs, eps):
    """x [..., 512] in 64 bits; cs [32, 2] of its position."""
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight.astype(np.float64)
    y = y.copy()
    c, s = cs[:, 0].astype(np.float64), cs[:, 1].astype(np.float64)
    a, b = y[..., D - ROT::2].copy(), y[..., D - ROT + 1::2].copy()
    y[..., D - ROT::2], y[..., D - ROT + 1::2] = a * c - b * s, a * s + b * c
    return y


def norm_rope_bound(x, weight, cs, eps, u):
    """|computed - exact| per channel: binary32 arithmetic (16 squares a lane, five
    joins, a root, a division and at most five more operations: 32 roundings of
    2^-24 at most, on |a||c| + |b||s| in the tail), then one rounding of u."""
    y = np.abs(x) / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.abs(weight).astype(np.float64)
    mag = y.copy()
    c, s = np.abs(cs[:, 0]).astype(np.float64), np.abs(cs[:, 1]).astype(np.float64)
    a, b = y[..., D - ROT::2], y[..., D - ROT + 1::2]
    mag[..., D - ROT::2], mag[..., D - ROT + 1::2] = a * c + b * s, a * s + b * c
    arith = 32 * 2.0 ** -24 * mag
    exact = np.abs(norm_rope(x, weight, cs, eps))
    return arith + u * (exact + arith) + (2.0 ** -10 if u == U_E4M3 else 0.0)   # E4M3's smallest step is 2^-9


def attend(q, keys, scale, u_p):
    """One query: q [64][512] and its keys [n][512], 64 bits.  Returns the output,
    the lse and bounds of both.

    The bound of the output: the final rounding, u = 2^-8 of the value; every
    weight's rounding to 16 bits, u_p relative (f16 also 2^-25 absolute, of a sum
    of at least 2^-12: the reference lags a maximum by e^8 < 2^12 at most, and the
    weight of the largest key is then at least its share); 2^-12 for the
    exponentials and for binary32 sums.  A logit is a sum of 512 exact products in
    binary32 (2^-24 each, taken 32 times for the adder's order and truncation)."""
    n = keys.shape[0]
    if n == 0:
        return np.zeros((H, D)), np.full(H, -math.inf), np.zeros((H, D)), np.zeros(H)
    logit = scale * (q @ keys.T)
    size = abs(scale) * (np.abs(q) @ np.abs(keys).T)
    top = logit.max(-1, keepdims=True)
    e = np.exp(logit - top)
    total = e.sum(-1, keepdims=True)
    out = (e / total) @ keys
    lse = (top + np.log(total))[:, 0]
    d_logit = 32 * 2.0 ** -24 * size.max(-1) + 2.0 ** -22 * np.abs(logit).max(-1)
    spread = (e / total) @ np.abs(keys)
    tiny = n * 2.0 ** -25 * 2.0 ** 12 / total * np.abs(keys).max() * (u_p == U_F16) * 2.0 ** -11
    b_out = U_BF16 * np.abs(out) + (1 + U_BF16) * (u_p + 2.0 ** -12 + 2 * d_logit[:, None]) * spread + tiny + 2.0 ** -126
    return out, lse, b_out, d_logit + 2.0 ** -20 * (1 + np.abs(lse))


def window_keys(rows, base, t, W, sinks=None):
    """The keys a query at position t sees: rows [S][512] of positions base.., sinks [n][512]."""
    if t < 0:
        return np.zeros((0, D))
    lo = max(0, t - W + 1)
    parts = [rows[max(0, lo - base):max(0, t + 1 - base)]]
    if sinks is not None:
        parts.append(sinks[:min(len(sinks), lo)])
    return np.concatenate(parts)


def dense_keys(entries, n_entries, m, rows, base, t):
    if t < 0:
        return np.zeros((0, D))
    return np.concatenate([entries[:min(n_entries, (t + 1) // m)], window_keys(rows, base, t, 128)])
