"""Precision and range of the window attention and of the dense attention: what a key of any
weight adds to the output, and queries and scores far from the ordinary."""
import math

import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
import oracle
import synth
from tests import keys_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(512)
NAN_BF16, NAN_E4M3, INF_BF16 = 0x7FC0, 0x7F, 0x7F80


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).cuda()


def bf16_bits(x):
    return synth.f32_to_bf16_bits(np.asarray(x, np.float32))


def draw_rows(g, fp8, *shape):
    r = synth.swa_rows(g, *shape)
    return oracle.swa_fp8_quantize(r) if fp8 else r


def as_rows(x, fp8):
    return oracle.swa_fp8_quantize(bf16_bits(x)) if fp8 else bf16_bits(x)


def run_window(q, rows, base, pos, W, sinks=None, scale=SCALE):
    B, Q = pos.shape
    out = torch.full((B, Q, 64, 512), 0x4242, dtype=torch.int16, device="cuda")
    lse = torch.full((B, Q, 64), 42.0, device="cuda")
    ws = csa2.Workspace(csa2.window_attn_workspace_size(B, Q, W, 0 if sinks is None else sinks.shape[1]))
    csa2.window_attn(up(q), up(rows), up(base), up(pos), scale, out, ws, W=W,
                     sinks=None if sinks is None else up(sinks), lse=lse)
    assert ws.sync_status()[0] == 0
    return ref.bf16(out.cpu().numpy().view(np.uint16)), lse.cpu().double().numpy()


def run_dense(kv, n, q, rows, base, pos, max_n, scale=SCALE):
    """kv [cap][288] on the GPU: a cache of one sequence."""
    Q = pos.shape[1]
    cache = csa2.Cache(1, kv.shape[0], 1)
    cache.main_kv[0, :kv.shape[0]].copy_(kv)
    cache.n_entries.fill_(n)
    out = torch.full((1, Q, 64, 512), 0x4242, dtype=torch.int16, device="cuda")
    lse = torch.full((1, Q, 64), 42.0, device="cuda")
    ws = csa2.Workspace(csa2.dense_attn_workspace_size(1, Q, max_n))
    csa2.dense_attn(cache, up(q), up(rows), up(base), up(pos), scale, out, ws, max_n=max_n, lse=lse)
    assert ws.sync_status()[0] == 0
    return ref.bf16(out.cpu().numpy().view(np.uint16)), lse.cpu().double().numpy()


def exact(q, keys, scale):
    """Output and lse of one query's heads [64][512] over keys [n][512], in 64 bits."""
    logit = scale * (q @ keys.T)
    top = logit.max(-1, keepdims=True)
    e = np.exp(logit - top)
    total = e.sum(-1, keepdims=True)
    return (e / total) @ keys, (top + np.log(total))[:, 0]


def check_rms(got, want):
    """Errors of many outputs are those of their rounding to bf16.

    The weights' roundings are independent of it and of one another.  At 11 bits (f16) a weight is
    off by an eighth of what the output's own rounding is off (2^-11 and 2^-8 at most, both spread
    alike), and more keys than one average out: the root of the mean squares grows by
    sqrt(1 + 1/64) = 1.008 at most.  At 8 bits it would grow by about sqrt(2), and a key left out of 1000
    alike adds 1/32 of an output.  The logits' errors (2^-20) and those of the sums are far below.
    The mean over the 32,768 or more outputs is itself known to about 0.5 %: 1.05 in all."""
    rounded = ref.bf16(bf16_bits(want.astype(np.float32)))
    own = np.sqrt(np.mean((rounded - want) ** 2))
    err = np.sqrt(np.mean((got - want) ** 2))
    assert err <= 1.05 * own, (err / own, own)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Q,W,n_sink,start", [
    (16, 1, 128, 4, 4095), (40, 3, 99, 0, 700), (1, 640, 128, 4, 1000), (160, 4, 30, 2, 50), (1, 2, 1000, 17, 3000),
    (1, 1, 4000, 5, 9000), (1, 320, 400, 3, 900)])
def test_window_errors_are_those_of_the_output(fp8, B, Q, W, n_sink, start):
    """One CTA a query, many queries over a ring, keys divided over CTAs."""
    g = synth.rng(61)
    pos = start + np.arange(Q)[None, :] + np.zeros((B, 1), np.int64)
    base = pos[:, 0] - W + 1
    q, rows = synth.main_queries(g, B, Q), draw_rows(g, fp8, B, Q + W - 1)
    sinks = draw_rows(g, fp8, B, n_sink) if n_sink else None
    o, _ = run_window(q, rows, base, pos, W, sinks)
    got, want = [], []
    for b in range(0, B, max(1, B // 8)):
        rv = ref.row_values(rows[b])
        for i in range(0, Q, max(1, Q // 8)):
            keys = ref.window_keys(rv, int(base[b]), int(pos[b, i]), W, ref.row_values(sinks[b]) if n_sink else None)
            got.append(o[b, i])
            want.append(exact(ref.bf16(q[b, i]), keys, SCALE)[0])
    check_rms(np.array(got), np.array(want))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Q", [3, 640])
def test_window_of_two_opposite_rows(fp8, Q):
    """Rows v, -v, v ..: an output is v times the difference of two weights near 1, which a weight
    of 8 bits (half a step below 1: 2^-9, of a sum of 2) gives up to 2^-10 off."""
    g = synth.rng(62)
    v = ref.row_values(draw_rows(g, True, 1))[0]
    rows = as_rows(np.where(np.arange(Q + 1)[:, None] % 2, -v, v), fp8)[None]
    q, scale = synth.main_queries(g, 1, Q), 0.03 * SCALE
    pos = 1 + np.arange(Q)[None, :]
    o, l = run_window(q, rows, np.zeros(1, np.int64), pos, 2, scale=scale)
    rv = ref.row_values(rows[0])
    for i in range(0, Q, max(1, Q // 20)):
        want, lse, tol, tol_l = ref.attend(ref.bf16(q[0, i]), rv[i:i + 2], scale, ref.U_F16 if fp8 else 2.0 ** -16)
        assert np.abs(want).max() < 0.5 * np.abs(v).max()
        assert np.all(np.abs(o[0, i] - want) <= tol), (i, np.max(np.abs(o[0, i] - want) / tol))
        assert np.all(np.abs(l[0, i] - lse) <= tol_l)


@pytest.mark.parametrize("n,max_n", [(1 << 17, 0), (1 << 17, 1 << 17), (1 << 20, 0), (70_001, 0)])
def test_dense_one_key_far_above_a_long_tail(n, max_n):
    """Entry 0 lies 12 to 23.8 (a head each) above all the others, which are alike: the others' share,
    alone in its dims, is N e^-gap / (1 + N e^-gap).  max_n = 0: one CTA walks the whole cache.

    Weights in f16 are exact to 2^-11 down to 2^-14, below to 2^-25, of a largest one of 2^8 or more
    (2^-33 each, N of them).  The tensor cores' sums of 16 products may lose 2^-23 of what is there
    each time, the softmax's sum 2^-24 for each run of 64 keys and lane; 2^-12 for the exponentials; the
    output's own rounding 2^-8."""
    kv = torch.zeros(n, 288, dtype=torch.uint8, device="cuda")
    kv[:, 256:] = 0x38                                        # scales 1
    kv[0, :128], kv[1:, 128:256] = 0x22, 0x22                 # 1 in dims 0 .. 255, in dims 256 .. 511
    row = np.zeros(512)
    row[256:] = 1.0
    rows = np.broadcast_to(bf16_bits(row), (1, 128, 512))
    q = np.zeros((1, 1, 64, 512))
    q[0, 0, :, :256] = (1 + np.arange(64) / 64)[:, None]
    o, l = run_dense(kv, n, bf16_bits(q), rows, np.array([n - 128]), np.array([[n - 1]]), max_n, 12 / 256)
    gap = 12 * (1 + np.arange(64) / 64)
    N = n - 1 + 128
    share = N * np.exp(-gap)
    total = 1 + share
    sums = N / 16 * 2.0 ** -23 + N / 64 * 2.0 ** -24
    tail = share / total
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + sums) * tail + N * 2.0 ** -33
    assert np.all(np.abs(o[0, 0, :, 256:] - tail[:, None]) <= tol[:, None]), \
        np.max(np.abs(o[0, 0, :, 256:] - tail[:, None]) / tol[:, None])
    assert np.all(np.abs(o[0, 0, :, :256] - (1 / total)[:, None]) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + sums) / total[:, None])
    assert np.all(np.abs(l[0, 0] - (gap + np.log(total))) <= sums + 2.0 ** -12 * tail + 2.0 ** -18)


def check_one_hot(o, q, keys, scale, what):
    """Logits of thousands and more: the output is the row of the largest one, wherever the next lies
    far below it (the logits' own error is 2^-19 of the sum of their products' sizes: 512 terms in binary32)."""
    logit, size = scale * (q @ keys.T), scale * (np.abs(q) @ np.abs(keys).T)
    order = np.sort(logit, -1)
    clear = order[:, -1] - order[:, -2] > 30 + 2.0 ** -18 * size.max(-1)
    assert clear.mean() > 0.5, what
    assert np.all(np.isfinite(o)), what
    top = keys[np.argmax(logit, -1)]
    assert np.all(np.abs(o - top)[clear] <= 2.0 ** -8 * np.abs(top)[clear] + 2.0 ** -30 * np.abs(keys).max()), what


@pytest.mark.parametrize("fp8", [False])
@pytest.mark.parametrize("Q,W", [(2, 64), (640, 64), (2, 700)])
@pytest.mark.parametrize("size", [1e4, 1e9, 1e12, 1e30])
def test_window_of_huge_queries(fp8, Q, W, size):
    """Queries far above f16's range, whichever kernel takes them."""
    g = synth.rng(63)
    rows = draw_rows(g, fp8, 1, Q + W - 1)
    q = bf16_bits(ref.bf16(synth.main_queries(g, 1, Q)) * size)
    pos = W - 1 + np.arange(Q)[None, :]
    o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W)
    rv = ref.row_values(rows[0])
    assert np.all(np.isfinite(l))
    for i in range(0, Q, max(1, Q // 20)):
        check_one_hot(o[0, i], ref.bf16(q[0, i]), rv[i:i + W], SCALE, (i, size))


@pytest.mark.parametrize("Q", [2, 640])
@pytest.mark.parametrize("size", [4e4, 1e6, 1e20, 1e35])
def test_window_range_of_q_over_e4m3_rows(Q, size):
    """A head's q of any size with a scale to match gives what the head of ordinary size gives."""
    g = synth.rng(64)
    W = 64
    rows = draw_rows(g, True, 1, Q + W - 1)
    small = ref.bf16(synth.main_queries(g, 1, Q))
    big = ref.bf16(bf16_bits(small * np.where(np.arange(64) % 3 == 1, size, 1.0)[:, None]))   # every third head
    pos = W - 1 + np.arange(Q)[None, :]
    rv = ref.row_values(rows[0])
    for scale, heads in ((SCALE, np.arange(64) % 3 != 1), (SCALE / size, np.arange(64) % 3 == 1)):
        o, l = run_window(bf16_bits(big), rows, np.zeros(1, np.int64), pos, W, scale=scale)
        assert np.all(np.isfinite(l[0][:, heads]))
        for i in range(0, Q, max(1, Q // 20)):
            want, lse, tol, tol_l = ref.attend(big[0, i], rv[i:i + W], scale, ref.U_F16)
            assert np.all(np.abs(o[0, i] - want)[heads] <= tol[heads]), (i, scale)
            assert np.all(np.abs(l[0, i] - lse)[heads] <= tol_l[heads])


@pytest.mark.parametrize("Q,W", [(2, 64), (640, 64), (2, 700)])
@pytest.mark.parametrize("size", [1e4, 1e9, 1e12, 1e30])
def test_huge_queries_over_e4m3_rows(Q, W, size):
    test_window_of_huge_queries(size=size, Q=Q, W=W, fp8=True)


@pytest.mark.parametrize("size", [1e5, 1e9, 1e30])
def test_huge_queries_over_the_cache(size):
    g = synth.rng(67)
    n = 700
    kv = g.integers(0, 256, (n, 288), dtype=np.uint8)
    kv[:, 256:] = g.integers(0x28, 0x30, (n, 32), dtype=np.uint8)
    rows, pos, base = draw_rows(g, False, 1, 130), np.array([[n - 3, n - 1, n - 2]]), np.array([n - 130])
    q = ref.bf16(synth.main_queries(g, 1, 3)) * np.where(np.arange(64) % 2, size, 1.0)[:, None]
    q[0, 1, :, 100:] /= size                                  # large and small dims in a head
    q = bf16_bits(q)
    o, l = run_dense(torch.from_numpy(kv).cuda(), n, q, rows, base, pos, n)
    entries, rv, odd = oracle.dequant_main(kv), ref.row_values(rows[0]), np.arange(64) % 2 == 1
    for i in range(3):
        keys, qv = ref.dense_keys(entries, n, 1, rv, int(base[0]), int(pos[0, i])), ref.bf16(q[0, i])
        check_one_hot(o[0, i][odd], qv[odd], keys, SCALE, (i, size))
        want, lse, tol, tol_l = ref.attend(qv, keys, SCALE, ref.U_F16)
        # heads of ordinary size beside them (f16 below 2^-14: 2^-25 of each product's q)
        tol += 2 * SCALE * 2.0 ** -25 * np.abs(keys).sum(-1).max() * np.abs(keys).max()
        assert np.all(np.abs(o[0, i] - want)[~odd] <= tol[~odd]), i


@pytest.mark.parametrize("Q", [2, 640])
def test_queries_that_are_not_finite_over_e4m3_rows(Q):
    """A head's infinity or NaN stays in that head, whatever the sizes of the others."""
    g = synth.rng(68)
    W = 40
    rows = draw_rows(g, True, 1, Q + W - 1)
    q = ref.bf16(synth.main_queries(g, 1, Q))
    q[0, :, 1::4] *= 1e20
    q[0, :, 5, 17], q[0, :, 6, 300] = np.inf, np.nan
    q[0, :, 9, 511] = -np.inf
    q = bf16_bits(q)
    pos = W - 1 + np.arange(Q)[None, :]
    o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W)
    rv, plain = ref.row_values(rows[0]), np.arange(64) % 4 != 1
    assert np.all(np.isnan(o[0, :, [5, 6, 9]]))
    plain[6] = False
    for i in range(0, Q, max(1, Q // 20)):
        want, lse, tol, tol_l = ref.attend(np.where(plain[:, None], ref.bf16(q[0, i]), 0.0), rv[i:i + W], SCALE, ref.U_F16)
        assert np.all(np.abs(o[0, i] - want)[plain] <= tol[plain])
        assert np.all(np.abs(l[0, i] - lse)[plain] <= tol_l[plain])


@pytest.mark.parametrize("kind", ["window", "dense"])
def test_scores_that_grow_by_the_last_bit(kind):
    """Scores (in powers of two) about 1.25 * 2^27, where neighbouring floats are 16 apart, growing by
    one step from one run of 64 keys to the next: a weight of 2^16 would be infinite in f16.  All keys
    are alike but for dim 256, which holds 0 .. 3."""
    row = np.zeros((256, 512))
    row[:, :256] = 1.0
    row[:, 256] = np.arange(256) // 64
    q = np.zeros((1, 1, 64, 512))
    q[..., :256], q[..., 256] = 40960.0, 1.0                 # 1.25 * 2^23 + 0 .. 3
    scale = 16 * math.log(2)
    pos = np.array([[255]])
    if kind == "window":                                      # enough queries for one CTA each
        q, pos = np.repeat(q, 305, 1), np.repeat(pos, 305, 1)
        o, l = run_window(bf16_bits(q), as_rows(row, True)[None], np.zeros(1, np.int64), pos, 256, scale=scale)
    else:
        kv = np.zeros((256, 288), np.uint8)
        kv[:, 256:], kv[:, :128] = 0x38, 0x22
        kv[:, 128] = np.array([0, 2, 4, 5])[np.arange(256) // 64]      # 0, 1, 2, 3
        near = np.zeros((1, 128, 512))                       # the window: scores of 0
        o, l = run_dense(torch.from_numpy(kv).cuda(), 256, bf16_bits(q), bf16_bits(near), np.array([128]), pos, 0, scale)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
    assert np.all(np.abs(o[..., :256] - 1) <= 2.0 ** -8)
    assert np.all((o[..., 256] >= 0) & (o[..., 256] <= 3)) and np.all(o[..., 257:] == 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_window_bad_rows_beside_finite_sinks(fp8):
    """Rows that are not finite among many queries with sinks: each query takes what it sees, and no more."""
    g = synth.rng(65)
    bads = (NAN_E4M3, 0xFF) if fp8 else (NAN_BF16, INF_BF16, 0xFF80)
    for W, n_sink in ((32, 4), (128, 16)):
        Q = 620
        pos = np.arange(Q)[None, :]
        rows, sinks, q = draw_rows(g, fp8, 1, Q), draw_rows(g, fp8, 1, n_sink), synth.main_queries(g, 1, Q)
        for n, (r, c) in enumerate([(0, 3), (200, 7), (201, 500), (333, 0), (430, 511), (619, 5)]):
            rows[0, r, c] = bads[n % len(bads)]
        o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W, sinks)
        rv, sv = ref.row_values(rows[0]), ref.row_values(sinks[0])
        finite = 0
        for t in range(Q):
            keys = ref.window_keys(rv, 0, t, W, sv)
            if np.all(np.isfinite(keys)):
                finite += 1
                want, lse, tol, tol_l = ref.attend(ref.bf16(q[0, t]), keys, SCALE, 2.0 ** -11)
                assert np.all(np.abs(o[0, t] - want) <= tol), t
                assert np.all(np.abs(l[0, t] - lse) <= tol_l), t
            else:
                assert np.any(np.isnan(o[0, t])), t
        assert finite > 60


@pytest.mark.parametrize("n,Q,max_n", [(1500, 320, 1500), (1500, 2, 1500), (9000, 2, 0)])
def test_dense_errors_are_those_of_the_output(n, Q, max_n):
    g = synth.rng(66)
    kv = g.integers(0, 256, (n, 288), dtype=np.uint8)
    kv[:, 256:] = g.integers(0x28, 0x30, (n, 32), dtype=np.uint8)
    rows, q = draw_rows(g, False, 1, Q + 127), synth.main_queries(g, 1, Q)
    pos = n - Q + np.arange(Q)[None, :]
    base = pos[:, 0] - 127
    o, _ = run_dense(torch.from_numpy(kv).cuda(), n, q, rows, base, pos, max_n)
    entries, rv = oracle.dequant_main(kv), ref.row_values(rows[0])
    some = list(range(0, Q, max(1, Q // 8)))
    want = [exact(ref.bf16(q[0, i]), ref.dense_keys(entries, n, 1, rv, int(base[0]), int(pos[0, i])), SCALE)[0] for i in some]
    check_rms(o[0, some], np.array(want))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Q,W", [(640, 60), (3, 2000), (16, 128)])
def test_calls_in_a_row_read_what_the_one_before_wrote(fp8, Q, W):
    """Rows and queries made by one call and read by the next, again and again over the same buffers
    (each call may start beside the end of the one before): the bits of calls that are waited for."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    S, n = Q + W - 1, 12
    k = torch.randn(n, S, 512, device="cuda", generator=gen).bfloat16()
    q = torch.randn(n, Q, 64, 512, device="cuda", generator=gen).bfloat16()
    cs, pos, base = csa2.rope_table(S).cuda(), torch.arange(S, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    rows = torch.zeros(1, S, 512, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    mine = torch.zeros(1, Q, 64, 512, dtype=torch.bfloat16, device="cuda")
    ws = csa2.Workspace(csa2.window_attn_workspace_size(1, Q, W, 0))
    got = []
    for wait in (False, True):
        out, lse = torch.zeros(n, 1, Q, 64, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 1, Q, 64, device="cuda")
        torch.cuda.synchronize()
        for i in range(n):
            for call in (lambda: csa2.qk_norm_rope(pos, cs, ws, k=k[i], rows=rows),
                         lambda: csa2.qk_norm_rope(pos[W - 1:], cs, ws, q=q[i], q_out=mine[0]),
                         lambda: csa2.window_attn(mine, rows, base, pos[None, W - 1:], SCALE, out[i], ws, W=W, lse=lse[i])):
                call()
                if wait:
                    torch.cuda.synchronize()
        got.append((out, lse))
    assert ws.sync_status()[0] == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not torch.equal(got[0][0][0], got[0][0][1])
