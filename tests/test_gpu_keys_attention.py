"""The window attention and the dense attention over the 4-bit cache against the
64-bit form, with the error bound of their arithmetic."""
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


def out_values(t):
    return ref.bf16(t.cpu().numpy().view(np.uint16))


def draw_rows(g, fp8, *shape):
    r = synth.swa_rows(g, *shape)
    return oracle.swa_fp8_quantize(r) if fp8 else r


def draw_entries(g, *shape):
    """Entries as the cache write leaves them: E2M1 pairs and E4M3 scales of 0.25 to 0.47."""
    kv = g.integers(0, 256, (*shape, 288), dtype=np.uint8)
    kv[..., 256:] = g.integers(0x28, 0x30, (*shape, 32), dtype=np.uint8)
    return kv


def check(got_o, got_l, q, keys, scale, u_p, what=""):
    o, l, b_o, b_l = ref.attend(q, keys, scale, u_p)
    if len(keys) == 0:
        assert np.all(got_o == 0) and np.all(got_l == -math.inf), what
        return
    assert np.all(np.isfinite(got_o)) and np.all(np.isfinite(got_l)), what
    assert np.all(np.abs(got_o - o) <= b_o), (what, np.max(np.abs(got_o - o) / b_o))
    assert np.all(np.abs(got_l - l) <= b_l), (what, np.max(np.abs(got_l - l) / b_l))


def run_window(q, rows, base, pos, W, sinks, scale=SCALE, status=0, ws=None, **kw):
    B, Q = pos.shape
    out = torch.full((B, Q, 64, 512), 0x4242, dtype=torch.int16, device="cuda")
    lse = torch.full((B, Q, 64), 42.0, device="cuda")
    ws = ws or csa2.Workspace(csa2.window_attn_workspace_size(B, Q, W, 0 if sinks is None else sinks.shape[1]))
    csa2.window_attn(up(q), up(rows), up(base), up(pos), scale, out, ws, W=W,
                     sinks=None if sinks is None else up(sinks), lse=lse, **kw)
    assert ws.sync_status()[0] == status
    return out_values(out), lse.cpu().double().numpy()


def verify_window(seed, B, Q, W, n_sink, fp8, pos, base, S, scale=SCALE, poison=True, status=0):
    g = synth.rng(seed)
    q = synth.main_queries(g, B, Q)
    rows = draw_rows(g, fp8, B, S)
    sinks = draw_rows(g, fp8, B, n_sink) if n_sink else None
    seen, seen_s = np.zeros((B, S), bool), np.zeros((B, max(1, n_sink)), bool)
    for b in range(B):
        for t in pos[b]:
            if t >= 0:
                lo = max(0, t - W + 1)
                seen[b, max(0, lo - base[b]):max(0, min(S, t + 1 - base[b]))] = True
                seen_s[b, :min(n_sink, lo)] = True
    if poison:                                          # what no query sees may hold anything
        rows[~seen] = NAN_E4M3 if fp8 else NAN_BF16
        if n_sink:
            sinks[~seen_s[:, :n_sink]] = NAN_E4M3 if fp8 else INF_BF16
    o, l = run_window(q, rows, base, pos, W, sinks, scale, status)
    for b in range(B):
        rv = ref.row_values(rows[b])
        sv = ref.row_values(sinks[b]) if n_sink else None
        for i in range(Q):
            keys = ref.window_keys(rv, int(base[b]), int(pos[b, i]), W, sv)
            check(o[b, i], l[b, i], ref.bf16(q[b, i]), keys, scale, ref.U_BF16, (b, i, pos[b, i]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Q,W,n_sink,start", [
    (1, 1, 1, 0, 0), (1, 1, 1, 1, 5), (2, 1, 128, 4, 0), (2, 1, 128, 4, 129), (3, 5, 128, 4, 126), (1, 7, 127, 3, 200),
    (1, 4, 129, 1, 1000), (2, 3, 33, 130, 90), (1, 2, 5, 300, 700), (1, 9, 400, 17, 250), (1, 3, 1000, 0, 2000),
    (2, 33, 64, 7, 3)])
def test_window_consecutive(fp8, B, Q, W, n_sink, start):
    pos = start + np.arange(Q)[None, :] + 11 * np.arange(B)[:, None]
    base = np.maximum(0, pos[:, 0] - W + 1)
    verify_window(1, B, Q, W, n_sink, fp8, pos, base, Q + W - 1 + 5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,n_sink", [(16, 4), (128, 4), (300, 2)])
def test_window_any_positions(fp8, W, n_sink):
    """Queries in any order, the same position twice, gaps, padding at the end and in the middle."""
    pos = np.array([[10, 9, 9, -1, 400, 401, 402, 405, 30, 31], [0, 1, 2, 3, 500, 499, 498, -1, -1, -5],
                    [-1] * 10, [510, 511, 0, 1, 255, 256, 3, 4, 100, 101]])
    verify_window(2, 4, 10, W, n_sink, fp8, pos, np.zeros(4, np.int64), 512)


@pytest.mark.parametrize("W,n_sink", [(1, 3), (50, 0), (128, 5)])
def test_window_neighbours_apart(W, n_sink):
    """Neighbouring queries whose windows touch, leave a small gap or lie in reverse order."""
    rows = []
    for t in (260, 130, 131):
        for d in (1, W - 1, W, W + 1, W + 7, W + 40, -1, -W + 1, -W, -W - 1, -W - 9):
            rows.append([t, max(0, t + d)])
    verify_window(14, len(rows), 2, W, n_sink, False, np.array(rows), np.zeros(len(rows), np.int64), 440)


def test_window_causal_neighbour_not_finite():
    """A row that the next query sees and this one does not may be infinite or NaN:
    this query's output stays finite, the next one's does not."""
    g = synth.rng(3)
    for fp8, bad in ((False, NAN_BF16), (False, INF_BF16), (True, NAN_E4M3)):
        pos = np.array([[99, 100, 101, 102, 103, 104]])
        rows, q = draw_rows(g, fp8, 1, 200), synth.main_queries(g, 1, 6)
        rows[0, 102, 7] = bad
        o, l = run_window(q, rows, np.zeros(1, np.int64), pos, 64, None)
        rv = ref.row_values(rows[0])
        for i in range(3):
            check(o[0, i], l[0, i], ref.bf16(q[0, i]), ref.window_keys(rv, 0, int(pos[0, i]), 64), SCALE, ref.U_BF16)
        assert np.all(np.isnan(o[0, 3:, :, 7]))
        # and one that has left the window
        pos = np.arange(160, 170)[None, :]
        q = synth.main_queries(g, 1, 10)
        o, l = run_window(q, rows, np.zeros(1, np.int64), pos, 64, None)
        for i in range(6, 10):
            check(o[0, i], l[0, i], ref.bf16(q[0, i]), ref.window_keys(rv, 0, int(pos[0, i]), 64), SCALE, ref.U_BF16)


def test_window_rows_not_supplied():
    pos = np.array([[50, 51]])
    for base, S in ((20, 32), (-10, 40), (60, 5), (0, 0), (1 << 40, 16), (-(1 << 40), 16)):
        verify_window(4, 1, 2, 40, 3, False, pos, np.array([base]), S, status=6)
    verify_window(4, 1, 2, 40, 3, True, pos, np.array([13]), 20, status=6)


def test_window_large_and_peaked_logits():
    """Logits far apart: the maximum grows chunk by chunk by more than e^8."""
    for W, n_sink in ((128, 4), (700, 20)):
        pos = np.array([[800, 801, 802]])
        g = synth.rng(5)
        q, rows = synth.main_queries(g, 1, 3), draw_rows(g, False, 1, 900)
        sinks = draw_rows(g, False, 1, n_sink)
        v = ref.bf16(rows) * (1 + np.arange(900)[None, :, None] / 90.0)
        rows = synth.f32_to_bf16_bits(v.astype(np.float32))
        for scale in (SCALE, 0.5, 4.0, -0.3, 0.0):
            o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W, sinks, scale)
            for i in range(3):
                keys = ref.window_keys(ref.row_values(rows[0]), 0, int(pos[0, i]), W, ref.row_values(sinks[0]))
                check(o[0, i], l[0, i], ref.bf16(q[0, i]), keys, scale, ref.U_BF16, (W, scale, i))


def test_window_split_over_ctas_and_many_queries():
    """One query over a wide window (its keys divided over many CTAs) and enough queries for one CTA each."""
    assert csa2.window_attn_workspace_size(1, 1, 4000, 5) > 256
    verify_window(6, 1, 1, 4000, 5, False, np.array([[9000]]), np.array([5001]), 4000)
    verify_window(6, 1, 1, 4000, 5, True, np.array([[1000]]), np.array([0]), 4000)
    assert csa2.window_attn_workspace_size(1, 640, 260, 5) == 256
    pos = np.arange(640)[None, :]
    verify_window(7, 1, 640, 260, 5, False, pos, np.array([0]), 640)


@pytest.mark.parametrize("kind", ["window", "window fp8", "ring", "ring fp8", "dense"])
def test_repeated_runs_are_identical(kind):
    """Many long runs of chunks on a warm cache, where copies arrive as early as they can:
    every repetition gives the same bits, and a sample of them is right."""
    g = synth.rng(21)
    fp8, Q, W = "fp8" in kind, 602, 120 if "ring" in kind else 1000
    rows, q = draw_rows(g, fp8, 1, Q + W - 1), synth.main_queries(g, 1, Q)
    pos = W + np.arange(Q)[None, :]
    base = np.ones(1, np.int64)
    dq, drows, dpos, dbase = up(q), up(rows), up(pos), up(base)
    out, lse = torch.empty(1, Q, 64, 512, dtype=torch.int16, device="cuda"), torch.empty(1, Q, 64, device="cuda")
    if kind == "dense":
        kv = draw_entries(g, 1, 1504)
        cache = make_cache(kv, [1500], 1)
        ws = csa2.Workspace(csa2.dense_attn_workspace_size(1, Q, 1504))
    else:
        ws = csa2.Workspace(csa2.window_attn_workspace_size(1, Q, W, 0))
    first = None
    for _ in range(20):
        if kind == "dense":
            csa2.dense_attn(cache, dq, drows, dbase, dpos, SCALE, out, ws, max_n=1504, lse=lse)
        else:
            csa2.window_attn(dq, drows, dbase, dpos, SCALE, out, ws, W=W, lse=lse)
        if first is None:
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert ws.sync_status()[0] == 0
    rv, o, l = ref.row_values(rows[0]), out_values(out), lse.cpu().double().numpy()
    for i in range(0, Q, 43):
        t = int(pos[0, i])
        keys = (ref.dense_keys(oracle.dequant_main(kv[0]), 1500, 1, rv, 1, t) if kind == "dense"
                else ref.window_keys(rv, 1, t, W))
        check(o[0, i], l[0, i], ref.bf16(q[0, i]), keys, SCALE, ref.U_F16 if kind == "dense" else ref.U_BF16, i)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Q,W,n_sink,start", [
    (1, 700, 128, 4, 0), (1, 609, 1, 0, 5), (1, 640, 1, 3, 1), (2, 333, 31, 0, 0), (3, 205, 100, 59, 40),
    (1, 611, 159, 0, 1000), (1, 650, 157, 2, 100), (20, 31, 64, 5, 3), (1, 620, 127, 1, 1 << 33)])
def test_window_many_queries(fp8, B, Q, W, n_sink, start):
    """Short windows of many neighbouring queries, with padding behind the shorter sequences."""
    pos = start + np.arange(Q)[None, :] + 7 * np.arange(B)[:, None]
    base = np.maximum(0, pos[:, 0] - W + 1)
    for b in range(1, B):
        pos[b, Q - 3 * b:] = -1
    verify_window(16, B, Q, W, n_sink, fp8, pos, base, Q + W - 1 + 3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Q,W,n_sink,start", [
    (1, 160, 32, 4, 0), (40, 8, 20, 3, 5), (152, 2, 9, 0, 100), (3, 100, 155, 0, 7), (160, 1, 3, 2, 0), (305, 1, 1, 0, 9),
    (7, 23, 128, 4, 60), (2, 77, 5, 154, 90)])
def test_window_one_or_two_tiles_a_cta(fp8, B, Q, W, n_sink, start):
    """Sizes about the one where the ring takes a call over; a CTA's run ends inside a sequence."""
    pos = start + np.arange(Q)[None, :] + 3 * (np.arange(B) % 5)[:, None]
    base = np.maximum(0, pos[:, 0] - W + 1)
    pos[1::3, Q // 2:] = -1
    verify_window(44, B, Q, W, n_sink, fp8, pos, base, Q + W - 1 + 2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,n_sink", [(40, 4), (128, 16), (159, 0)])
def test_window_many_queries_in_any_order(fp8, W, n_sink):
    """The same with jumps, repeated and descending positions, padding and rows that are missing."""
    g = synth.rng(17)
    pos = g.integers(0, 800, (2, 320))
    pos[0, 40:200] = 300 + np.arange(160)
    pos[0, 200:260] = 500 - np.arange(60)
    pos[1, 10:50] = np.repeat(np.arange(600, 620), 2)
    pos[1, 60:90] = 100 + 3 * np.arange(30)
    pos[1, 100:140] = np.where(np.arange(40) % 2, 200 + np.arange(40), 600 + np.arange(40))
    pos[g.random((2, 320)) < 0.1] = -1
    verify_window(18, 2, 320, W, n_sink, fp8, pos, np.array([0, 0]), 800)
    verify_window(19, 2, 320, W, n_sink, fp8, pos, np.array([250, -100]), 500, status=6)


def test_window_many_queries_not_finite():
    """Rows and sinks that are not finite among many queries: only who sees them is touched."""
    g = synth.rng(20)
    for fp8, bads in ((False, (NAN_BF16, INF_BF16, 0xFF80)), (True, (NAN_E4M3, 0xFF))):
        for W, n_sink in ((32, 4), (128, 4)):
            Q = 620
            pos = np.arange(Q)[None, :]
            rows, sinks, q = draw_rows(g, fp8, 1, Q), draw_rows(g, fp8, 1, n_sink), synth.main_queries(g, 1, Q)
            where = [(0, 3), (200, 7), (201, 500), (333, 0), (430, 511), (619, 5)]
            for n, (r, c) in enumerate(where):
                rows[0, r, c] = bads[n % len(bads)]
            sinks[0, 2, 9] = bads[0]                          # seen from position W + 2 on
            o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W, sinks)
            rv = ref.row_values(rows[0])
            for t in list(range(W + 2)) + [r + d for r, _ in where for d in (-2, -1)]:
                if not 0 <= t < Q or t >= W + 2:
                    continue
                keys = ref.window_keys(rv, 0, t, W, ref.row_values(sinks[0]))
                if np.all(np.isfinite(keys)):
                    check(o[0, t], l[0, t], ref.bf16(q[0, t]), keys, SCALE, ref.U_BF16, t)
                else:
                    assert np.any(np.isnan(o[0, t]))
            assert np.all(np.any(np.isnan(o[0, W + 2:]), axis=(1, 2)))
            # without the sink: the windows between the bad rows
            o, l = run_window(q, rows, np.zeros(1, np.int64), pos, W, None)
            seen = 0
            for t in range(Q):
                keys = ref.window_keys(rv, 0, t, W)
                if np.all(np.isfinite(keys)):
                    seen += 1
                    check(o[0, t], l[0, t], ref.bf16(q[0, t]), keys, SCALE, ref.U_BF16, t)
                else:
                    assert np.any(np.isnan(o[0, t]))
            assert seen > 60


@pytest.mark.parametrize("fp8", [False, True])
def test_window_bad_rows_everywhere_repeated(fp8):
    """Tiles with and without a bad row take turns (every ring warp has to agree which is which):
    each run ends, and gives the same bits."""
    g = synth.rng(41)
    B, Q, W = 3, 640, 60
    rows, q = draw_rows(g, fp8, B, Q), synth.main_queries(g, B, Q)
    for b, step in enumerate((61, 97, 3)):                    # some, few and no windows without one
        for n, r in enumerate(range(5, Q, step)):
            rows[b, r, (37 * n) % 512] = NAN_E4M3 if fp8 else NAN_BF16
    bad = np.isnan(ref.row_values(rows)).any(axis=-1)
    want = np.array([[bad[b, max(0, t - W + 1):t + 1].any() for t in range(Q)] for b in range(B)])
    q, rows, base = up(q), up(rows), up(np.zeros(B, np.int64))
    pos = up(np.broadcast_to(np.arange(Q), (B, Q)))
    ws = csa2.Workspace(csa2.window_attn_workspace_size(B, Q, W, 0))
    runs = [(torch.zeros(B, Q, 64, 512, dtype=torch.int16, device="cuda"), torch.zeros(B, Q, 64, device="cuda"))
            for _ in range(20)]
    for o, l in runs:
        csa2.window_attn(q, rows, base, pos, SCALE, o, ws, W=W, lse=l)
    assert ws.sync_status()[0] == 0
    np.testing.assert_array_equal(runs[0][1].isnan().any(dim=-1).cpu().numpy(), want)
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l.view(torch.int32), runs[0][1].view(torch.int32))


def run_dense(cache, q, rows, base, pos, max_n, scale=SCALE, status=0, stream=None):
    B, Q = pos.shape
    out = torch.full((B, Q, 64, 512), 0x4242, dtype=torch.int16, device="cuda")
    lse = torch.full((B, Q, 64), 42.0, device="cuda")
    ws = csa2.Workspace(csa2.dense_attn_workspace_size(B, Q, max_n))
    csa2.dense_attn(cache, up(q), up(rows), up(base), up(pos), scale, out, ws, max_n=max_n, lse=lse)
    assert ws.sync_status()[0] == status
    return out_values(out), lse.cpu().double().numpy()


def make_cache(kv, ns, m):
    B, cap = kv.shape[:2]
    cache = csa2.Cache(B, cap, m)
    cache.main_kv[:, :cap].copy_(up(kv))
    cache.n_entries.copy_(torch.tensor(ns, dtype=torch.int32))
    return cache


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Q,m,ns,last", [
    (1, 1, 1, [0], 0), (1, 1, 1, [1], 0), (1, 1, 2, [1], 0), (1, 2, 2, [1], 1), (2, 1, 1, [127, 128], None),
    (3, 1, 1, [129, 1, 300], None), (2, 5, 2, [200, 77], None), (1, 3, 1, [1500], None), (1, 40, 1, [700], None),
    (2, 4, 1, [600, 900], 350)])
def test_dense(fp8, B, Q, m, ns, last):
    g = synth.rng(8)
    cap = -(-max(ns) // 8) * 8 + 8
    kv = draw_entries(g, B, cap)
    ends = np.array([(n * m - 1) if last is None else last for n in ns])
    pos = ends[:, None] - (Q - 1) + np.arange(Q)[None, :]
    base = np.maximum(0, pos[:, 0] - 127)
    rows, q = draw_rows(g, fp8, B, Q + 127 + 3), synth.main_queries(g, B, Q)
    for b in range(B):                                  # behind the last entry and the last row: anything
        kv[b, min(ns[b], (pos[b].max() + 1) // m):] = 0x7F
        rows[b, max(0, pos[b].max() + 1 - base[b]):] = NAN_E4M3 if fp8 else NAN_BF16
    o, l = run_dense(make_cache(kv, ns, m), q, rows, base, pos, cap)
    for b in range(B):
        entries = oracle.dequant_main(kv[b, :ns[b]])
        rv = ref.row_values(rows[b])
        for i in range(Q):
            keys = ref.dense_keys(entries, ns[b], m, rv, int(base[b]), int(pos[b, i]))
            check(o[b, i], l[b, i], ref.bf16(q[b, i]), keys, SCALE, ref.U_F16, (b, i))


def test_dense_newest_entry_not_finite():
    """An entry whose stored scale is NaN, seen by the newer queries only (m = 2: by every second pair)."""
    g = synth.rng(15)
    for m, n in ((1, 300), (2, 200), (1, 5000)):
        kv, rows, q = draw_entries(g, 1, n), draw_rows(g, False, 1, 140), synth.main_queries(g, 1, 6)
        pos = n * m - 6 + np.arange(6)[None, :]
        bad = n - 3
        kv[0, bad, 270] = 0x7F
        base = np.array([pos[0, 0] - 127])
        o, l = run_dense(make_cache(kv, [n], m), q, rows, base, pos, n)
        entries, rv = oracle.dequant_main(kv[0]), ref.row_values(rows[0])
        for i in range(6):
            t = int(pos[0, i])
            if bad < min(n, (t + 1) // m):
                assert np.all(np.isnan(o[0, i])) and np.all(np.isnan(l[0, i]))
            else:
                check(o[0, i], l[0, i], ref.bf16(q[0, i]), ref.dense_keys(entries, n, m, rv, int(base[0]), t), SCALE,
                      ref.U_F16, (m, i))


def test_dense_one_cta_a_query_equals_the_split():
    """640 queries (one CTA each) and a few of them in a call of their own (keys divided over CTAs)."""
    g = synth.rng(9)
    kv, rows, q = draw_entries(g, 1, 1504), draw_rows(g, False, 1, 800), synth.main_queries(g, 1, 640)
    pos = 860 + np.arange(640)[None, :]
    base = np.array([733])
    cache = make_cache(kv, [1500], 1)
    assert csa2.dense_attn_workspace_size(1, 640, 1504) == 256
    o, l = run_dense(cache, q, rows, base, pos, 1504)
    entries, rv = oracle.dequant_main(kv[0]), ref.row_values(rows[0])
    for i in (0, 1, 2, 63, 64, 127, 300, 638, 639):
        keys = ref.dense_keys(entries, 1500, 1, rv, 733, int(pos[0, i]))
        check(o[0, i], l[0, i], ref.bf16(q[0, i]), keys, SCALE, ref.U_F16, i)
        o1, l1 = run_dense(cache, q[:, i:i + 1], rows, base, pos[:, i:i + 1], 1504)
        check(o1[0, 0], l1[0, 0], ref.bf16(q[0, i]), keys, SCALE, ref.U_F16, i)


@pytest.mark.parametrize("B,n,max_n", [(1, 9000, 9000), (4, 2500, 2500), (5, 2500, 2500), (12, 1200, 1200),
                                       (60, 900, 900), (1, 70, 9000), (1, 0, 9000), (6, 150, 40000), (50, 3, 30000)])
def test_dense_joins(B, n, max_n):
    """Few queries of many states, more queries of fewer, states without keys."""
    g = synth.rng(43)
    kv = draw_entries(g, B, max(8, -(-n // 8) * 8))
    q, rows = synth.main_queries(g, B, 1), draw_rows(g, False, B, 140)
    pos = np.full((B, 1), max(n, 139)) + np.arange(B)[:, None]
    base = pos[:, 0] - 139
    ns = [max(0, n - 3 * b) for b in range(B)]
    assert csa2.dense_attn_workspace_size(B, 1, max_n) > 256
    o, l = run_dense(make_cache(kv, ns, 1), q, rows, base, pos, max_n)
    for b in sorted({0, 1, B // 2, B - 1} & set(range(B))):
        keys = ref.dense_keys(oracle.dequant_main(kv[b]), ns[b], 1, ref.row_values(rows[b]), int(base[b]), int(pos[b, 0]))
        check(o[b, 0], l[b, 0], ref.bf16(q[b, 0]), keys, SCALE, ref.U_F16, b)


def test_dense_padding_positions_and_bounds():
    g = synth.rng(10)
    kv, rows, q = draw_entries(g, 2, 64), draw_rows(g, False, 2, 200), synth.main_queries(g, 2, 3)
    pos = np.array([[59, -1, 20], [-1, -1, -1]])
    cache = make_cache(kv, [60, 64], 1)
    o, l = run_dense(cache, q, rows, np.zeros(2, np.int64), pos, 64)
    for b in range(2):
        for i in range(3):
            keys = ref.dense_keys(oracle.dequant_main(kv[b]), [60, 64][b], 1, ref.row_values(rows[b]), 0, int(pos[b, i]))
            check(o[b, i], l[b, i], ref.bf16(q[b, i]), keys, SCALE, ref.U_F16, (b, i))
    # more entries than the cache holds: reported, the cache's are attended; fewer than none: none
    pos = np.array([[150], [150]])
    o, l = run_dense(make_cache(kv, [100, 64], 1), q[:, :1], rows, np.zeros(2, np.int64), pos, 64, status=6)
    for b in range(2):
        keys = ref.dense_keys(oracle.dequant_main(kv[b]), 64, 1, ref.row_values(rows[b]), 0, 150)
        check(o[b, 0], l[b, 0], ref.bf16(q[b, 0]), keys, SCALE, ref.U_F16, b)
    o, l = run_dense(make_cache(kv, [-3, 64], 1), q[:, :1], rows, np.zeros(2, np.int64), pos, 64)
    keys = ref.window_keys(ref.row_values(rows[0]), 0, 150, 128)
    check(o[0, 0], l[0, 0], ref.bf16(q[0, 0]), keys, SCALE, ref.U_F16)
    # max_n only plans the work
    for max_n in (0, 8, 1 << 20):
        o, l = run_dense(cache, q[:, :1], rows, np.zeros(2, np.int64), np.array([[63], [63]]), max_n)
        keys = ref.dense_keys(oracle.dequant_main(kv[1]), 64, 1, ref.row_values(rows[1]), 0, 63)
        check(o[1, 0], l[1, 0], ref.bf16(q[1, 0]), keys, SCALE, ref.U_F16, max_n)


def test_dense_growing_maxima():
    """Entries that grow along the cache: the running maximum moves in nearly every chunk."""
    g = synth.rng(11)
    n = 1400
    kv = draw_entries(g, 1, n)
    kv[0, :, 256:] = (0x20 + np.arange(n) // 32)[:, None]         # E4M3 scales 0.125 .. 5.5
    rows, q = draw_rows(g, False, 1, 200), synth.main_queries(g, 1, 2)
    pos, base = np.array([[n - 2, n - 1]]), np.array([n - 129])
    cache = make_cache(kv, [n], 1)
    for scale in (SCALE, 1.0, -0.2):
        o, l = run_dense(cache, q, rows, base, pos, 128, scale)      # few CTAs: long runs of chunks
        for i in range(2):
            keys = ref.dense_keys(oracle.dequant_main(kv[0]), n, 1, ref.row_values(rows[0]), int(base[0]), int(pos[0, i]))
            check(o[0, i], l[0, i], ref.bf16(q[0, i]), keys, scale, ref.U_F16, (scale, i))


def test_the_largest_positions_and_the_farthest_buffers():
    """Positions up to 2^63 - 1, and buffers that begin far before or behind every query."""
    g = synth.rng(42)
    top = (1 << 63) - 1
    for Q in (2, 460):                                        # one CTA a query, and the ring
        S = Q + 40
        for fp8 in (False, True):
            rows, q = draw_rows(g, fp8, 1, S), synth.main_queries(g, 1, Q)
            pos, base = top - Q + 1 + np.arange(Q)[None, :], np.array([top - S + 1])
            o, l = run_window(q, rows, base, pos, 41, None)
            rv = ref.row_values(rows[0])
            for i in range(0, Q, 51):
                first = int(pos[0, i]) - int(base[0])
                check(o[0, i], l[0, i], ref.bf16(q[0, i]), rv[max(0, first - 40):first + 1], SCALE,
                      ref.U_F16 if fp8 and Q == 2 else ref.U_BF16, i)
            for far, at in ((-top - 1, 50), (top, 50)):       # nothing of the window was supplied
                o, l = run_window(q, rows, np.array([far]), at + np.arange(Q)[None, :], 41, None, status=6)
                assert np.all(o == 0) and np.all(l == -math.inf)
    kv, ns = draw_entries(g, 1, 200), [200]
    rows, q = draw_rows(g, False, 1, 130), synth.main_queries(g, 1, 2)
    rv = ref.row_values(rows[0])
    for m in (1, 2):
        pos = np.array([[top - 1, top]])
        o, l = run_dense(make_cache(kv, ns, m), q, rows, np.array([top - 129]), pos, 200)
        for i in range(2):
            keys = np.concatenate([rv[1 + i:129 + i], oracle.dequant_main(kv[0])])
            check(o[0, i], l[0, i], ref.bf16(q[0, i]), keys, SCALE, ref.U_F16, (m, i))


def test_two_calls_at_once_another_stream_and_graphs():
    """Calls on two streams with a workspace each, and two graphs that share one and are replayed in turn."""
    g = synth.rng(12)
    kv, rows = draw_entries(g, 1, 1200), draw_rows(g, False, 1, 400)
    q = up(synth.main_queries(g, 1, 4))
    pos, base = torch.arange(1196, 1200, device="cuda")[None], torch.tensor([1000], device="cuda")
    cache, swa = make_cache(kv, [1200], 1), up(rows)
    n = max(csa2.dense_attn_workspace_size(1, 4, 1200), csa2.window_attn_workspace_size(1, 4, 180, 0))

    def dense(o, ws, **kw):
        csa2.dense_attn(cache, q, swa, base, pos, SCALE, o, ws, max_n=1200, **kw)

    def window(o, ws, **kw):
        csa2.window_attn(q, swa, base, pos, SCALE, o, ws, W=180, **kw)

    want, got = [torch.empty_like(q) for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    ws = [csa2.Workspace(n) for _ in range(2)]
    dense(want[0], ws[0])
    window(want[1], ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        dense(got[0], ws[0], stream=streams[0])
        window(got[1], ws[1], stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for call, o in ((dense, got[0]), (window, got[1])):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(o, ws[0])
            call(o, ws[0])
        graphs.append(graph)
    for o in got:
        o.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ws[0].sync_status()[0] == 0 and ws[1].sync_status()[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_the_layer_from_projections_to_outputs(fp8):
    """As a layer uses them: queries and window rows from the projections, the cache
    written, the dense attention over it, and a window-only layer beside it."""
    g = synth.rng(13)
    T, Q, n_sink = 640, 6, 4
    x = synth.latents(g, 1, T)
    cs = csa2.rope_table(T).cuda()
    ws = csa2.Workspace(max(csa2.dense_attn_workspace_size(1, Q, T), csa2.window_attn_workspace_size(1, Q, 128, n_sink)))
    cache = csa2.Cache(1, T, 1)
    w0, w1 = synth.compressor_weights(g)
    csa2.compress_quantize(cache, up(x), torch.zeros(1, dtype=torch.int64, device="cuda"), up(w0), up(w1), cs,
                           up(synth.index_projection(g)), ws)
    cache.n_entries.fill_(T)
    rows = torch.zeros(1, T, 512, dtype=torch.uint8 if fp8 else torch.int16, device="cuda")
    csa2.qk_norm_rope(torch.arange(T, device="cuda"), cs, ws, k=up(x)[0], rows=rows)
    q_in = synth.main_queries(g, Q)
    pos = torch.arange(T - Q, T, device="cuda")
    q = torch.empty(1, Q, 64, 512, dtype=torch.int16, device="cuda")
    csa2.qk_norm_rope(pos, cs, ws, q=up(q_in), q_out=q[0])
    base = torch.zeros(1, dtype=torch.int64, device="cuda")
    dense, win = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(2, 1, Q, 64, device="cuda")
    csa2.dense_attn(cache, q, rows, base, pos[None], SCALE, dense, ws, max_n=T, lse=lse[0])
    csa2.window_attn(q, rows, base, pos[None], SCALE, win, ws, W=128, sinks=rows[:, :n_sink].contiguous(), lse=lse[1])
    assert ws.sync_status()[0] == 0
    rv = ref.row_values(rows.cpu().numpy()[0] if fp8 else rows.cpu().numpy()[0].view(np.uint16))
    entries = oracle.dequant_main(cache.main_kv.cpu().numpy()[0])
    qv, l = out_values(q)[0], lse.cpu().double().numpy()
    for i in range(Q):
        t = T - Q + i
        check(out_values(dense)[0, i], l[0, 0, i], qv[i], ref.dense_keys(entries, T, 1, rv, 0, t), SCALE, ref.U_F16, i)
        check(out_values(win)[0, i], l[1, 0, i], qv[i], ref.window_keys(rv, 0, t, 128, rv[:n_sink]), SCALE, ref.U_BF16, i)
    # a selection of every entry gives the sparse attention the same keys
    few = csa2.Cache(1, 64, 1)
    few.main_kv.copy_(cache.main_kv[:, :64])
    few.n_entries.fill_(64)
    p1 = torch.tensor([[63]], device="cuda")
    sel = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 1, 64)
    a, b = torch.empty_like(q[:, :1]), torch.empty_like(q[:, :1])
    csa2.dense_attn(few, q[:, :1].contiguous(), rows, base, p1, SCALE, a, ws, max_n=64)
    ws2 = csa2.Workspace(csa2.decode_workspace_size(csa2.MODE_REUSE, 1, 1, 64, 8, 64))
    csa2.decode(csa2.MODE_REUSE, few, q_pos=p1, q=q[:, :1].contiguous(), swa=rows, swa_base_pos=base, scale=SCALE, sel=sel,
                out=b, ws=ws2, swa_fp8=fp8)
    va, vb = out_values(a)[0, 0], out_values(b)[0, 0]
    keys = np.concatenate([entries[:64], rv[:64]])
    bound = ref.attend(qv[0], keys, SCALE, ref.U_F16)[2]
    assert np.all(np.abs(va - vb) <= 2 * bound)


def test_offsets_past_32_bits_in_the_cache():
    """The second sequence of a cache of 4.3 GB a sequence, and the end of the first: entries
    far behind 2^32 bytes.  All entries but the last thousand are zeros (logits 0)."""
    g = synth.rng(22)
    cap, m = 15_000_008, 1
    cache = csa2.Cache(2, cap, m)
    assert cap * 288 > 1 << 32
    tail = draw_entries(g, 2, 1000)
    ns = [cap - 3, 1000]
    cache.main_kv[0, ns[0] - 1000:ns[0]].copy_(up(tail[0]))
    cache.main_kv[1, :1000].copy_(up(tail[1]))
    cache.n_entries.copy_(torch.tensor(ns, dtype=torch.int32))
    rows, q = draw_rows(g, False, 2, 128), synth.main_queries(g, 2, 1)
    pos = np.array([[ns[0] - 1], [999]])
    base = pos[:, 0] - 127
    o, l = run_dense(cache, q, rows, base, pos, cap)
    for b in range(2):
        far = oracle.dequant_main(tail[b])
        qv = ref.bf16(q[b, 0])
        keys = np.concatenate([far, ref.row_values(rows[b])])
        zeros = ns[b] - 1000                                  # each adds exp(0) to the sum
        logit = SCALE * (qv @ keys.T)
        e = np.exp(logit)
        total = e.sum(-1, keepdims=True) + zeros
        want = (e / total) @ keys
        # many terms of the sum: 2^-24 each at most, 64 at a time in one register
        tol = ref.U_BF16 * np.abs(want) + (2.0 ** -10 + zeros / 64 / 152 * 2.0 ** -24) * ((e / total) @ np.abs(keys)) + \
            1128 * 2.0 ** -25 * np.abs(keys).max() / total
        assert np.all(np.abs(o[b, 0] - want) <= tol)
        assert np.all(np.abs(l[b, 0] - np.log(total[:, 0])) <= 1e-3)


@pytest.mark.parametrize("Q", [3, 460])
def test_offsets_past_32_bits_in_the_rows(Q):
    """Window rows behind 2^32 bytes, for few queries and for many."""
    g = synth.rng(23)
    S, W = 4_300_000, 100
    assert (S - Q - W) * 1024 > 1 << 32
    rows = torch.zeros(1, S, 512, dtype=torch.int16, device="cuda")
    last = draw_rows(g, False, 1, Q + W)
    rows[0, S - Q - W:] = up(last)[0]
    q = synth.main_queries(g, 1, Q)
    pos, base = 7 + np.arange(S - Q, S)[None, :], np.array([7])
    out = torch.empty(1, Q, 64, 512, dtype=torch.int16, device="cuda")
    lse = torch.empty(1, Q, 64, device="cuda")
    ws = csa2.Workspace(csa2.window_attn_workspace_size(1, Q, W, 0))
    csa2.window_attn(up(q), rows, up(base), up(pos), SCALE, out, ws, W=W, lse=lse)
    assert ws.sync_status()[0] == 0
    o, l, rv = out_values(out), lse.cpu().double().numpy(), ref.row_values(last[0])
    for i in range(0, Q, 1 if Q < 10 else 51):
        check(o[0, i], l[0, i], ref.bf16(q[0, i]), ref.window_keys(rv, 7 + S - Q - W, int(pos[0, i]), W), SCALE, ref.U_BF16, i)


def test_offsets_past_32_bits_in_queries_and_outputs():
    """65,600 queries in one call: q and the output pass 2^32 bytes."""
    Q, W = 65_600, 20
    assert Q * 64 * 512 * 2 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty(1, Q, 64, 512, dtype=torch.bfloat16, device="cuda")
    q.normal_(generator=gen)
    rows = torch.randn(1, Q, 512, device="cuda", generator=gen).to(torch.float8_e4m3fn).view(torch.uint8)
    pos, base = torch.arange(Q, device="cuda")[None], torch.zeros(1, dtype=torch.int64, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, Q, 64, device="cuda")
    ws = csa2.Workspace(csa2.window_attn_workspace_size(1, Q, W, 0))
    csa2.window_attn(q, rows, base, pos, SCALE, out, ws, W=W, lse=lse)
    assert ws.sync_status()[0] == 0
    rv = ref.row_values(rows[0].cpu().numpy())
    for t in (0, 1, 30000, 32767, 32768, 65535, 65536, 65599):
        check(out[0, t].double().cpu().numpy(), lse[0, t].double().cpu().numpy(), q[0, t].double().cpu().numpy(),
              ref.window_keys(rv, 0, t, W), SCALE, ref.U_BF16, t)
    # one wide window over the same queries' buffer, two of them
    two = q[:, -2:].contiguous()
    o2, l2 = torch.empty_like(two), torch.empty(1, 2, 64, device="cuda")
    ws = csa2.Workspace(csa2.window_attn_workspace_size(1, 2, 900, 0))
    csa2.window_attn(two, rows, base, pos[:, -2:].contiguous(), SCALE, o2, ws, W=900, lse=l2)
    assert ws.sync_status()[0] == 0
    for i in range(2):
        check(o2[0, i].double().cpu().numpy(), l2[0, i].double().cpu().numpy(), two[0, i].double().cpu().numpy(),
              ref.window_keys(rv, 0, Q - 2 + i, 900), SCALE, ref.U_BF16, i)
