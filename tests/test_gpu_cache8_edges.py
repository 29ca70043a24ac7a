"""The 8-bit cache where its calls can go wrong between CTAs and at the ends of their ranges."""
import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
from tests import cache8_ref as c8
from tests.test_gpu_cache8 import SCALE, attend_and_check, attn_case, cache_of, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Q,n,W,fp8", [(152, 1300, 128, True), (60, 3000, 0, False), (300, 1300, 200, False)])
def test_attention_pairs_read_what_the_other_cta_wrote(Q, n, W, fp8):
    """Each CTA of a pair widens half of the dims of every key, and one of them issues the products of both: the
    same bits from every call, alone and beside a call that keeps the GPU's memory busy."""
    pos = n - Q + np.arange(Q)[None, :]
    codes, scales, q, rows, base = attn_case(31, 1, Q, -(-n // 8) * 8, [n], 1, W, fp8, pos)
    out, lse = attend_and_check(codes, scales, [n], 1, q, rows, base, pos, W)
    cache, qd, pd = cache_of(codes, scales, [n]), q.cuda(), dev(pos)
    rd, bd = (rows.cuda(), dev(base)) if W else (None, None)
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(1, Q, n, W))
    a = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    b, beside = torch.zeros_like(a), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(40):
        got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)
        if i % 2:
            with torch.cuda.stream(beside):
                b.copy_(a)
        csa2.cache8_attn(cache, qd, pd, SCALE, got, ws, max_n=n, W=W, swa=rd, swa_base_pos=bd, lse=got_lse)
        assert torch.equal(got, out) and torch.equal(got_lse, lse), i
    torch.cuda.synchronize()
    assert ws.sync_status()[0] == 0


@pytest.mark.parametrize("B,Q,n", [(76, 2, 600), (5, 9, 100), (1, 152, 1300)])
def test_pairs_one_behind_another(B, Q, n):
    """A CTA of a pair ends when nothing is on its way to it: calls follow each other without a pause, on SMs whose
    shared memory the next one takes at once."""
    pos = n - Q + np.repeat(np.arange(Q)[None, :], B, 0)
    codes, scales, q, _, _ = attn_case(32, 1, Q, -(-n // 8) * 8, [n], 1, 0, False, pos[:1])
    cache = cache_of(codes.repeat(B, 0), scales.repeat(B, 0), [n] * B)
    qd, pd = q.repeat(B, 1, 1, 1).cuda(), dev(pos)
    ws = csa2.Workspace(max(csa2.cache8_attn_workspace_size(B, Q, n), csa2.attn_weights_workspace_size(B, Q, n)))
    calls = []
    for _ in range(30):
        out, lse = torch.zeros_like(qd), torch.zeros(B, Q, 64, device="cuda")
        w = torch.zeros(B, cache.cap, device="cuda")
        csa2.cache8_attn(cache, qd, pd, SCALE, out, ws, max_n=n, lse=lse)
        csa2.attn_weights(cache, qd, pd, lse, SCALE, w, ws, max_n=n)
        csa2.attn_weights(cache, qd, pd, lse, SCALE, w, ws, max_n=n, prev=w)
        calls.append((out, lse, w))
    assert ws.sync_status()[0] == 0
    for got in calls[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got, calls[0]))
    # all sequences are alike, and every query spreads its 64 heads' weights, twice (lse off by 2^-20 (1 + |lse|))
    assert torch.equal(calls[0][0], calls[0][0][:1].expand_as(qd)) and torch.equal(calls[0][2], calls[0][2][:1].expand(B, -1))
    total = calls[0][2].double().sum(1)
    assert torch.all((total - 128 * Q).abs() <= 1e-4 * 128 * Q)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [0, 1300])
def test_attention_pairs_tell_each_other_of_rows_that_are_not_finite(n, fp8):
    """Either half of the dims (a CTA each), met by the last chunk or long before the end: exactly the queries that
    see the row become NaN."""
    Q, W = 152, 40
    pos = 1200 + np.arange(Q)[None, :]
    codes, scales, q, rows, base = attn_case(33, 1, Q, 1304, [n], 1, W, fp8, pos)
    cache, qd, pd, bd = cache_of(codes, scales, [n]), q.cuda(), dev(pos), dev(base)
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(1, Q, 1300, W))
    for at in (1200, 1201, 1350, 1351):                # seen by both queries of its pair, by the second alone, by the last two, one
        for dim in (3, 255, 256, 511):
            bad = rows.clone()
            bad[0, at - int(base[0]), dim] = 0x7F if fp8 else float("inf" if dim == 3 else "nan")
            out, lse = torch.zeros_like(qd), torch.zeros(1, Q, 64, device="cuda")
            csa2.cache8_attn(cache, qd, pd, SCALE, out, ws, max_n=1300, W=W, swa=bad.cuda(), swa_base_pos=bd, lse=lse)
            sees = torch.from_numpy((pos[0] >= at) & (pos[0] < at + W)).cuda()
            assert torch.equal(torch.isnan(out[0].float()).all(-1).all(-1), sees), (at, dim)
            assert torch.equal(torch.isnan(out[0].float()).any(-1).any(-1), sees), (at, dim)
            assert torch.equal(torch.isnan(lse[0]).all(-1), sees) and torch.equal(torch.isnan(lse[0]).any(-1), sees)
    assert ws.sync_status()[0] == 0


@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("Q,n,max_n", [(1, 200, 200), (2, 200, 200), (1, 3000, 3000), (152, 1300, 1300), (60, 3000, 3000)])
def test_attention_at_the_last_positions_without_a_window(Q, n, max_n, m):
    """2^63 - 1 has no successor: a CTA a query or pairs, divided over CTAs or not."""
    top = (1 << 63) - 1
    pos = np.array([[top - i for i in range(Q)]], np.int64)
    codes, scales, q, _, _ = attn_case(34, 1, Q, -(-n // 8) * 8, [n], m, 0, False, np.zeros((1, Q), np.int64))
    attend_and_check(codes, scales, [n], m, q, None, None, pos, 0, max_n=max_n)


@pytest.mark.parametrize("Q,n,W,max_n", [(60, 2992, 20, 1300), (60, 2992, 20, 2000), (152, 1300, 20, 500)])
def test_attention_pairs_of_more_entries_than_their_split_was_made_for(Q, n, W, max_n):
    """Calls that take pairs (test_cache8_abi.py has the plan) over more chunks than max_n lets them expect."""
    pos = n - Q + np.arange(Q)[None, :]
    case = attn_case(35, 1, Q, -(-n // 8) * 8, [n], 1, W, False, pos)
    attend_and_check(*case[:2], [n], 1, *case[2:], pos, W, max_n=max_n)


@pytest.mark.parametrize("B,Q,n,W", [(300, 1, 90, 0), (40, 3, 100, 20), (1, 1, 600, 0), (2, 76, 1300, 9)])
def test_attention_of_padded_batches(B, Q, n, W):
    """Padded queries, whatever their q holds, give zeros; the others what they give in a batch without padding."""
    pos = n - Q + np.repeat(np.arange(Q)[None, :], B, 0)
    codes, scales, q, rows, base = attn_case(36, B, Q, -(-n // 8) * 8, [n] * B, 1, W, False, pos)
    cache, bd = cache_of(codes, scales, [n] * B), dev(base) if W else None
    pad = np.random.default_rng(36).random((B, Q)) < 0.5
    pad[0, 0] = True
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(B, Q, n, W))
    got = []
    for padded in (False, True):
        qd, p = q.cuda(), pos.copy()
        if padded:
            qd[torch.from_numpy(pad).cuda()] = float("nan")
            p[pad] = -1
        out, lse = torch.full_like(qd, 3.0), torch.full((B, Q, 64), 3.0, device="cuda")
        csa2.cache8_attn(cache, qd, dev(p), SCALE, out, ws, max_n=n, W=W, swa=rows.cuda() if W else None, swa_base_pos=bd, lse=lse)
        got.append((out, lse))
    assert ws.sync_status()[0] == 0
    at = torch.from_numpy(pad).cuda()
    assert torch.all(got[1][0][at] == 0) and torch.all(got[1][1][at] == -float("inf"))
    assert torch.equal(got[1][0][~at], got[0][0][~at]) and torch.equal(got[1][1][~at], got[0][1][~at])


@pytest.mark.parametrize("Q,n", [(1, 300), (152, 1300)])
@pytest.mark.parametrize("power", [-52, 80])
def test_scales_at_the_ends_of_their_range(power, Q, n):
    """Scales from 2^-60 to 2^80, with softmax scales that bring the scores back: attention and weights."""
    pos = n - Q + np.arange(Q)[None, :]
    codes, scales, q, _, _ = attn_case(37, 1, Q, -(-n // 8) * 8, [n], 1, 0, False, pos, spread=1.0, q_size=0.7)
    scales = np.minimum(np.maximum(scales * np.float32(2.0 ** power), np.float32(2.0 ** -60)), np.float32(2.0 ** 80))
    scale = float(np.float32(SCALE * 2.0 ** -power))
    cache, qd, pd = cache_of(codes, scales, [n]), q.cuda(), dev(pos)
    out, lse, w = torch.zeros_like(qd), torch.zeros(1, Q, 64, device="cuda"), torch.zeros(1, cache.cap, device="cuda")
    ws = csa2.Workspace(max(csa2.cache8_attn_workspace_size(1, Q, n), csa2.attn_weights_workspace_size(1, Q, n)))
    csa2.cache8_attn(cache, qd, pd, scale, out, ws, max_n=n, lse=lse)
    csa2.attn_weights(cache, qd, pd, lse, scale, w, ws, max_n=n)
    assert ws.sync_status()[0] == 0
    e, got, got_lse = c8.entries(codes[0], scales[0]), out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    want, tol = np.zeros(cache.cap), np.zeros(cache.cap)
    for i in range(Q):
        seen, qi = int(pos[0, i]) + 1, q[0, i].double().numpy()
        o, l, b_o, b_l = c8.attend(qi, e[:seen], scale, scales[0].max())
        assert np.all(np.abs(got[i] - o) <= b_o) and np.all(np.abs(got_lse[i] - l) <= b_l), i
        more, t = c8.gathered(qi, e[:seen], got_lse[i], scale)
        want[:seen] += more
        tol[:seen] += t
    assert np.all(np.abs(w[0].double().cpu().numpy() - want) <= tol)
