"""The 8-bit cache: csa2_cache8_write against its definition, bit for bit, and
csa2_cache8_attn against the 64-bit form."""
import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
from tests import cache8_ref as c8
from tests import keys_ref as ref

pytestmark = pytest.mark.gpu
H, D = 64, 512
SCALE = 512 ** -0.5


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def latents(g, *shape):
    z = torch.randn(*shape, D, generator=g)
    return (z / z.pow(2).mean(-1, keepdim=True).sqrt()).bfloat16()


def cache_of(codes, scales, n, m=1):
    c = csa2.Cache8(codes.shape[0], codes.shape[1], m)
    c.codes.copy_(dev(codes))
    c.scales.copy_(dev(scales))
    c.n_entries.copy_(dev(np.asarray(n, np.int32)))
    return c


def old_cache(seed, B, cap):
    rng = np.random.default_rng(seed)
    return rng.integers(-127, 128, (B, cap, D)).astype(np.int8), (0.02 * rng.random((B, cap // 8)) + 0.01).astype(np.float32)


def write_and_check(codes, scales, n, x, start, n_new, status=0, strided=None):
    cache, ws = cache_of(codes, scales, n), csa2.Workspace(256)
    want = c8.write(codes, scales, n, x.double().numpy(), start, x.shape[1] * np.ones(len(start), int) if n_new is None else n_new)
    csa2.cache8_write(cache, x.cuda() if strided is None else strided, dev(np.asarray(start, np.int64)), ws,
                      n_new=None if n_new is None else dev(np.asarray(n_new, np.int32)))
    assert ws.sync_status()[0] == status
    assert np.array_equal(cache.scales.cpu().numpy(), want[1])
    assert np.array_equal(cache.codes.cpu().numpy(), want[0])
    assert np.array_equal(cache.n_entries.cpu().numpy(), n)
    return cache


@pytest.mark.parametrize("B,T,cap,start,n_new,n", [
    (1, 1, 8, [0], None, [0]), (1, 1, 8, [7], None, [7]), (3, 1, 40, [5, 8, 31], None, [5, 8, 31]),
    (2, 8, 64, [0, 8], None, [0, 8]), (2, 13, 64, [3, 16], [13, 5], [3, 16]), (2, 77, 200, [101, 0], [0, 77], [101, 0]),
    (1, 5, 40, [10], None, [40]), (2, 3, 24, [9, 9], None, [14, 9]), (1, 300, 304, [0], [299], [0])])
def test_write(B, T, cap, start, n_new, n):
    g = torch.Generator().manual_seed(T)
    codes, scales = old_cache(T, B, cap)
    write_and_check(codes, scales, np.asarray(n, np.int32), latents(g, B, T), start, n_new)


def test_write_from_a_wider_matrix():
    g = torch.Generator().manual_seed(3)
    codes, scales = old_cache(3, 2, 32)
    x = latents(g, 2, 9)
    wide = torch.full((18, 640), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:576] = x.flatten(0, 1).cuda()
    write_and_check(codes, scales, np.zeros(2, np.int32), x, [3, 0], None, strided=wide[:, 64:576].unflatten(0, (2, 9)))


@pytest.mark.parametrize("start,n_new,n", [([-2], [6], [0]), ([13], [6], [13]), ([16], [6], [0]), ([1 << 62], [6], [0]),
                                           ([-(1 << 62)], [6], [0]), ([4], [9], [4]), ([4], [-1], [4])])
def test_write_reports_what_lies_outside(start, n_new, n):
    g = torch.Generator().manual_seed(5)
    codes, scales = old_cache(5, 1, 16)
    write_and_check(codes, scales, np.asarray(n, np.int32), latents(g, 1, 6), start, n_new, status=6)


def test_write_nothing_and_padded_rows():
    """No tokens; and of a padded batch only the first n_new, whatever the others hold."""
    codes, scales = old_cache(6, 2, 16)
    write_and_check(codes, scales, np.zeros(2, np.int32), torch.zeros(2, 0, D, dtype=torch.bfloat16), [0, 3], None)
    x = latents(torch.Generator().manual_seed(6), 2, 9)
    x[0, 4:], x[1, 1:] = float("nan"), float("inf")
    write_and_check(codes, scales, np.zeros(2, np.int32), x, [0, 3], [4, 1])


def test_write_ties_go_to_even():
    x = torch.zeros(1, 8, D)
    x[0, :, :127] = torch.arange(127)[None] - 62.5                 # -62.5 .. 63.5, ties of scale 1
    x[0, :, 127] = 127.0
    x = torch.cat([x * 2.0 ** -20, x, x * 2.0 ** 30], 1).bfloat16()
    codes, scales = old_cache(1, 1, 24)
    cache = write_and_check(codes, scales, np.zeros(1, np.int32), x, [0], None)
    assert cache.codes[0, 0, :4].tolist() == [-62, -62, -60, -60]


def test_write_values_of_every_size():
    g = torch.Generator().manual_seed(8)
    x = latents(g, 1, 48).float()
    x[0, 0:8] *= 2.0 ** -70                                                       # below the least scale
    x[0, 8:16] = 0
    x[0, 16:24] *= 2.0 ** 124
    x[0, 24, 3], x[0, 24, 5], x[0, 25, 7] = float("inf"), float("-inf"), float("nan")
    x[0, 32, 9] = float("nan")
    x[0, 40:48] *= 2.0 ** -50
    codes, scales = old_cache(8, 1, 48)
    write_and_check(codes, scales, np.zeros(1, np.int32), x.bfloat16(), [0], None)


def test_write_one_by_one_grows_the_scale():
    g = torch.Generator().manual_seed(9)
    x = latents(g, 2, 24) * torch.linspace(0.3, 2.0, 24)[None, :, None].bfloat16()
    codes, scales = np.full((2, 32, D), 77, np.int8), np.full((2, 4), np.nan, np.float32)
    cache, ws = cache_of(codes, scales, [0, 0]), csa2.Workspace(256)
    n = np.zeros(2, np.int32)
    for i in range(24):
        csa2.cache8_write(cache, x[:, i:i + 1].cuda(), dev(np.full(2, i)), ws)
        cache.n_entries.add_(1)
        codes, scales = c8.write(codes, scales, n, x[:, i:i + 1].double().numpy(), [i, i], [1, 1])
        n += 1
    assert ws.sync_status()[0] == 0
    assert np.array_equal(cache.codes.cpu().numpy(), codes)
    assert np.array_equal(cache.scales.cpu().numpy()[:, :3], scales[:, :3])


# ------------------------------------------------------------------ attention
def attn_case(seed, B, Q, cap, n, m, W, fp8, pos, spread=0.0, q_size=1.5):
    """An 8-bit cache of unit latents (blocks sized by 2^(spread * normal)), queries, window rows."""
    g = torch.Generator().manual_seed(seed)
    x = latents(g, B, cap).double().numpy()
    size = np.exp2(np.round(spread * torch.randn(B, cap // 8, 1, 1, generator=g).double().numpy()))
    x = (x.reshape(B, cap // 8, 8, D) * size).reshape(B, cap, D)
    codes, scales = c8.write(np.zeros((B, cap, D), np.int8), np.zeros((B, cap // 8), np.float32), [0] * B, x, [0] * B,
                             [cap] * B)
    q = (q_size * torch.randn(B, Q, H, D, generator=g)).bfloat16()
    base = np.maximum(0, np.where(pos >= 0, pos, 1 << 60).min(1) - W + 1) if W else None
    rows = None
    if W:
        rows = latents(g, B, int(pos.max() - base.min()) + 1)
        rows = rows.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else rows
    return codes, scales, q, rows, base


def attend_and_check(codes, scales, n, m, q, rows, base, pos, W, status=0, max_n=None):
    B, Q = pos.shape
    max_n = max_n or int(max(n))
    cache = cache_of(codes, scales, n, m)
    out = torch.full((B, Q, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Q, H), 3.0, device="cuda")
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(B, Q, max_n, W))
    csa2.cache8_attn(cache, q.cuda(), dev(pos), SCALE, out, ws, max_n=max_n, W=W,
                     swa=None if rows is None else rows.cuda(), swa_base_pos=None if base is None else dev(base), lse=lse)
    assert ws.sync_status()[0] == status
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        e = c8.entries(codes[b], scales[b])
        w = None if rows is None else ref.row_values(rows[b].numpy() if rows.dtype == torch.uint8
                                                     else rows[b].view(torch.int16).numpy().view(np.uint16))
        for i in range(Q):
            t = int(pos[b, i])
            keys = np.zeros((0, D))
            if t >= 0:
                keys = e[:min(n[b], (t + 1) // m, codes.shape[1])]
                if W:
                    keys = np.concatenate([keys, ref.window_keys(w, int(base[b]), t, W)])
            seen = -(-min(n[b], max(0, (t + 1) // m)) // 8)
            most = scales[b][:seen].max(initial=0.0) if t >= 0 else 0.0
            o, l, b_o, b_l = c8.attend(q[b, i].double().numpy(), keys, SCALE, most)
            assert np.all(np.abs(got[b, i] - o) <= b_o), (b, i, np.max(np.abs(got[b, i] - o) / b_o))
            if keys.shape[0] == 0:
                assert np.all(got_lse[b, i] == -np.inf)
            else:
                assert np.all(np.abs(got_lse[b, i] - l) <= b_l), (b, i)
    return out, lse


@pytest.mark.parametrize("B,Q,cap,n,m,W,fp8,last", [
    (1, 1, 8, [1], 1, 0, False, [0]), (1, 1, 64, [64], 1, 0, False, [63]), (1, 1, 72, [65], 1, 1, False, [64]),
    (2, 3, 208, [200, 77], 1, 128, False, [199, 76]), (2, 5, 208, [200, 3], 2, 99, True, [398, 6]),
    (1, 4, 608, [600], 1, 0, False, [599]), (3, 2, 1000, [1000, 1, 999], 2, 130, False, [1999, 1, 1500]),
    (1, 160, 136, [130], 1, 64, True, [129]), (1, 153, 72, [70], 2, 0, False, [120])])
def test_attention(B, Q, cap, n, m, W, fp8, last):
    pos = np.asarray(last)[:, None] - (Q - 1) + np.arange(Q)[None, :]              # some before position 0: padding
    attend_and_check(*attn_case(cap + Q, B, Q, cap, n, m, W, fp8, pos)[:2], n, m,
                     *attn_case(cap + Q, B, Q, cap, n, m, W, fp8, pos)[2:], pos, W)


def test_attention_queries_that_see_nothing():
    pos = np.array([[-1, 0, 1, -5], [-(1 << 60), 3, -1, 0]])
    n = [9, 0]
    case = attn_case(1, 2, 4, 16, n, 2, 0, False, pos)
    attend_and_check(*case[:2], n, 2, *case[2:], pos, 0)


@pytest.mark.parametrize("Q,spread,q_size", [(1, 2.0, 0.5), (1, 3.0, 0.02), (160, 3.0, 0.1)])
def test_attention_scales_of_every_size(Q, spread, q_size):
    """Blocks of very different scales: the weights of the small ones must survive beside the large."""
    pos = 499 - np.arange(Q)[None, :]
    case = attn_case(int(spread), 1, Q, 504, [500], 1, 64, False, pos, spread=spread, q_size=q_size)
    attend_and_check(*case[:2], [500], 1, *case[2:], pos, 64)


@pytest.mark.parametrize("power", [-58, -30, 9])
def test_attention_all_scales_tiny_or_large(power):
    pos = np.array([[299]])
    codes, scales, q, _, _ = attn_case(4, 1, 1, 304, [300], 1, 0, False, pos)
    scales = (scales.astype(np.float64) * 2.0 ** power).astype(np.float32)
    q = (q.double() * 2.0 ** (-power if power > 0 else 0)).bfloat16()
    attend_and_check(codes, np.maximum(scales, np.float32(2.0 ** -60)), [300], 1, q, None, None, pos, 0)


def test_attention_blocks_of_zeros():
    pos = np.array([[255, 7, 260]])
    codes, scales, q, _, _ = attn_case(6, 1, 3, 264, [264], 1, 0, False, pos)
    codes[0, :128] = 0
    scales[0, :16] = 0.0                                                          # never written: zeros
    attend_and_check(codes, scales, [264], 1, q, None, None, pos, 0)


def test_attention_what_is_not_seen_may_hold_anything():
    n, pos = [37, 64], np.array([[30, 36], [63, 50]])
    codes, scales, q, rows, base = attn_case(7, 2, 2, 72, n, 1, 9, False, pos)
    scales[0, 5:], scales[1, 8:] = np.nan, np.inf
    rows[0, int(pos[0].max() - base[0]) + 1:] = float("nan")
    attend_and_check(codes, scales, n, 1, q, rows, base, pos, 9)


# Calls that go to pairs of CTAs: enough queries of enough entries (152 of 1200 and more; divided over CTAs, 60 of
# 3000)
@pytest.mark.parametrize("B,Q,cap,n,m,W,fp8,last", [
    (1, 152, 1304, [1300], 1, 0, False, [1299]), (2, 76, 1448, [1441, 1300], 2, 130, False, [2880, 2590]),
    (4, 37, 1608, [1600, 1600, 1333, 20], 1, 99, True, [1599, 1000, 1332, 19]), (1, 60, 3000, [2999], 1, 128, False, [2998]),
    (2, 31, 3000, [2999, 1777], 2, 64, True, [5997, 3554]), (1, 151, 1304, [70], 1, 200, False, [1500])])
def test_attention_pairs(B, Q, cap, n, m, W, fp8, last):
    pos = np.asarray(last)[:, None] - (Q - 1) + np.arange(Q)[None, :]              # some before position 0: padding
    case = attn_case(cap + Q, B, Q, cap, n, m, W, fp8, pos)
    n_call = [max(n)] * B                                                          # (max_n: the rule's input)
    attend_and_check(*case[:2], n, m, *case[2:], pos, W, max_n=max(1300, *n_call))


@pytest.mark.parametrize("spread,q_size", [(2.0, 0.5), (3.0, 0.02)])
def test_attention_pairs_scales_of_every_size(spread, q_size):
    pos = 1299 - np.arange(152)[None, :]
    case = attn_case(21, 1, 152, 1304, [1300], 1, 64, False, pos, spread=spread, q_size=q_size)
    attend_and_check(*case[:2], [1300], 1, *case[2:], pos, 64)


def test_attention_pairs_queries_beyond_f16_and_blocks_of_zeros():
    pos = np.repeat(np.array([[1299, 640, 7, 600]]), 38, 1)
    codes, scales, q, _, _ = attn_case(22, 1, 152, 1304, [1300], 1, 0, False, pos)
    codes[0, :640], scales[0, :80] = 0, 0.0                                        # never written: zeros
    scales *= np.float32(2.0 ** -20)
    q[0, ::3, 5] *= 2.0 ** 20
    q[0, 1::4, 60] *= 2.0 ** 30
    attend_and_check(codes, scales, [1300], 1, q, None, None, pos, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_rows_that_only_the_newer_query_sees(fp8):
    """A window row with a NaN: the queries that see it become NaN, their neighbours stay as they are."""
    pos = 1100 + np.arange(152)[None, :]
    codes, scales, q, rows, base = attn_case(14, 1, 152, 1304, [1300], 1, 16, fp8, pos)
    cache, ws = cache_of(codes, scales, [1300]), csa2.Workspace(csa2.cache8_attn_workspace_size(1, 152, 1300, 16))
    got = []
    for bad in (False, True):
        if bad:
            rows = rows.clone()
            rows[0, 1183 - int(base[0]), 300] = 0x7F if fp8 else float("nan")
        out = torch.zeros(1, 152, H, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(1, 152, H, device="cuda")
        csa2.cache8_attn(cache, q.cuda(), dev(pos), SCALE, out, ws, max_n=1300, W=16, swa=rows.cuda(), swa_base_pos=dev(base), lse=lse)
        got.append((out, lse))
    assert ws.sync_status()[0] == 0
    (out, lse), (bad_out, bad_lse) = got
    assert torch.all(torch.isfinite(out.float()))
    sees = slice(83, 99)                                                           # positions 1183 .. 1198
    assert torch.all(torch.isnan(bad_out[0, sees])) and torch.all(torch.isnan(bad_lse[0, sees]))
    keep = [i for i in range(152) if not 83 <= i < 99]
    assert torch.equal(bad_out[0, keep], out[0, keep]) and torch.equal(bad_lse[0, keep], lse[0, keep])


@pytest.mark.parametrize("W,fp8", [(0, False), (40, False), (200, True)])
def test_attention_neighbours_far_apart(W, fp8):
    """Two queries of a pair whose windows lie apart, meet or overlap, one of them padding, and queries in no order."""
    pos = np.tile(np.array([[600, 10, 300, 341, 5, -1, 44, 45, -7]]), (1, 17))[:, :151]
    n = [1300]
    codes, scales, q, rows, base = attn_case(15, 1, 151, 1304, n, 1, W, fp8, pos)
    if W:
        base = np.zeros(1, np.int64)
        g = torch.Generator().manual_seed(16)
        rows = latents(g, 1, 601)
        rows = rows.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else rows
    attend_and_check(codes, scales, n, 1, q, rows, base, pos, W)


def test_attention_reports():
    pos = np.array([[63]])
    codes, scales, q, _, _ = attn_case(8, 1, 1, 64, [70], 1, 0, False, pos)
    attend_and_check(codes, scales, [70], 1, q, None, None, pos, 0, status=6)      # n_entries beyond cap
    codes, scales, q, rows, base = attn_case(8, 1, 1, 64, [60], 1, 8, False, pos)
    attend_and_check(codes, scales, [60], 1, q, rows[:, 3:], base + 3, pos, 8, status=6)


def test_attention_queries_beyond_f16():
    pos = np.array([[199]])
    codes, scales, q, _, _ = attn_case(11, 1, 1, 200, [200], 1, 0, False, pos)
    q[0, 0, 3] *= 2.0 ** 20
    scales *= np.float32(2.0 ** -20)
    attend_and_check(codes, scales, [200], 1, q, None, None, pos, 0)


def test_attention_offsets_beyond_32_bits():
    cap, n = 4_400_000, 100
    cache = csa2.Cache8(2, cap, 1)
    pos = np.array([[99], [cap - 1]])
    codes, scales, q, _, _ = attn_case(12, 2, 1, 104, [n, n], 1, 0, False, np.array([[99], [99]]))
    cache.codes[:, :104].copy_(dev(codes))
    cache.scales[:, :13].copy_(dev(scales))
    cache.codes[1, cap - 104:].copy_(dev(codes[0]))
    cache.scales[1, cap // 8 - 13:].copy_(dev(scales[0]))
    cache.n_entries.copy_(dev(np.array([n, cap], np.int32)))
    out, lse = torch.zeros(2, 1, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 1, H, device="cuda")
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(2, 1, cap, 0))
    csa2.cache8_attn(cache, q.cuda(), dev(pos), SCALE, out, ws, max_n=cap, lse=lse)
    assert ws.sync_status()[0] == 0
    keys = np.concatenate([c8.entries(codes[1], scales[1]), np.zeros((cap - 208, D), np.int8), c8.entries(codes[0], scales[0])])
    for b, k in ((0, c8.entries(codes[0], scales[0])[:n]), (1, keys)):
        logit = SCALE * (q[b, 0].double().numpy() @ k.T)
        top = logit.max(-1)
        want = top + np.log(np.exp(logit - top[:, None]).sum(-1))
        # sums of one entry a chunk and lane over at most 70,000 chunks of several CTAs: 2^-24 each for the 900 of
        # one, and what keys_ref.attend allows the logits
        assert np.all(np.abs(lse[b, 0].double().cpu().numpy() - want) <= 1e-4)


def test_attention_captured_and_on_another_stream():
    n, pos = [500, 123], np.array([[499], [122]])
    codes, scales, q, rows, base = attn_case(13, 2, 1, 504, n, 1, 32, False, pos)
    out, lse = attend_and_check(codes, scales, n, 1, q, rows, base, pos, 32)
    cache, qd, pd, rd, bd = cache_of(codes, scales, n), q.cuda(), dev(pos), rows.cuda(), dev(base)
    got = torch.zeros_like(out)
    ws = csa2.Workspace(csa2.cache8_attn_workspace_size(2, 1, 500, 32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    csa2.cache8_attn(cache, qd, pd, SCALE, got, ws, max_n=500, W=32, swa=rd, swa_base_pos=bd, stream=s)
    s.synchronize()
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.cache8_attn(cache, qd, pd, SCALE, got, ws, max_n=500, W=32, swa=rd, swa_base_pos=bd)
    got.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out) and ws.sync_status()[0] == 0


@pytest.mark.parametrize("Q,n,W", [(152, 1300, 32), (60, 3000, 0)])
def test_attention_pairs_captured_and_beside_themselves(Q, n, W):
    """Graphs of the same call on two workspaces, replayed at once; its queries divided over CTAs (60 of 3000) or not."""
    pos = n - Q + np.arange(Q)[None, :]
    codes, scales, q, rows, base = attn_case(17, 1, Q, -(-n // 8) * 8, [n], 1, W, False, pos)
    out, lse = attend_and_check(codes, scales, [n], 1, q, rows, base, pos, W)
    cache, qd, pd = cache_of(codes, scales, [n]), q.cuda(), dev(pos)
    rd, bd = (rows.cuda(), dev(base)) if W else (None, None)
    calls = []
    for _ in range(2):
        got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)
        ws = csa2.Workspace(csa2.cache8_attn_workspace_size(1, Q, n, W))
        ws.buf[256:].fill_(0xFF)                                                   # NaN where no state is written
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            csa2.cache8_attn(cache, qd, pd, SCALE, got, ws, max_n=n, W=W, swa=rd, swa_base_pos=bd, lse=got_lse)
        calls.append((graph, got, got_lse, ws, torch.cuda.Stream()))
    for _ in range(3):
        for graph, _, _, _, s in calls:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, got_lse, ws, _ in calls:
        assert torch.equal(got, out) and torch.equal(got_lse, lse) and ws.sync_status()[0] == 0


def test_attention_pairs_more_entries_than_max_n():
    """max_n sizes the split and nothing else."""
    pos = 2990 - 60 + np.arange(60)[None, :]
    case = attn_case(18, 1, 60, 2992, [2992], 1, 20, False, pos)
    attend_and_check(*case[:2], [2992], 1, *case[2:], pos, 20, max_n=1)
    attend_and_check(*case[:2], [2992], 1, *case[2:], pos, 20, max_n=1 << 40)
