"""The attention weight that cache entries gather (csa2_attn_weights, 4-bit and 8-bit
cache) against the 64-bit form."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
import oracle
from tests import cache8_ref as c8

pytestmark = pytest.mark.gpu
H, D = 64, 512
SCALE = 512 ** -0.5


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_cache(seed, bits, B, cap, n, m):
    """A cache of random entries and their values [B][cap][512] in 64 bits."""
    rng = np.random.default_rng(seed)
    if bits == 8:
        c = csa2.Cache8(B, cap, m)
        codes = rng.integers(-127, 128, (B, c.cap, D)).astype(np.int8)
        scales = (0.02 * rng.random((B, c.cap // 8)) + 0.005).astype(np.float32)
        c.codes.copy_(dev(codes))
        c.scales.copy_(dev(scales))
        values = np.stack([c8.entries(codes[b], scales[b]) for b in range(B)])
    else:
        c = csa2.Cache(B, cap, m, index=False)
        kv = rng.integers(0, 256, (B, c.cap, 288)).astype(np.uint8)
        kv[..., 256:] = rng.integers(0x28, 0x30, (B, c.cap, 32))
        c.main_kv.copy_(dev(kv))
        values = np.stack([oracle.dequant_main(kv[b]).astype(np.float64) for b in range(B)])
    c.n_entries.copy_(dev(np.asarray(n, np.int32)))
    return c, values


def some_lse(q, values, n, m, pos):
    """The queries' log-sum-exp over the entries they see (float32), -inf where there are none."""
    lse = np.full(q.shape[:3], -np.inf)
    for b in range(q.shape[0]):
        for i in range(q.shape[1]):
            seen = min(n[b], max(0, (int(pos[b, i]) + 1) // m)) if pos[b, i] >= 0 else 0
            if seen:
                x = SCALE * (values[b, :seen] @ q[b, i].T)
                lse[b, i] = x.max(0) + np.log(np.exp(x - x.max(0)).sum(0)) + 0.1
    return lse.astype(np.float32)


def check(cache, values, n, m, q, pos, lse, prev=None, decay=1.0, max_n=None, status=0):
    B, Q = pos.shape
    cap = cache.cap
    max_n = cap if max_n is None else max_n
    out = torch.full((B, cap), 5.0, device="cuda")
    ws = csa2.Workspace(csa2.attn_weights_workspace_size(B, Q, max_n))
    csa2.attn_weights(cache, q.cuda(), dev(pos), dev(lse), SCALE, out, ws, max_n=max_n,
                      prev=None if prev is None else dev(prev), decay=decay)
    assert ws.sync_status()[0] == status
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    for b in range(B):
        want, tol = np.zeros(cap), np.zeros(cap)
        if prev is not None:
            want += decay * prev[b].astype(np.float64)
            tol += 2.0 ** -23 * np.abs(want)
        for i in range(Q):
            seen = min(n[b], cap, (int(pos[b, i]) + 1) // m) if pos[b, i] >= 0 else 0
            if seen:
                w, t = c8.gathered(qd[b, i], values[b, :seen], lse[b, i].astype(np.float64), SCALE)
                want[:seen] += w
                tol[:seen] += t
        last = min(n[b], cap, max_n)
        assert np.all(got[b, last:] == 5.0)
        err = np.abs(got[b] - want)[:last]
        assert np.all(err <= tol[:last]), (b, np.max(err / (tol[:last] + 1e-300)))
    return out


CASES = [(1, 1, 8, [1], 1, [0]), (1, 1, 128, [128], 1, [127]), (1, 1, 136, [129], 2, [255]), (3, 1, 1000, [1000, 3, 517], 1, [999, 2, 516]),
         (1, 2, 264, [260], 1, [259]), (2, 3, 264, [260, 100], 2, [519, 60]), (1, 37, 520, [513], 1, [512]),
         (1, 300, 136, [130], 2, [258]), (2, 5, 2000, [1999, 0], 1, [1998, 4]), (16, 1, 304, [300 - 9 * b for b in range(16)], 1, [299] * 16)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,Q,cap,n,m,last", CASES)
def test_weights(bits, B, Q, cap, n, m, last):
    cache, values = make_cache(cap + Q, bits, B, cap, n, m)
    pos = np.asarray(last)[:, None] - (Q - 1) + np.arange(Q)[None, :]
    g = torch.Generator().manual_seed(Q)
    q = (1.5 * torch.randn(B, Q, H, D, generator=g)).bfloat16()
    lse = some_lse(q.double().numpy(), values, n, m, pos)
    prev = np.random.default_rng(1).random((B, cache.cap)).astype(np.float32) if Q != 2 else None
    check(cache, values, n, m, q, pos, lse, prev, decay=0.75)


@pytest.mark.parametrize("Q", [1, 1100, 2051])
def test_weights_of_many_queries_on_few_entries(Q):
    """More query groups than one CTA takes; queries in no order, some without any entry."""
    n = [11]
    cache, values = make_cache(2, 4, 1, 16, n, 1)
    rng = np.random.default_rng(3)
    pos = rng.integers(-2, 40, (1, Q))
    q = torch.from_numpy(rng.standard_normal((1, Q, H, D)).astype(np.float32)).bfloat16()
    lse = some_lse(q.double().numpy(), values, n, 1, pos)
    check(cache, values, n, 1, q, pos, lse)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Q", [1, 4])
def test_weights_what_is_not_seen_may_hold_anything(bits, Q):
    n, cap = [130, 140], 264
    cache, values = make_cache(4, bits, 2, cap, n, 1)
    pos = np.array([[119], [-1]]) - np.arange(Q)[None, ::-1] * np.array([[1], [0]])
    q = torch.randn(2, Q, H, D, generator=torch.Generator().manual_seed(4)).bfloat16()
    lse = some_lse(q.double().numpy(), values, n, 1, pos)
    lse[0, 0, 5] = -np.inf                                                         # a head that saw nothing
    q[0, 0, 5] = float("nan")
    q[1] = float("inf")                                                            # padding
    if bits == 8:
        cache.scales[0, 15:], cache.scales[1, 3:] = float("nan"), float("inf")
    else:
        cache.main_kv[0, 120:, 256:] = 0x7F                                        # E4M3 NaN
        cache.main_kv[1, :, 256:] = 0xFF
    check(cache, values, n, 1, q, pos, lse)


def test_weights_reports_and_leaves_the_rest():
    cache, values = make_cache(5, 4, 2, 64, [64, 64], 1)
    pos = np.array([[63], [63]])
    q = torch.randn(2, 1, H, D, generator=torch.Generator().manual_seed(5)).bfloat16()
    lse = some_lse(q.double().numpy(), values, [64, 64], 1, pos)
    check(cache, values, [64, 64], 1, q, pos, lse, max_n=40, status=6)             # more entries than max_n
    cache.n_entries[1] = 100
    check(cache, values, [64, 64], 1, q, pos, lse, status=6)                       # more than cap
    cache.n_entries[1] = -3
    check(cache, values, [64, 0], 1, q, pos, lse)


def test_weights_without_queries_fade():
    cache, values = make_cache(6, 8, 2, 64, [64, 9], 1)
    prev = np.random.default_rng(6).random((2, 64)).astype(np.float32)
    check(cache, values, [64, 9], 1, torch.zeros(2, 0, H, D, dtype=torch.bfloat16), np.zeros((2, 0), np.int64),
          np.zeros((2, 0, H), np.float32), prev, decay=0.5)


def test_weights_queries_beyond_f16():
    n = [200]
    cache, values = make_cache(7, 4, 1, 200, n, 1)
    pos = np.array([[199, 150]])
    q = torch.randn(1, 2, H, D, generator=torch.Generator().manual_seed(7)).bfloat16()
    q[0, 0, 3] *= 2.0 ** 17
    q[0, 1, 60] *= 2.0 ** 100
    lse = some_lse(q.double().numpy(), values, n, 1, pos)
    assert np.all(np.isfinite(lse))
    lse[0, 0, 3] += 3e5                                                            # its largest weights underflow: nothing to bound
    lse[0, 1, 60] += 1e37
    check(cache, values, n, 1, q, pos, lse)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,Q,cap", [(40, 2, 1000), (76, 2, 600), (25, 4, 1300), (19, 5, 800), (38, 1, 1500)])
def test_weights_several_steps_of_a_run(bits, B, Q, cap):
    """Enough sequences that a CTA, or a pair, takes several steps of entries with the same one or few queries."""
    n = [cap - 7 * b for b in range(B)]
    cache, values = make_cache(13, bits, B, cap, n, 1)
    pos = np.asarray(n)[:, None] - Q + np.arange(Q)[None, :]
    q = torch.randn(B, Q, H, D, generator=torch.Generator().manual_seed(13)).bfloat16()
    check(cache, values, n, 1, q, pos, some_lse(q.double().numpy(), values, n, 1, pos))


@pytest.mark.parametrize("bits,Q", [(4, 1), (8, 1), (4, 3), (8, 3), (8, 6)])
@pytest.mark.parametrize("what", ["lse", "q", "overflow"])
def test_weights_that_are_no_finite_numbers(bits, Q, what):
    """A head's NaN, or a weight beyond binary32, reaches every entry that its query sees and no other."""
    n = [200]
    cache, values = make_cache(12, bits, 1, 200, n, 1)
    pos = np.full((1, Q), 199)
    pos[0, 0] = 149
    q = torch.randn(1, Q, H, D, generator=torch.Generator().manual_seed(12)).bfloat16()
    lse = some_lse(q.double().numpy(), values, n, 1, pos)
    clean = check(cache, values, n, 1, q, pos, lse)
    if what == "q":
        q[0, 0, 33, 100] = float("nan")
    else:
        lse[0, 0, 33] = np.nan if what == "lse" else -1000.0                       # scores lie within 100 of 0
    w = torch.full((1, 200), 5.0, device="cuda")
    ws = csa2.Workspace(csa2.attn_weights_workspace_size(1, Q, 200))
    csa2.attn_weights(cache, q.cuda(), dev(pos), dev(lse), SCALE, w, ws, max_n=200)
    assert ws.sync_status()[0] == 0
    assert torch.all(w[0, :150] == float("inf") if what == "overflow" else torch.isnan(w[0, :150]))
    assert torch.equal(w[0, 150:], clean[0, 150:])


def test_weights_in_place_repeat_and_add_up():
    """prev = weights; the same inputs give the same bits; the sum of a head's weights is 1."""
    n, Q = [700], 9
    cache, values = make_cache(8, 8, 1, 704, n, 1)
    pos = np.full((1, Q), 699)
    q = torch.randn(1, Q, H, D, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    out, lse = torch.zeros(1, Q, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, Q, H, device="cuda")
    ws = csa2.Workspace(max(csa2.cache8_attn_workspace_size(1, Q, 704), csa2.attn_weights_workspace_size(1, Q, 704)))
    csa2.cache8_attn(cache, q, dev(pos), SCALE, out, ws, max_n=704, lse=lse)
    w = torch.zeros(1, 704, device="cuda")
    csa2.attn_weights(cache, q, dev(pos), lse, SCALE, w, ws, max_n=704)
    once = w.clone()
    assert abs(once.double().sum().item() - Q * H) <= 1e-4 * Q * H                 # lse off by 2^-20 (1 + |lse|)
    csa2.attn_weights(cache, q, dev(pos), lse, SCALE, w, ws, max_n=704, prev=w)
    assert torch.equal(w[:, :700], 2 * once[:, :700])                              # exact doubling
    graph, at = torch.cuda.CUDAGraph(), dev(pos)
    with torch.cuda.graph(graph):
        csa2.attn_weights(cache, q, at, lse, SCALE, w, ws, max_n=704)
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, once) and ws.sync_status()[0] == 0


def test_weights_offsets_beyond_32_bits():
    cap = 8_000_000                                                                # 2.3 GB a sequence
    cache = csa2.Cache(2, cap, 1, index=False)
    rng = np.random.default_rng(9)
    kv = rng.integers(0, 256, (128, 288)).astype(np.uint8)
    kv[:, 256:] = rng.integers(0x28, 0x30, (128, 32))
    cache.main_kv[1, cap - 128:].copy_(dev(kv))
    cache.n_entries.copy_(dev(np.array([3, cap], np.int32)))
    pos, q = np.array([[2], [cap - 1]]), torch.randn(2, 1, H, D, generator=torch.Generator().manual_seed(9)).bfloat16()
    lse = np.full((2, 1, H), 20.0, np.float32)
    w = torch.zeros(2, cap, device="cuda")
    ws = csa2.Workspace(csa2.attn_weights_workspace_size(2, 1, cap))
    csa2.attn_weights(cache, q.cuda(), dev(pos), dev(lse), SCALE, w, ws, max_n=cap)
    assert ws.sync_status()[0] == 0
    want, tol = c8.gathered(q[1, 0].double().numpy(), oracle.dequant_main(kv).astype(np.float64), lse[1, 0].astype(np.float64), SCALE)
    assert np.all(np.abs(w[1, cap - 128:].double().cpu().numpy() - want) <= tol)
    flat = 64 * np.exp(-20.0)                                                      # entries of zeros
    assert torch.all((w[1, :cap - 128].double() - flat).abs() <= 1e-5 * flat)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Q", [0, 1, 3])
def test_weights_of_no_entries_report_too(bits, Q):
    """max_n = 0, or a cache without room: nothing is written, and a sequence that has entries is reported."""
    cache, values = make_cache(14, bits, 2, 64, [0, 0], 1)
    q, pos, lse = torch.zeros(2, Q, H, D, dtype=torch.bfloat16), np.full((2, Q), 70), np.zeros((2, Q, H), np.float32)
    for n, status in (([0, 5], 6), ([0, -2], 0)):
        cache.n_entries.copy_(dev(np.asarray(n, np.int32)))
        check(cache, values, [0, 0], 1, q, pos, lse, max_n=0, status=status)
    w, ws = torch.full((2, 8), 5.0, device="cuda"), csa2.Workspace(csa2.attn_weights_workspace_size(2, Q, 64))
    qd, ld = torch.zeros(2, 4, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, H, device="cuda")
    pd = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    a = csa2.WeightsArgs(B=2, Q=Q, scale=SCALE, decay=1.0, max_n=64, q_pos=pd.data_ptr(), q=qd.data_ptr(), lse=ld.data_ptr(),
                         weights=w.data_ptr())
    if bits == 8:
        c = csa2.Cache8Struct(codes=cache.codes.data_ptr(), scales=cache.scales.data_ptr(), cap=0,
                              n_entries=cache.n_entries.data_ptr(), m=1)
    else:
        c = csa2.CacheStruct(main_kv=cache.main_kv.data_ptr(), cap=0, n_entries=cache.n_entries.data_ptr(), m=1)
    call = csa2.load().csa2_cache8_attn_weights if bits == 8 else csa2.load().csa2_attn_weights
    for n, status in (([0, 1], 6), ([0, 0], 0)):
        cache.n_entries.copy_(dev(np.asarray(n, np.int32)))
        assert call(ctypes.byref(c), ctypes.byref(a), ws.buf.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream) == 0
        assert ws.sync_status()[0] == status
    assert torch.all(w == 5.0)


@pytest.mark.parametrize("Q", [64, 35 * 1024])
def test_weights_of_divided_queries_keep_what_is_small(Q):
    """One query's weights are 2^24 times the others': each CTA's sum of those alone is less than half of the last place
    of the total (35 * 1024 queries are 35 CTAs' at least).  Queries of zeros, so that a weight is exp(-lse)."""
    n = 11
    cache, _ = make_cache(15, 4, 1, 16, [n], 1)

    def weigh(lse):
        k = lse.shape[0]
        w = torch.zeros(1, 16, device="cuda")
        ws = csa2.Workspace(csa2.attn_weights_workspace_size(1, k, 16))
        csa2.attn_weights(cache, torch.zeros(1, k, H, D, dtype=torch.bfloat16, device="cuda"),
                          torch.full((1, k), n, device="cuda"), lse[None, :, None].expand(1, k, H).contiguous(), SCALE, w, ws, max_n=16)
        assert ws.sync_status()[0] == 0
        assert torch.all(w[0, :n] == w[0, 0])                                      # entries are alike
        return w[0, 0].double().item()

    per_cta = 2 if Q == 64 else 1024                                               # queries of a CTA's sum, or fewer
    lse = torch.full((Q,), -np.log(50.0 / (H * per_cta)), dtype=torch.float32, device="cuda")
    big = torch.tensor([-24 * np.log(2.0)] + [np.inf] * 3, dtype=torch.float32, device="cuda")
    small, large = weigh(lse[:4]) / 4, weigh(big)                                  # (2^-23 of themselves: 64 equal weights sum exactly)
    assert 2 ** 29.9 < large < 2 ** 30.1 and 40 < small * per_cta < 60
    lse[0] = big[0]
    # Roundings to binary32 of compensated sums: of a half's queries, of the two halves, over CTAs, of the result: 2^-24 each
    # of the total; `small` by 2^-22 of itself
    want = large + (Q - 1) * small
    assert abs(weigh(lse) - want) <= 4 * 2.0 ** -24 * want + 2.0 ** -22 * (Q - 1) * small


@pytest.mark.parametrize("Q", [1, 2])
@pytest.mark.parametrize("bits,scale,keys", [(4, SCALE * 2.0 ** -17, 1.0), (8, SCALE * 2.0 ** -17, 1.0), (8, SCALE, 2.0 ** -18)])
def test_weights_of_large_queries_are_their_softmax(bits, scale, keys, Q):
    """Heads of 2^17 to 2^30, brought back to ordinary scores by the softmax scale or by the entries, with their own lse:
    weights of 1 / n and more, as far as scores let them."""
    n = [200]
    cache, values = make_cache(16, bits, 1, 200, n, 1)
    if keys != 1.0:
        cache.scales.mul_(keys)
        values = values * keys
    pos = np.array([[199, 150][:Q]])
    q = torch.randn(1, Q, H, D, generator=torch.Generator().manual_seed(16))
    q = (q * 2.0 ** 17 * torch.exp2(torch.arange(H) % 3)[:, None]).bfloat16()
    q[0, 0, 7] *= 2.0 ** 11                                                        # scores of thousands: one entry has all
    qd = q.double().numpy()
    # a head goes to f16 by a power of two that puts its largest below 2^16: what then is at least 2^-14 is exact
    top = np.exp2(np.floor(np.log2(np.abs(qd).max(-1, keepdims=True))) - 15)
    assert np.all((np.abs(qd) >= 2.0 ** -14 * np.maximum(top, 1)) | (qd == 0))
    lse, want, tol = np.zeros((1, Q, H), np.float32), np.zeros(200), np.zeros(200)
    for i in range(Q):
        k = values[0, :pos[0, i] + 1]
        x = scale * (k @ qd[0, i].T)
        lse[0, i] = x.max(0) + np.log(np.exp(x - x.max(0)).sum(0))
        w, t = c8.gathered(qd[0, i], k, lse[0, i].astype(np.float64), scale)
        want[:len(k)] += w
        tol[:len(k)] += t
    assert abs(want.sum() - Q * H) < 0.1 and np.median(tol[:151] / want[:151]) < 1e-2
    out, ws = torch.zeros(1, 200, device="cuda"), csa2.Workspace(csa2.attn_weights_workspace_size(1, Q, 200))
    csa2.attn_weights(cache, q.cuda(), dev(pos), dev(lse), scale, out, ws, max_n=200)
    assert ws.sync_status()[0] == 0
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert np.all(err <= tol), np.max(err / tol)
