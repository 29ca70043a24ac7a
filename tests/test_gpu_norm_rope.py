"""Queries and window keys from their projections (csa2_qk_norm_rope) against the
64-bit form, with the error bound of its arithmetic."""
import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
from tests import keys_ref as ref

pytestmark = pytest.mark.gpu
P = 300


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def make(seed, T, q_gap=0, k_gap=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    q = (scale * torch.randn(T, 64 * 512 + q_gap, generator=g)).bfloat16().cuda()
    k = (scale * torch.randn(T, 512 + k_gap, generator=g)).bfloat16().cuda()
    w = (1 + 0.3 * torch.randn(2, 512, generator=g)).cuda()
    return q[:, :64 * 512].unflatten(1, (64, 512)), k[:, :512], w[0].contiguous(), w[1].contiguous()


def check(got, x, w, cs, eps, u):
    want, tol = ref.norm_rope(x, w, cs, eps), ref.norm_rope_bound(x, w, cs, eps, u)
    if u == ref.U_E4M3:
        want = np.clip(want, -448, 448)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("T,q_gap,k_gap,weights,fp8,eps", [
    (1, 0, 0, True, False, 1e-6), (3, 8, 8, False, True, 1e-6), (4, 0, 0, True, True, 1e-5),
    (5, 1000, 512, True, False, 0.0), (67, 640, 24, True, True, 1e-6), (130, 0, 0, False, False, 1e-3)])
def test_against_the_formula(T, q_gap, k_gap, weights, fp8, eps):
    q, k, qw, kw = make(T, T, q_gap, k_gap)
    cs = csa2.rope_table(P)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, P, T)
    pos[rng.random(T) < 0.2] = -1
    slot = rng.permutation(T + 3)[:T]
    if T > 4:
        slot[1] = -1
    rows = torch.full((T + 3, 512), 0x55 if fp8 else 7.0, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    out = torch.full((T, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = csa2.Workspace(256)
    csa2.qk_norm_rope(torch.from_numpy(pos).cuda(), cs.cuda(), ws, q=q, q_weight=qw if weights else None, q_out=out,
                      k=k, k_weight=kw if weights else None, rows=rows, k_slot=torch.from_numpy(slot).cuda(), eps=eps)
    assert ws.sync_status()[0] == 0
    got_q = ref.bf16(bits(out))
    got_r = ref.row_values(rows.cpu().numpy() if fp8 else bits(rows))
    xq, xk = q.cpu().double().numpy(), k.cpu().double().numpy()
    written = set()
    for t in range(T):
        if pos[t] < 0:
            assert np.all(got_q[t] == 7.0)
            continue
        check(got_q[t], xq[t], qw.cpu().numpy() if weights else None, cs[pos[t]].numpy(), eps, ref.U_BF16)
        if slot[t] >= 0:
            written.add(int(slot[t]))
            check(got_r[slot[t]], xk[t], kw.cpu().numpy() if weights else None, cs[pos[t]].numpy(), eps,
                  ref.U_E4M3 if fp8 else ref.U_BF16)
    left = [r for r in range(T + 3) if r not in written]     # rows that no token names stay as they were
    assert np.all(got_r[left] == (ref.row_values(np.array([0x55], np.uint8))[0] if fp8 else 7.0))


def test_in_place_parts_and_default_rows():
    """q alone in place; k alone with row t for token t: the same values as the whole call."""
    T = 9
    q, k, qw, kw = make(5, T)
    pos, cs, ws = torch.arange(T, device="cuda"), csa2.rope_table(P).cuda(), csa2.Workspace(256)
    out, rows = torch.empty_like(q), torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    csa2.qk_norm_rope(pos, cs, ws, q=q, q_weight=qw, q_out=out, k=k, k_weight=kw, rows=rows)
    mine, rows2 = q.clone(), torch.empty_like(rows)
    csa2.qk_norm_rope(pos, cs, ws, q=mine, q_weight=qw, q_out=mine)
    csa2.qk_norm_rope(pos, cs, ws, k=k, k_weight=kw, rows=rows2.view(3, 3, 512))
    assert ws.sync_status()[0] == 0
    assert torch.equal(mine, out) and torch.equal(rows2, rows)


def test_bad_positions_and_slots_are_reported_and_skipped():
    q, k, _, _ = make(6, 4)
    cs = csa2.rope_table(P).cuda()
    for pos, slot, with_q, detail in (([0, P, 1, 2], [0, 1, 2, 3], True, P), ([0, 1, -2, 2], [0, 1, 2, 3], False, -2),
                                      ([0, 1, 2, 3], [0, 4, 2, 3], True, 4), ([0, 1, 2, 3], [0, 1, 2, -7], True, -7)):
        ws = csa2.Workspace(256)
        out = torch.full((4, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        rows = torch.full((4, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        kw = dict(q=q, q_out=out) if with_q else {}
        csa2.qk_norm_rope(torch.tensor(pos, device="cuda"), cs, ws, k=k, rows=rows,
                          k_slot=torch.tensor(slot, device="cuda"), **kw)
        st, d = ws.sync_status()
        assert (st, d) == (6, detail)
        for t in range(4):
            bad_pos = not 0 <= pos[t] < P
            if with_q:
                assert bool((out[t] == 7.0).all()) == bad_pos
            if 0 <= slot[t] < 4:
                assert bool((rows[slot[t]] == 7.0).all()) == bad_pos


def test_special_values():
    """A zero row stays zero, a row's NaN and infinities stay in that row, and E4M3 saturates."""
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    x[1, 5] = float("nan")
    x[2, 0] = 1.0                                       # sqrt(512) = 22.6 after the norm
    x[3, :] = 3.0
    rows = torch.zeros(4, 512, dtype=torch.uint8, device="cuda")
    ws = csa2.Workspace(256)
    w = torch.full((512,), 100.0, device="cuda")
    csa2.qk_norm_rope(torch.zeros(4, dtype=torch.int64, device="cuda"), csa2.rope_table(1).cuda(), ws, k=x, k_weight=w,
                      rows=rows)
    got = rows.cpu().view(torch.float8_e4m3fn).float()
    assert torch.all(got[0] == 0) and torch.all(torch.isnan(got[1]))
    assert got[2, 0] == 448 and torch.all(got[2, 1:] == 0)
    assert torch.all((got[3] - 100.0).abs() <= 100 * ref.U_E4M3)


def test_another_stream_and_a_replayed_graph():
    T = 40
    q, k, qw, kw = make(7, T)
    pos, cs, ws = torch.arange(T, device="cuda"), csa2.rope_table(P).cuda(), csa2.Workspace(256)
    out, rows = torch.empty_like(q), torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    csa2.qk_norm_rope(pos, cs, ws, q=q, q_weight=qw, q_out=out, k=k, k_weight=kw, rows=rows)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out2, rows2 = torch.empty_like(out), torch.empty_like(rows)
    torch.cuda.synchronize()
    csa2.qk_norm_rope(pos, cs, ws, q=q, q_weight=qw, q_out=out2, k=k, k_weight=kw, rows=rows2, stream=s)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(rows, rows2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.qk_norm_rope(pos, cs, ws, q=q, q_weight=qw, q_out=out2, k=k, k_weight=kw, rows=rows2)
    out2.zero_()
    rows2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(rows, rows2)


def test_offsets_past_32_bits():
    """66,000 tokens in place: the queries pass 2^32 bytes."""
    T = 66_000
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.empty(T, 64, 512, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    at = [0, 1, 32767, 32768, 65535, 65536, 65999]
    x = q[at].double().cpu().numpy()
    k = q[:, 5].clone()
    xk = k[at].double().cpu().numpy()
    cs, ws = csa2.rope_table(P), csa2.Workspace(256)
    pos = torch.arange(T, device="cuda") % P
    rows = torch.empty(T, 512, dtype=torch.uint8, device="cuda")
    csa2.qk_norm_rope(pos, cs.cuda(), ws, q=q, q_out=q, k=k, rows=rows)
    assert ws.sync_status()[0] == 0
    for n, t in enumerate(at):
        check(q[t].double().cpu().numpy(), x[n], None, cs[t % P].numpy(), 1e-6, ref.U_BF16)
        check(ref.row_values(rows[t].cpu().numpy()), xk[n], None, cs[t % P].numpy(), 1e-6, ref.U_E4M3)


@pytest.mark.parametrize("T,q_gap,k_gap,weights,fp8,eps", [
    (600, 0, 0, True, False, 1e-6), (601, 8, 8, False, True, 1e-6), (777, 640, 24, True, True, 1e-5)])
def test_long_calls_against_the_formula(T, q_gap, k_gap, weights, fp8, eps):
    """From 600 tokens on a warp takes two heads."""
    test_against_the_formula(T, q_gap, k_gap, weights, fp8, eps)


@pytest.mark.parametrize("parts", ["both", "q", "k", "in place"])
def test_a_long_call_is_its_tokens_calls(parts):
    """A long call gives the bits of short ones, padding, bad positions and bad slots among its tokens."""
    T = 1203
    q, k, qw, kw = make(9, T, 64, 8)
    cs, ws = csa2.rope_table(P).cuda(), csa2.Workspace(256)
    rng = np.random.default_rng(9)
    pos, slot = rng.integers(0, P, T), rng.permutation(T + 40)[:T]
    pos[rng.integers(0, T, 60)] = -1
    pos[[7, 650]], pos[[8, 900]] = P, -2
    slot[rng.integers(0, T, 30)] = -1
    slot[[11, 700]] = T + 40
    pos, slot = torch.from_numpy(pos).cuda(), torch.from_numpy(slot).cuda()
    got = []
    for step in (T, 401):
        src = q.contiguous() if parts == "in place" else q
        out = src if parts == "in place" else torch.full((T, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        rows = torch.full((T + 40, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        for a in range(0, T, step):
            s = slice(a, a + step)
            kw_q = {} if parts == "k" else dict(q=src[s], q_weight=qw, q_out=out[s])
            kw_k = {} if parts == "q" else dict(k=k[s], k_weight=kw, rows=rows, k_slot=slot[s])
            csa2.qk_norm_rope(pos[s], cs, ws, **kw_q, **kw_k)
        assert ws.sync_status()[0] == 6
        got.append((out, rows))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
