"""The calls of the 8-bit cache, the gathered weights and the eviction as a server makes them,
one after another: a prompt is written and attended, its weights gathered, the cache
cut in place, and decoding goes on over what stayed and what is new."""
import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
import oracle
from tests import cache8_ref as c8
from tests import keys_ref as ref

pytestmark = pytest.mark.gpu
H, D = 64, 512
SCALE = 512 ** -0.5


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def queries(g, *shape):
    return (1.5 * torch.randn(*shape, H, D, generator=g)).bfloat16().cuda()


def check_attention(out, lse, q, keys, most=0.0):
    o, l, b_o, b_l = c8.attend(q.double().cpu().numpy(), keys, SCALE, most)
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= b_o)
    assert np.all(np.abs(lse.double().cpu().numpy() - l) <= b_l)


def check_weights(w, before, q, keys_of, lse):
    """w [cap] after the queries q [Q][64][512], query i over the entries keys_of[i]."""
    want, tol = before.astype(np.float64), 2.0 ** -22 * np.abs(before)
    for i, keys in enumerate(keys_of):
        a, t = c8.gathered(q[i].double().cpu().numpy(), keys, lse[i].double().cpu().numpy(), SCALE)
        want[:len(keys)] += a
        tol[:len(keys)] += t
    err = np.abs(w.double().cpu().numpy() - want)
    assert np.all(err <= tol), np.max(err - tol)


def test_8_bit_cache_from_prompt_to_decoding():
    B, T, cap, budget, steps = 2, 300, 336, 128, 5
    lens = np.array([300, 221])
    g = torch.Generator().manual_seed(1)
    rope = csa2.rope_table(T + steps).cuda()
    cache, ws = csa2.Cache8(B, cap, 1), csa2.Workspace(1 << 26)
    k = torch.randn(B, T, D, generator=g).bfloat16().cuda()
    pos = np.where(np.arange(T)[None] < lens[:, None], np.arange(T)[None], -1)
    rows = torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    csa2.qk_norm_rope(dev(pos.ravel()), rope, ws, k=k.flatten(0, 1), rows=rows)
    csa2.cache8_write(cache, rows, torch.zeros(B, dtype=torch.int64, device="cuda"), ws, n_new=dev(lens.astype(np.int32)))
    cache.n_entries.copy_(dev(lens.astype(np.int32)))
    # the prompt's last queries, their weights, the cut
    Q = 4
    q = queries(g, B, Q)
    q_pos = lens[:, None] - Q + np.arange(Q)[None]
    out, lse = torch.zeros(B, Q, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Q, H, device="cuda")
    w = torch.zeros(B, cap, device="cuda")
    csa2.cache8_attn(cache, q, dev(q_pos), SCALE, out, ws, max_n=cap, lse=lse)
    csa2.attn_weights(cache, q, dev(q_pos), lse, SCALE, w, ws, max_n=cap)
    values = [c8.entries(cache.codes[b].cpu().numpy(), cache.scales[b].cpu().numpy())[:lens[b]] for b in range(B)]
    weights = w.cpu().numpy().copy()
    for b in range(B):
        for i in range(Q):
            check_attention(out[b, i], lse[b, i], q[b, i], values[b][:q_pos[b, i] + 1], cache.scales[b].max().item())
        check_weights(w[b], np.zeros(cap, np.float32), q[b], [values[b][:t + 1] for t in q_pos[b]], lse[b])
    kept = torch.zeros(B, budget // 8, dtype=torch.int32, device="cuda")
    csa2.evict(cache, w, kept, cache.n_entries, ws, budget=budget, unit=8, first=8, recent=16, to_weights=w)
    n = cache.n_entries.cpu().numpy().astype(np.int64)
    for b in range(B):
        units, entries = c8.evicted(weights[b], lens[b], 8, budget, 8, 16)
        assert n[b] == len(entries) and kept[b].tolist() == units.tolist()
        values[b], weights[b] = values[b][entries], np.concatenate([weights[b, entries], np.zeros(cap - len(entries), np.float32)])
    left = lens - n
    # decoding: new rows keep their real positions, the cache's numbers are shifted
    out, lse = out[:, :1].contiguous(), lse[:, :1].contiguous()
    for step in range(steps):
        t = lens + step
        row = torch.zeros(B, 1, D, dtype=torch.bfloat16, device="cuda")
        csa2.qk_norm_rope(dev(t), rope, ws, k=torch.randn(B, D, generator=g).bfloat16().cuda(), rows=row)
        csa2.cache8_write(cache, row, cache.n_entries.long(), ws)
        cache.n_entries.add_(1)
        q = queries(g, B, 1)
        csa2.cache8_attn(cache, q, dev((t - left)[:, None]), SCALE, out, ws, max_n=cap, lse=lse)
        csa2.attn_weights(cache, q, dev((t - left)[:, None]), lse, SCALE, w, ws, max_n=cap, prev=w)
        for b in range(B):
            now = c8.entries(cache.codes[b].cpu().numpy(), cache.scales[b].cpu().numpy())[:n[b] + step + 1]
            s = cache.scales[b].max().item()
            assert np.all(np.abs(now[:-1] - values[b]) <= s)                       # kept codes may be rounded again
            assert np.all(np.abs(now[-1] - row[b, 0].double().cpu().numpy()) <= 0.5001 * s)
            check_attention(out[b, 0], lse[b, 0], q[b, 0], now, s)
            check_weights(w[b], weights[b], q[b], [now], lse[b])
            values[b], weights[b] = now, w[b].cpu().numpy()
    assert ws.sync_status()[0] == 0


def test_4_bit_cache_cut_and_written_on():
    B, T, m, budget = 2, 600, 2, 100
    n0, cap, more = T // m, 320, 8
    g = torch.Generator().manual_seed(2)
    rope = csa2.rope_table(n0 + 16).cuda()
    x = (0.5 * torch.randn(B, T + more, D, generator=g)).bfloat16().cuda()
    w0, w1 = (0.5 + torch.rand(2, D, generator=g)).cuda()
    w_idx = (torch.randn(128, D, generator=g) / 20).bfloat16().cuda()
    cache, whole, ws = csa2.Cache(B, cap, m), csa2.Cache(B, cap, m), csa2.Workspace(1 << 26)
    zero = torch.zeros(B, dtype=torch.int64, device="cuda")
    csa2.compress_quantize(cache, x[:, :T].contiguous(), zero, w0, w1, rope, w_idx, ws)
    csa2.compress_quantize(whole, x, zero, w0, w1, rope, w_idx, ws)                  # never cut
    cache.n_entries.fill_(n0)
    swa = torch.randn(B, 256, D, generator=g).bfloat16().cuda()
    base = T + more - 256
    q, pos = queries(g, B, 3), np.full((B, 1), T - 3) + np.arange(3)[None]
    out, lse = torch.zeros(B, 3, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 3, H, device="cuda")
    w = torch.zeros(B, cap, device="cuda")
    csa2.dense_attn(cache, q, swa, dev(np.full(B, base)), dev(pos), SCALE, out, ws, max_n=cap, lse=lse)
    csa2.attn_weights(cache, q, dev(pos), lse, SCALE, w, ws, max_n=cap)
    values = [oracle.dequant_main(cache.main_kv[b].cpu().numpy()).astype(np.float64) for b in range(B)]
    near = ref.row_values(swa.view(torch.int16).cpu().numpy().view(np.uint16))
    for b in range(B):
        check_weights(w[b], np.zeros(cap, np.float32), q[b], [values[b][:(t + 1) // m] for t in pos[b]], lse[b])
    weights = w.cpu().numpy()
    kept = torch.zeros(B, budget, dtype=torch.int32, device="cuda")
    csa2.evict(cache, w, kept, cache.n_entries, ws, budget=budget, first=4, recent=32, to_weights=w)
    left = n0 - budget
    # four more entries, at their real rotation
    for b in range(B):
        csa2.compress_quantize(cache.sequence(b), x[b:b + 1, T:].contiguous(), torch.full((1,), budget, device="cuda"), w0, w1,
                               rope[left:].contiguous(), w_idx, ws)
    cache.n_entries.add_(more // m)
    n = budget + more // m
    for b in range(B):
        _, entries = c8.evicted(weights[b], n0, 1, budget, 4, 32)
        entries = np.concatenate([entries, n0 + np.arange(more // m)])
        for name in ("main_kv", "idx_codes", "idx_scales"):
            a, o = getattr(cache, name)[b].cpu().numpy(), getattr(whole, name)[b].cpu().numpy()
            assert np.array_equal(a[:n], o[entries]), name
    # decoding over it, without a selection and with one that takes every entry
    t = T + more - 1
    q, pos = queries(g, B, 1), np.full((B, 1), t - m * left)
    out, lse = out[:, :1].contiguous(), lse[:, :1].contiguous()
    csa2.dense_attn(cache, q, swa, dev(np.full(B, base - m * left)), dev(pos), SCALE, out, ws, max_n=cap, lse=lse)
    chosen, sel = torch.zeros_like(out), torch.zeros(B, 1, 512, dtype=torch.int32, device="cuda")
    csa2.decode(csa2.MODE_FULL, cache, q_pos=dev(pos), q=q, swa=swa, swa_base_pos=dev(np.full(B, base - m * left)), scale=SCALE, sel=sel,
                out=chosen, ws=ws, M=64, max_n=cap, q_idx=torch.randn(B, 1, 32, 128, generator=g).bfloat16().cuda(),
                w_head=torch.rand(B, 1, 32, generator=g).cuda(), pool_blocks=torch.zeros(B, 1, 64, dtype=torch.int32, device="cuda"))
    assert ws.sync_status()[0] == 0
    for b in range(B):
        keys = np.concatenate([oracle.dequant_main(cache.main_kv[b, :n].cpu().numpy()).astype(np.float64), near[b, t - 127 - base:t + 1 - base]])
        check_attention(out[b, 0], lse[b, 0], q[b, 0], keys)
        assert sel[b, 0, :n].tolist() == list(range(n)) and sel[b, 0, n].item() == -1
        check_attention(chosen[b, 0], lse[b, 0], q[b, 0], keys)


def test_two_streams_at_once():
    """The same chain of calls on two streams, each with its caches and its workspace, eight times over."""
    B, cap, budget = 4, 20_000, 6_000

    def chain(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache, to = csa2.Cache8(B, cap, 1), csa2.Cache8(B, budget, 1)
        x = torch.randn(B, cap, D, generator=g, device="cuda").bfloat16()
        q = torch.randn(B, 2, H, D, generator=g, device="cuda").bfloat16()
        pos = torch.tensor([[cap - 2, cap - 1]] * B, device="cuda")
        out, lse = torch.zeros(B, 2, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 2, H, device="cuda")
        w, to_w = torch.zeros(B, cap, device="cuda"), torch.zeros(B, budget, device="cuda")
        kept, n = torch.zeros(B, budget // 8, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        ws = csa2.Workspace(max(csa2.cache8_attn_workspace_size(B, 2, cap), csa2.attn_weights_workspace_size(B, 2, (1 << 31) - 1),
                                csa2.evict_workspace_size(cache, budget, 8)))
        zero = torch.zeros(B, dtype=torch.int64, device="cuda")
        cache.n_entries.fill_(cap)

        def run(stream=None):
            csa2.cache8_write(cache, x, zero, ws, stream=stream)
            csa2.cache8_attn(cache, q, pos, SCALE, out, ws, max_n=cap, stream=stream)
            csa2.cache8_attn(cache, q, pos, SCALE, out, ws, max_n=cap, lse=lse, stream=stream)
            csa2.attn_weights(cache, q, pos, lse, SCALE, w, ws, max_n=(1 << 31) - 1, stream=stream)
            csa2.evict(cache, w, kept, n, ws, budget=budget, unit=8, to=to, to_weights=to_w, stream=stream)
        return run, (cache.codes, cache.scales, out, lse, w, to_w, kept, n, to.codes, to.scales), ws

    chains = [chain(1), chain(2)]
    want = []
    for run, outputs, _ in chains:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outputs])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for run, outputs, _ in chains:
            for t in outputs[2:]:
                t.zero_()
        torch.cuda.synchronize()
        for (run, _, _), s in zip(chains, streams):
            run(s)
        torch.cuda.synchronize()
        for (_, outputs, ws), had in zip(chains, want):
            assert ws.sync_status()[0] == 0
            for t, u in zip(outputs, had):
                assert torch.equal(t, u)
