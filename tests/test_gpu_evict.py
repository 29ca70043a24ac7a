"""Eviction (csa2_evict, 4-bit and 8-bit cache) against its definition, bit for bit: which
units stay, what moves where, and what is left alone."""
import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2
from tests import cache8_ref as c8

pytestmark = pytest.mark.gpu
D = 512
ARRAYS = {4: ("main_kv", "idx_codes", "idx_scales"), 8: ("codes", "scales")}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_cache(seed, bits, B, cap, n, index=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = csa2.Cache8(B, cap, 1) if bits == 8 else csa2.Cache(B, cap, 1, index=index)
    for name in ARRAYS[bits]:
        t = getattr(c, name)
        if t is None:
            continue
        if t.dtype == torch.float32:
            t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
        else:
            lo, hi = (0, 256) if t.dtype == torch.uint8 else (-127, 128)
            t.copy_(torch.randint(lo, hi, t.shape, generator=g, device="cuda", dtype=t.dtype))
    c.n_entries.copy_(dev(np.asarray(n, np.int32)))
    return c


def make_weights(seed, B, cap, kind):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal((B, cap))).astype(np.float32)
    if kind == "ties":
        w = np.round(rng.random((B, cap)) * 3).astype(np.float32) * np.float32(0.25)
    elif kind == "equal":
        w[:] = 1.0
    elif kind == "rising":
        w[:] = np.arange(cap)
    elif kind == "falling":
        w[:] = -np.arange(cap, dtype=np.float32)
    elif kind == "any":                                                            # signs, zeros of both, infinities, NaN
        w = rng.standard_normal((B, cap)).astype(np.float32) * 1e-3
        at = rng.integers(0, 8, (B, cap))
        for k, v in enumerate([0.0, -0.0, np.inf, -np.inf, np.nan]):
            w[at == k] = v
    return w


def run_and_check(bits, unit, B, cap, n, budget, first, recent, w, in_place, to_cap=None, with_weights=True, index=True,
                  alias_n=False, status=0, own_weights=False, seed=0):
    cache = make_cache(seed, bits, B, cap, n, index)
    cap = cache.cap
    names = [a for a in ARRAYS[bits] if getattr(cache, a) is not None]
    had = {a: getattr(cache, a).cpu().numpy().copy() for a in names}
    to = cache if in_place else make_cache(seed + 1, bits, B, to_cap or budget, [0] * B, index)
    before = {a: getattr(to, a).cpu().numpy().copy() for a in names}
    weights = dev(w)
    to_w = None
    if with_weights:
        to_w = weights if in_place and not own_weights else torch.full((B, to.cap), 7.0, device="cuda")
    kept = torch.full((B, budget // unit), 99, dtype=torch.int32, device="cuda")
    n_out = cache.n_entries if alias_n else torch.full((B,), 99, dtype=torch.int32, device="cuda")
    ws = csa2.Workspace(csa2.evict_workspace_size(cache, budget, unit))
    csa2.evict(cache, weights, kept, n_out, ws, budget=budget, unit=unit, first=first, recent=recent,
               to=None if in_place else to, to_weights=to_w)
    assert ws.sync_status()[0] == status
    for b in range(B):
        nb = min(max(n[b], 0), cap)
        units, entries = c8.evicted(w[b], nb, unit, budget, first, recent)
        want = np.full(budget // unit, -1)
        want[:len(units)] = units
        assert np.array_equal(kept[b].cpu().numpy(), want), b
        assert n_out[b].item() == len(entries)
        for a in names:
            rows = before[a][b].copy()
            if a == "scales":
                rows[:len(units)] = had[a][b][units]
            else:
                rows[:len(entries)] = had[a][b][entries]
            assert np.array_equal(getattr(to, a)[b].cpu().numpy(), rows), (a, b)
        if to_w is not None:
            rows = np.zeros(to.cap, np.float32)
            rows[:len(entries)] = w[b, entries]
            assert np.array_equal(to_w[b].cpu().numpy().view(np.int32), rows.view(np.int32)), b
    if not in_place:
        for a in names:
            assert np.array_equal(getattr(cache, a).cpu().numpy(), had[a])
        assert np.array_equal(weights.cpu().numpy().view(np.int32), w.view(np.int32))


SMALL = [(4, 1, 2, 40, [37, 12], 16, 0, 0), (4, 1, 1, 8, [8], 1, 0, 1), (4, 1, 1, 8, [8], 1, 1, 0), (4, 1, 3, 1000, [1000, 0, 333], 333, 4, 64),
         (4, 8, 2, 1000, [997, 41], 200, 8, 16), (8, 8, 2, 1000, [997, 41], 200, 3, 20), (8, 8, 1, 24, [20], 16, 0, 0),
         (8, 8, 1, 3000, [2999], 2400, 0, 0), (4, 8, 1, 3000, [2993], 8, 0, 0), (4, 1, 1, 3000, [2900], 2899, 1, 1)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "rising", "falling", "any"])
@pytest.mark.parametrize("bits,unit,B,cap,n,budget,first,recent", SMALL)
def test_evict(bits, unit, B, cap, n, budget, first, recent, kind, in_place):
    cap = -(-cap // 8) * 8
    run_and_check(bits, unit, B, cap, n, budget, first, recent, make_weights(cap, B, cap, kind), in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bits,unit", [(4, 1), (4, 8), (8, 8)])
def test_evict_many_chunks(bits, unit, in_place):
    """Long sequences: many chunks in flight, slices of keys of several turns; few and many entries leave."""
    for n, budget, kind in ((70_001, 69_000, "spread"), (70_001, 8_000, "ties"), (40_000, 39_992, "falling")):
        cap = -(-n // 8) * 8
        run_and_check(bits, unit, 2, cap, [n, n - 12_345], budget // unit * unit, 16, 100, make_weights(n, 2, cap, kind), in_place)


def test_evict_slices_beyond_shared_memory():
    n = 8 * 49_152 + 4_321
    cap = -(-n // 8) * 8
    run_and_check(4, 1, 1, cap, [n], 200_000, 4, 128, make_weights(1, 1, cap, "ties"), True, index=False)
    run_and_check(4, 1, 1, cap, [n], 3_000, 0, 0, make_weights(2, 1, cap, "spread"), False, index=False)


@pytest.mark.parametrize("B", [1, 9])
def test_evict_slices_of_every_cluster_beyond_shared_memory(B):
    """One sequence: 16 CTAs; nine: 8 CTAs each.  The keys of a slice are read anew in every pass."""
    n = 16 * 49_152 + 1_234 if B == 1 else 8 * 49_152 + 1_234
    cap = -(-n // 8) * 8
    w = make_weights(3, B, cap, "ties" if B == 1 else "spread")
    run_and_check(4, 1, B, cap, [n - 1000 * b for b in range(B)], 150_000, 4, 100, w, B == 1, index=False)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_without_weights_or_index_keys(in_place):
    w = make_weights(3, 2, 304, "spread")
    run_and_check(4, 1, 2, 304, [300, 304], 100, 0, 0, w, in_place, with_weights=False, index=False)
    run_and_check(8, 8, 2, 304, [300, 304], 104, 0, 0, w, in_place, with_weights=False)


def test_evict_weights_to_their_own_buffer_in_place():
    w = make_weights(4, 2, 1000, "falling")                                        # the first ones stay where they are
    run_and_check(4, 1, 2, 1000, [1000, 200], 500, 0, 0, w, True, own_weights=True)


def test_evict_into_a_larger_cache_and_n_entries_itself():
    w = make_weights(5, 3, 504, "spread")
    run_and_check(4, 1, 3, 504, [500, 100, 0], 200, 0, 8, w, False, to_cap=40_000)
    run_and_check(8, 8, 3, 504, [500, 100, 3], 200, 0, 8, w, True, alias_n=True)


def test_evict_reports():
    w = make_weights(6, 2, 64, "spread")
    run_and_check(4, 1, 2, 64, [70, 64], 20, 0, 0, w, False, status=6)
    run_and_check(4, 1, 2, 64, [-5, 64], 20, 0, 0, w, False)


def test_evict_captured_twice_on_one_workspace():
    """Two captured calls share a workspace and are replayed in turn; eight runs of the same call agree."""
    B, cap, budget = 2, 20_000, 6_000
    w = make_weights(7, B, cap, "ties")
    cache, ws = make_cache(7, 4, B, cap, [cap, 15_000]), None
    ws = csa2.Workspace(csa2.evict_workspace_size(cache, budget, 1))
    weights = dev(w)
    runs = []
    for k in range(2):
        to = make_cache(8 + k, 4, B, budget, [0] * B)
        kept, n_out = torch.zeros(B, budget, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        csa2.evict(cache, weights, kept, n_out, ws, budget=budget, to=to, recent=64 * k)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            csa2.evict(cache, weights, kept, n_out, ws, budget=budget, to=to, recent=64 * k)
        runs.append((graph, to, kept, to.main_kv.clone(), kept.clone()))
    for _ in range(4):
        for graph, to, kept, rows, had in runs:
            to.main_kv.zero_()
            kept.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(kept, had) and torch.equal(to.main_kv, rows)
    assert ws.sync_status()[0] == 0


def test_evict_offsets_beyond_32_bits():
    cap, budget = 8_000_000, 5_000_000                                             # 2.3 GB a sequence
    cache = csa2.Cache(2, cap, 1, index=False)
    kv = cache.main_kv
    kv[..., :8] = torch.arange(2 * cap, device="cuda").view(2, cap, 1).expand(-1, -1, 1).contiguous().view(torch.uint8).view(2, cap, 8)
    cache.n_entries.copy_(dev(np.array([cap, cap], np.int32)))
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.rand(2, cap, generator=g, device="cuda")
    kept, n_out = torch.zeros(2, budget, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = csa2.Workspace(csa2.evict_workspace_size(cache, budget, 1))
    csa2.evict(cache, w, kept, n_out, ws, budget=budget)
    assert ws.sync_status()[0] == 0 and n_out.tolist() == [budget, budget]
    for b in range(2):
        order = torch.sort(w[b], descending=True, stable=True).indices[:budget].sort().values
        assert torch.equal(kept[b].long(), order)
        assert torch.equal(kv[b, :budget, :8].contiguous().view(torch.int64)[:, 0], order + b * cap)
