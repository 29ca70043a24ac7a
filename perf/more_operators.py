"""Cases of the 8-bit cache and of eviction: the write of entries in 8 bits with one
scale for each block of 8 (``write8``), the attention over such a cache (``attn8``),
the attention weight that every cache entry has gathered (``weights``, 4-bit or 8-bit
cache), and the eviction of the entries that gathered least (``evict``).

``own`` false: plain torch in 32 bits.  ``own`` true: the library's calls.
"""
import math

import numpy as np
import torch

own = False

H, D, BLK, WIN = 64, 512, 8, 128           # query heads, latent, entries of a block, the layer's window
SCALE = 1.0 / math.sqrt(D)
FLOOR = 2.0 ** -60                         # the least scale of a block
ARRAYS = ("main_kv", "idx_codes", "idx_scales")


def listed():
    return [
        # one decode step of 16 sequences appends an entry each, inside blocks that hold some: latency
        {"name": "write8 decode 16", "op": "write8", "B": 16, "T": 1, "start": 3000, "pad": 0, "fresh": False},
        # prefill chunks of odd, ragged lengths behind what is cached
        {"name": "write8 chunk 4x8191", "op": "write8", "B": 4, "T": 8191, "start": 1003, "pad": 700, "fresh": False},
        # one query over a short cache, no window: latency
        {"name": "attn8 decode 1x600", "op": "attn8", "B": 1, "Q": 1, "n": 600, "m": 1, "W": 0, "fp8": False,
         "ragged": 0, "pad": 0},
        # a decode step over long caches
        {"name": "attn8 decode 16x131072", "op": "attn8", "B": 16, "Q": 1, "n": 131072, "m": 1, "W": 128, "fp8": False,
         "ragged": 1000, "pad": 0},
        # a short padded chunk over odd lengths of an m = 2 cache, E4M3 window
        {"name": "attn8 chunk 3x37 10007", "op": "attn8", "B": 3, "Q": 37, "n": 10007, "m": 2, "W": 128, "fp8": True,
         "ragged": 3001, "pad": 5},
        # a prefill chunk over everything before it
        {"name": "attn8 chunk 2048 8192", "op": "attn8", "B": 1, "Q": 2048, "n": 8192, "m": 1, "W": 128, "fp8": False,
         "ragged": 0, "pad": 0},
        # the weights of one decode step over long 4-bit caches, added to what earlier steps gave
        {"name": "weights decode 16x131072", "op": "weights", "bits": 4, "B": 16, "Q": 1, "n": 131072, "m": 1,
         "ragged": 1000, "pad": 0, "decay": 1.0},
        # a short padded chunk over odd lengths of an 8-bit cache, older weights fading
        {"name": "weights 8-bit 3x37 10007", "op": "weights", "bits": 8, "B": 3, "Q": 37, "n": 10007, "m": 2,
         "ragged": 3001, "pad": 5, "decay": 0.9},
        # the weights that a prefill chunk gives, before a first eviction
        {"name": "weights chunk 2048 8192", "op": "weights", "bits": 4, "B": 1, "Q": 2048, "n": 8192, "m": 1,
         "ragged": 0, "pad": 0, "decay": 0.0},
        # a few short caches cut to odd sizes: latency
        {"name": "evict 4x2000 to 701", "op": "evict", "bits": 4, "unit": 1, "B": 4, "n": 2000, "m": 1, "budget": 701,
         "first": 4, "recent": 64, "ragged": 333},
        # long 4-bit caches with their index keys, halved entry by entry
        {"name": "evict 16x131072 to 65536", "op": "evict", "bits": 4, "unit": 1, "B": 16, "n": 131072, "m": 1,
         "budget": 65536, "first": 4, "recent": 128, "ragged": 1000},
        # one very long 8-bit cache, cut block by block
        {"name": "evict 8-bit 1048573 to 524288", "op": "evict", "bits": 8, "unit": 8, "B": 1, "n": 1048573, "m": 1,
         "budget": 524288, "first": 8, "recent": 1024, "ragged": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write8", "attn8", "weights", "evict"])
    if op == "write8":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, 32768 // B)
        return {"op": op, "B": B, "T": T, "start": _log(rng, 1, 4096) - 1, "pad": rng.choice([0, rng.randint(0, T)]),
                "fresh": rng.random() < 0.3}
    if op == "evict":
        bits = rng.choice([4, 8])
        unit = 8 if bits == 8 else rng.choice([1, 8])
        n = _log(rng, 64, 1048576)
        budget = max(40, _log(rng, 32, n)) // unit * unit
        return {"op": op, "bits": bits, "unit": unit, "B": _log(rng, 1, max(1, min(64, 1048576 // n))), "n": n,
                "m": rng.choice([1, 2]), "budget": budget, "first": rng.randint(0, min(8, budget // 8)),
                "recent": rng.randint(0, budget // 4), "ragged": rng.choice([0, rng.randint(0, n)])}
    n, m = _log(rng, 1, 131072), rng.choice([1, 2])
    BQ = _log(rng, 1, max(1, min(2048, 14_000_000 // n)))
    Q = min(1 if rng.random() < 0.4 else _log(rng, 1, BQ), n * m)
    case = {"op": op, "B": max(1, min(BQ // Q, 2_000_000 // n)), "Q": Q, "n": n, "m": m,
            "ragged": rng.choice([0, rng.randint(0, n)]), "pad": rng.choice([0, rng.randint(0, Q - 1)])}
    if op == "attn8":
        return {**case, "W": rng.choice([0, 128, _log(rng, 1, 1024)]), "fp8": rng.random() < 0.5}
    return {**case, "bits": rng.choice([4, 8]), "decay": rng.choice([0.0, 1.0, 0.9])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _latents(g, *shape):
    """bf16 rows of unit root mean square, as the norm and rotation leave them."""
    z = _randn(g, *shape, D)
    return (z * torch.rsqrt((z * z).mean(-1, keepdim=True))).to(torch.bfloat16)


def _cap(n):
    return -(-n // BLK) * BLK


def _lengths(case):
    """Entries of each sequence."""
    least = -(-case.get("Q", 1) // case["m"])
    return np.array([max(least, case["n"] - (case["ragged"] * b) % case["n"]) for b in range(case["B"])], np.int64)


def _positions(case, ns):
    """q_pos [B][Q]: the newest Q tokens of each sequence, -1 behind the last of a shorter one."""
    B, Q = case["B"], case["Q"]
    pos = (ns * case["m"] - Q)[:, None] + np.arange(Q)[None, :]
    for b in range(B):
        pos[b, max(1, Q - (case["pad"] * b) % Q):] = -1
    return pos


def _cache8(g, B, cap):
    """Codes [B][cap][512] and scales [B][cap / 8] of entries that came through the write."""
    codes = torch.empty(B, cap, D, device="cuda", dtype=torch.int8)
    scales = torch.empty(B, cap // BLK, device="cuda")
    for b in range(B):
        for a in range(0, cap, 65536):
            x = _latents(g, min(65536, cap - a))
            scales[b, a // BLK:(a + 65536) // BLK] = s = _block_scale(x.float().abs().unflatten(0, (-1, BLK)).amax((1, 2)))
            codes[b, a:a + 65536] = torch.round(x.double() / s.double().repeat_interleave(BLK)[:, None]).to(torch.int8)
    return codes, scales


def _cache4(g, B, cap, index):
    """Entries as the cache write leaves them: 256 bytes of E2M1 pairs, then 32 E4M3 scales; index keys."""
    def bytes_(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)
    kv = torch.cat([torch.cat([bytes_(0, 256, 1, cap, 256), bytes_(0x28, 0x30, 1, cap, 32)], -1) for _ in range(B)])
    return kv, bytes_(0, 256, B, cap, 64) if index else None, bytes_(110, 130, B, cap, 4) if index else None


def _own_cache(s, case, cap):
    import fp4_kv_cache_csa2_gb300 as csa2
    if case.get("bits", 8) == 8:
        c = csa2.Cache8(case["B"], BLK, case.get("m", 1))
        c.codes, c.scales = s["codes"], s["scales"]
    else:
        c = csa2.Cache(case["B"], BLK, case["m"], index=False)
        c.main_kv, c.idx_codes, c.idx_scales = s["main_kv"], s.get("idx_codes"), s.get("idx_scales")
    c.cap, c.n_entries = cap, s["n_entries"]
    return c


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if own:
        import fp4_kv_cache_csa2_gb300 as csa2
    B = case["B"]
    if case["op"] == "write8":
        T = case["T"]
        first = np.array([BLK * (case["start"] // BLK) if case["fresh"] else case["start"] + 5 * b for b in range(B)])
        count = np.array([T - (case["pad"] * b) % T for b in range(B)])
        cap = _cap(int((first + T).max()) + 2 * BLK)
        s["x"] = torch.cat([_latents(g, 1, T) for _ in range(B)])
        s["codes"], s["scales"] = _cache8(g, B, cap)
        s["start"], s["count"] = torch.from_numpy(first).cuda(), torch.from_numpy(count.astype(np.int32)).cuda()
        s["n_entries"] = s["start"].to(torch.int32)                    # what is cached before the call
        if own:
            s["cache"], s["ws"] = _own_cache(s, case, cap), csa2.Workspace(csa2.WS_HEADER_BYTES)
        return s
    cap, ns = _cap(case["n"]), _lengths(case)
    s["n_entries"] = torch.from_numpy(ns.astype(np.int32)).cuda()
    if case["op"] == "evict":
        out_cap = _cap(case["budget"])
        if case["bits"] == 8:
            s["codes"], s["scales"] = _cache8(g, B, cap)
            s["to_codes"] = torch.zeros(B, out_cap, D, device="cuda", dtype=torch.int8)
            s["to_scales"] = torch.zeros(B, out_cap // BLK, device="cuda")
        else:
            for name, t in zip(ARRAYS, _cache4(g, B, cap, True)):
                s[name], s["to_" + name] = t, torch.zeros(B, out_cap, t.shape[-1], device="cuda", dtype=torch.uint8)
        # gathered weights: a few entries have most, some have none
        w = torch.exp(2.0 * _randn(g, B, cap))
        s["weights"] = torch.where(torch.rand(B, cap, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
        s["to_weights"] = torch.zeros(B, out_cap, device="cuda")
        s["kept"] = torch.zeros(B, case["budget"] // case["unit"], device="cuda", dtype=torch.int32)
        s["n_out"] = torch.zeros(B, device="cuda", dtype=torch.int32)
        if own:
            s["cache"] = _own_cache(s, case, cap)
            to = {k[3:]: v for k, v in s.items() if k.startswith("to_")}
            s["to"] = _own_cache({**to, "n_entries": s["n_out"]}, case, out_cap)
            s["ws"] = csa2.Workspace(csa2.evict_workspace_size(s["cache"], case["budget"], case["unit"]))
        return s
    Q = case["Q"]
    pos = _positions(case, ns)
    s["pos"] = torch.from_numpy(pos).cuda()
    s["q"] = torch.cat([(1.5 * _randn(g, 1, Q, H, D)).to(torch.bfloat16) for _ in range(B)])
    if case.get("bits", 8) == 8:
        s["codes"], s["scales"] = _cache8(g, B, cap)
    else:
        s["main_kv"] = _cache4(g, B, cap, False)[0]
    if case["op"] == "attn8":
        W = case["W"]
        s["rows"] = s["base"] = None
        if W:
            base = np.maximum(0, pos[:, 0] - W + 1)
            rows = _latents(g, B, W - 1 + Q)
            s["rows"] = rows.to(torch.float8_e4m3fn).view(torch.uint8) if case["fp8"] else rows
            s["base"] = torch.from_numpy(base).cuda()
        s["out"] = torch.zeros(B, Q, H, D, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros(B, Q, H, device="cuda")
        if own:
            s["cache"] = _own_cache(s, case, cap)
            s["ws"] = csa2.Workspace(csa2.cache8_attn_workspace_size(B, Q, cap, W))
        return s
    # the log-sum-exp that the attention of the same queries gave: the entries, and a little for the window
    s["lse"] = torch.empty(B, Q, H, device="cuda")
    for b in range(B):
        keys = _entries(s, b)
        seen = _visible(case, s["pos"][b], int(ns[b]))
        for a in range(0, Q, 256):
            sc = torch.matmul(s["q"][b, a:a + 256].float(), keys.T) * SCALE
            sc.masked_fill_(~_below(cap, seen[a:a + 256])[:, None], -math.inf)
            s["lse"][b, a:a + 256] = torch.logsumexp(sc, -1) + 0.05
    s["prev"] = torch.rand(B, cap, generator=g, device="cuda") if case["decay"] else None
    s["weights"] = torch.zeros(B, cap, device="cuda")
    if own:
        s["cache"] = _own_cache(s, case, cap)
        s["ws"] = csa2.Workspace(csa2.attn_weights_workspace_size(B, Q, cap))
    return s


# ------------------------------------------------------------------ the calls and the plain forms
def run(s):
    c = s["case"]
    if not own:
        return {"write8": _plain_write8, "attn8": _plain_attn8, "weights": _plain_weights, "evict": _plain_evict}[c["op"]](s)
    import fp4_kv_cache_csa2_gb300 as csa2
    if c["op"] == "write8":
        csa2.cache8_write(s["cache"], s["x"], s["start"], s["ws"], n_new=s["count"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["op"] == "attn8":
        csa2.cache8_attn(s["cache"], s["q"], s["pos"], SCALE, s["out"], s["ws"], max_n=s["cache"].cap, W=c["W"],
                         swa=s["rows"], swa_base_pos=s["base"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "weights":
        csa2.attn_weights(s["cache"], s["q"], s["pos"], s["lse"], SCALE, s["weights"], s["ws"], max_n=s["cache"].cap,
                          prev=s["prev"], decay=c["decay"])
        return {"weights": s["weights"]}
    csa2.evict(s["cache"], s["weights"], s["kept"], s["n_out"], s["ws"], budget=c["budget"], unit=c["unit"],
               first=c["first"], recent=c["recent"], to=s["to"], to_weights=s["to_weights"])
    return _evicted(s)


def _evicted(s):
    names = ["to_codes", "to_scales"] if s["case"]["bits"] == 8 else ["to_" + a for a in ARRAYS]
    return {k: s[k] for k in ["kept", "n_out", "to_weights", *names]}


def _block_scale(most):
    """Scale of a block whose largest magnitude is `most`."""
    return (most.double() / 127.0).float().clamp(min=FLOOR)


def _plain_write8(s):
    x, codes, scales = s["x"], s["codes"], s["scales"]
    B, T = x.shape[:2]
    cap = codes.shape[1]
    nb = (T + 2 * BLK - 2) // BLK                                        # blocks that a run of T entries can touch
    block = (s["start"] // BLK).clamp(max=cap // BLK - nb)[:, None] + torch.arange(nb, device="cuda")
    entry = block[..., None] * BLK + torch.arange(BLK, device="cuda")   # [B][nb][8]
    i = entry - s["start"][:, None, None]
    new = (i >= 0) & (i < s["count"][:, None, None]) & (entry < cap)
    old = ~new & ((i < 0) | (entry < s["n_entries"][:, None, None])) & (entry < cap)
    touched = new.any(-1)
    seq = torch.arange(B, device="cuda")[:, None]
    rows = x[seq[..., None], i.clamp(0, T - 1)]                          # [B][nb][8][512] bf16
    most = torch.where(new, rows.abs().amax(-1).float(), 0.0).amax(-1)
    s_old = scales[seq, block]
    scale = _block_scale(most)
    scale = torch.where(old.any(-1), torch.maximum(scale, s_old), scale)
    by_block = codes.unflatten(1, (-1, BLK))
    had = by_block[seq, block]
    wide = scale.double()[..., None, None]
    kept = torch.round(had.double() * s_old.double()[..., None, None] / wide).to(torch.int8)
    fresh = torch.round(rows.double() / wide).to(torch.int8)
    value = torch.where(new[..., None], fresh, torch.where(old[..., None], kept, had))
    by_block[seq, block] = torch.where(touched[..., None, None], value, had)
    scales[seq, block] = torch.where(touched, scale, s_old)
    return {"codes": codes, "scales": scales}


def _dequantised(kv):
    """4-bit entries [..., 288] -> latents [..., 512]: E2M1 codes (even channel in the low nibble) times E4M3 scales."""
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=kv.device)
    values = torch.cat([half, -half])
    codes = kv[..., :256]
    v = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1).flatten(-2)
    scale = kv[..., 256:].contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (32, 16)) * scale[..., None]).flatten(-2)


def _entries(s, b):
    """Entries of sequence b in 32 bits, [cap][512]."""
    if "codes" in s:
        return s["codes"][b].float() * s["scales"][b].repeat_interleave(BLK)[:, None]
    return _dequantised(s["main_kv"][b])


def _visible(case, pos, n):
    """Entries that queries at these positions see."""
    return ((pos + 1) // case["m"]).clamp(min=0, max=n)


def _below(n, seen):
    return torch.arange(n, device=seen.device) < seen[..., None]


def _window_keys(rows, base, pos, W):
    """Keys [B][Q][W][512] of positions pos-W+1 .. pos and which of them are visible."""
    B = rows.shape[0]
    p = pos[..., None] - (W - 1) + torch.arange(W, device=pos.device)
    seen = (p >= 0) & (pos[..., None] >= 0)
    at = (p - base[:, None, None]).clamp(0, rows.shape[1] - 1)
    values = rows.view(torch.float8_e4m3fn).float() if rows.dtype == torch.uint8 else rows.float()
    return values[torch.arange(B, device=pos.device)[:, None, None], at], seen


def _plain_attn8(s):
    c = s["case"]
    q = s["q"].float()
    B, Q = q.shape[:2]
    entries = s["codes"].float() * s["scales"].repeat_interleave(BLK, 1)[..., None]
    n = entries.shape[1]
    visible = torch.minimum((s["pos"] + 1) // c["m"], s["n_entries"][:, None].long())
    sc = torch.matmul(q.flatten(1, 2), entries.transpose(-1, -2)).unflatten(1, (Q, H)) * SCALE
    parts = [torch.where(_below(n, visible)[:, :, None], sc, -math.inf)]
    if c["W"]:
        near, seen = _window_keys(s["rows"], s["base"], s["pos"], c["W"])
        parts.append(torch.where(seen[:, :, None], torch.matmul(q, near.transpose(-1, -2)) * SCALE, -math.inf))
    top = torch.stack([p.amax(-1) for p in parts]).amax(0)
    ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = [torch.exp(p - ref[..., None]) for p in parts]
    total = sum(x.sum(-1) for x in e)
    o = torch.matmul(e[0].flatten(1, 2), entries).unflatten(1, (Q, H))
    if c["W"]:
        o = o + torch.matmul(e[1], near)
    some = torch.where(total > 0, total, torch.ones_like(total))
    return {"out": (o / some[..., None]).to(torch.bfloat16), "lse": ref + torch.log(total)}


def _plain_weights(s):
    c = s["case"]
    q = s["q"].float()
    B, Q = q.shape[:2]
    if c["bits"] == 8:
        entries = s["codes"].float() * s["scales"].repeat_interleave(BLK, 1)[..., None]
    else:
        entries = _dequantised(s["main_kv"])
    n = entries.shape[1]
    visible = torch.minimum((s["pos"] + 1) // c["m"], s["n_entries"][:, None].long())
    sc = torch.matmul(q.flatten(1, 2), entries.transpose(-1, -2)).unflatten(1, (Q, H)) * SCALE
    p = torch.exp(sc - s["lse"][..., None])
    p = torch.where(_below(n, visible)[:, :, None], p, 0.0)
    w = p.sum((1, 2), dtype=torch.float64)
    if s["prev"] is not None:
        w = w + c["decay"] * s["prev"].double()
    out = torch.where(_below(n, s["n_entries"].long()), w.float(), s["weights"])
    return {"weights": out}


def _plain_evict(s):
    c = s["case"]
    unit, K = c["unit"], c["budget"] // c["unit"]
    n = s["n_entries"].long()[:, None]
    w = s["weights"]
    B, cap = w.shape
    w = torch.where(_below(cap, n[:, 0]), w, torch.zeros_like(w))
    value = w.unflatten(1, (-1, unit)).amax(-1).double()
    U = value.shape[1]
    u = torch.arange(U, device=w.device)
    count = (n + unit - 1) // unit
    forced = u < -(-c["first"] // unit)
    if c["recent"]:
        forced = forced | (u >= (n - c["recent"]).clamp(min=0) // unit)
    value = torch.where(forced, 1e41, value)
    value = torch.where(u < count, value, -1e41)
    best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :K]
    if best.shape[1] < K:
        best = torch.nn.functional.pad(best, (0, K - best.shape[1]))
    stays = torch.arange(K, device=w.device) < torch.clamp(count, max=K)
    kept = torch.sort(torch.where(stays, best, U), dim=1).values
    s["kept"].copy_(torch.where(stays, kept, -1))
    entry = (torch.where(stays, kept, 0)[..., None] * unit + torch.arange(unit, device=w.device)).flatten(1)
    there = stays.repeat_interleave(unit, 1) & (entry < n)
    s["n_out"].copy_(there.sum(1))
    seq = torch.arange(B, device=w.device)[:, None]
    at = entry.clamp(max=cap - 1)
    s["to_weights"].zero_()
    s["to_weights"][:, :K * unit] = torch.where(there, w[seq, at], 0.0)
    moved = [a for a in ("codes", *ARRAYS) if a in s]
    for a in moved:
        for b in range(B):
            s["to_" + a][b, :K * unit] = torch.where(there[b, :, None], s[a][b, at[b]], s["to_" + a][b, :K * unit])
    if "scales" in s:
        s["to_scales"][:, :K] = torch.where(stays, s["scales"][seq, torch.where(stays, kept, 0)], s["to_scales"][:, :K])
    return _evicted(s)


# ------------------------------------------------------------------ the definition in 64 bits
def _wide_entries(s, b):
    if "codes" in s:
        return s["codes"][b].double() * s["scales"][b].double().repeat_interleave(BLK)[:, None]
    magnitude = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    byte = s["main_kv"][b, :, :256].long()
    code = torch.empty(byte.shape[0], D, dtype=torch.int64, device="cuda")
    code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
    scale = s["main_kv"][b, :, 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return magnitude[code % 8] * (1.0 - 2.0 * (code // 8)) * scale


def exact(case, seed):
    s = prepare(case, seed)
    return {"write8": _exact_write8, "attn8": _exact_attn8, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _exact_write8(s):
    x = s["x"].float().cpu().numpy()
    codes, scales = s["codes"].cpu().numpy().copy(), s["scales"].cpu().numpy().copy()
    out = scales.astype(np.float64)
    for b, (first, count) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
        for r in range(first // BLK, -(-(first + count) // BLK)):
            lo, hi = max(first, BLK * r), min(first + count, BLK * r + BLK)
            rows = x[b, lo - first:hi - first].astype(np.float64)
            wide = max(np.abs(rows).max() / 127.0, FLOOR)
            before = slice(BLK * r, lo)                                  # (nothing is cached behind the call's entries)
            if lo > BLK * r and scales[b, r] > np.float32(wide):
                wide = float(scales[b, r])
            scale = float(np.float32(wide))
            codes[b, before] = np.rint(codes[b, before] * float(scales[b, r]) / scale)
            codes[b, lo:hi] = np.rint(rows / scale)
            out[b, r] = wide
    return {"codes": torch.from_numpy(codes).cuda(), "scales": torch.from_numpy(out).cuda()}


def _exact_attn8(s):
    c = s["case"]
    B, Q = s["pos"].shape
    out = torch.zeros(B, Q, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    pos, ns = s["pos"].tolist(), s["n_entries"].tolist()
    for b in range(B):
        entries = _wide_entries(s, b)
        near, base = entries[:0], 0
        if c["W"]:
            near = s["rows"][b].view(torch.float8_e4m3fn).double() if c["fp8"] else s["rows"][b].double()
            base = int(s["base"][b])
        for i in range(Q):
            t = pos[b][i]
            if t < 0:
                continue
            keys = torch.cat([entries[:min(ns[b], (t + 1) // c["m"])], near[max(0, t - c["W"] + 1) - base:t + 1 - base]])
            if keys.shape[0] == 0:
                continue
            logit = torch.einsum("hd,nd->hn", s["q"][b, i].double(), keys) / math.sqrt(D)
            out[b, i], lse[b, i] = torch.einsum("hn,nd->hd", torch.softmax(logit, -1), keys), torch.logsumexp(logit, -1)
    return {"out": out, "lse": lse}


def _exact_weights(s):
    c = s["case"]
    B, Q = s["pos"].shape
    out = s["weights"].double()
    ns, pos = s["n_entries"].tolist(), s["pos"].tolist()
    for b in range(B):
        entries = _wide_entries(s, b)
        total = torch.zeros(entries.shape[0], dtype=torch.float64, device="cuda")
        for i in range(Q):
            n = min(ns[b], (pos[b][i] + 1) // c["m"]) if pos[b][i] >= 0 else 0
            if n == 0:
                continue
            logit = torch.einsum("nd,hd->nh", entries[:n], s["q"][b, i].double()) / math.sqrt(D)
            total[:n] += torch.exp(logit - s["lse"][b, i].double()).sum(-1)
        if s["prev"] is not None:
            total += c["decay"] * s["prev"][b].double()
        out[b, :ns[b]] = total[:ns[b]]
    return {"weights": out}


def _exact_evict(s):
    c = s["case"]
    unit, K = c["unit"], c["budget"] // c["unit"]
    out = {k: v.cpu().numpy().copy() for k, v in _evicted(s).items()}
    weights = s["weights"].cpu().numpy()
    names = [a for a in ("codes", *ARRAYS) if a in s]
    had = {a: s[a].cpu().numpy() for a in names}
    out["to_weights"][:] = 0
    for b, n in enumerate(s["n_entries"].tolist()):
        U = -(-n // unit)
        best = np.array([weights[b, u * unit:min(n, u * unit + unit)].max() for u in range(U)]) if unit > 1 else weights[b, :n]
        must = np.zeros(U, bool)
        must[:-(-c["first"] // unit)] = True
        if c["recent"]:
            must[max(0, n - c["recent"]) // unit:] = True
        order = np.lexsort((np.arange(U), -best.astype(np.float64), ~must))
        kept = np.sort(order[:K])
        entries = (kept[:, None] * unit + np.arange(unit)).ravel()
        entries = entries[entries < n]
        out["kept"][b] = -1
        out["kept"][b, :len(kept)] = kept
        out["n_out"][b] = len(entries)
        out["to_weights"][b, :len(entries)] = weights[b, entries]
        for a in names:
            out["to_" + a][b, :len(entries)] = had[a][b, entries]
        if "scales" in s:
            out["to_scales"][b, :len(kept)] = s["scales"][b].cpu().numpy()[kept]
    return {k: torch.from_numpy(v).cuda() for k, v in out.items()}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B = case["B"]
    if case["op"] == "write8":
        T = case["T"]
        rows = sum(T - (case["pad"] * b) % T for b in range(B))
        return {"bytes": rows * (2 * D + D + 4 / BLK) + 12 * B, "flops": rows * D * 4}
    ns = _lengths(case)
    entry = D + 4 / BLK if case.get("bits", 8) == 8 else 288
    if case["op"] == "evict":
        stays = np.minimum(ns, case["budget"])
        entry = entry if case["bits"] == 8 else 288 + 64 + 4
        return {"bytes": float(4 * ns.sum() + stays.sum() * (2 * entry + 8 + 4 / case["unit"])), "flops": float(ns.sum())}
    pos = _positions(case, ns)
    entries = np.where(pos >= 0, np.minimum((pos + 1) // case["m"], ns[:, None]), 0)
    live = int((pos >= 0).sum())
    kv = float(entries.max(1).sum()) * entry
    q = live * H * D * 2 + 8 * pos.size
    if case["op"] == "weights":
        return {"bytes": q + live * H * 4 + kv + 4.0 * float(ns.sum()) * (2 if case["decay"] else 1),
                "flops": float(entries.sum()) * H * D * 2}
    W, row = case["W"], D * (1 if case["fp8"] else 2)
    near = np.where(pos >= 0, np.minimum(pos + 1, W), 0)
    if W:
        base = np.maximum(0, pos[:, 0] - W + 1)
        kv += float(sum(int(pos[b].max() - base[b] + 1) * row for b in range(B)))
    return {"bytes": q + pos.size * H * (D * 2 + 4) + kv, "flops": float(entries.sum() + near.sum()) * H * D * 4}
