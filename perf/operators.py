"""Cases of the operators around the layer's attention: the per-head norm and
rotation of queries and window keys (``norm_rope``), the attention of a
window-only layer with a few first tokens that stay visible (``window``), and
the attention over every visible entry of the 4-bit cache (``dense``).

``own`` false: plain torch in 32 bits.  ``own`` true: the library's calls.
"""
import math

import numpy as np
import torch

own = False

H, D, ROT, WIN = 64, 512, 64, 128          # query heads, latent, rotated tail, the layer's window
THETA = 160000.0
EPS = 1e-6
SCALE = 1.0 / math.sqrt(D)


def listed():
    return [
        # one decode step of 16 sequences: latency of a small call
        {"name": "norm_rope decode 16", "op": "norm_rope", "T": 16, "fp8": False, "weights": True, "pad": 0,
         "start": 131000, "gap": 0},
        # a ragged batch, padding tokens among them, queries inside a wider fused projection
        {"name": "norm_rope ragged 777", "op": "norm_rope", "T": 777, "fp8": False, "weights": True, "pad": 45,
         "start": 3, "gap": 640},
        # a prefill chunk of 8192 tokens with the window stored as E4M3
        {"name": "norm_rope chunk 8192", "op": "norm_rope", "T": 8192, "fp8": True, "weights": False, "pad": 0,
         "start": 16384, "gap": 0},
        # one decode step of a window-only layer, 16 sequences
        {"name": "window decode 16", "op": "window", "B": 16, "Q": 1, "W": 128, "sinks": 4, "fp8": False,
         "start": 4095, "pad": 0},
        # verification of three drafted tokens per sequence, E4M3 rows, odd window without sinks
        {"name": "window verify 40x3", "op": "window", "B": 40, "Q": 3, "W": 99, "sinks": 0, "fp8": True,
         "start": 700, "pad": 1},
        # a prefill chunk of a window-only layer
        {"name": "window chunk 8192", "op": "window", "B": 1, "Q": 8192, "W": 128, "sinks": 4, "fp8": False,
         "start": 8192, "pad": 0},
        # a wide window on a short chunk of two sequences, E4M3 rows
        {"name": "window wide 1000", "op": "window", "B": 2, "Q": 301, "W": 1000, "sinks": 17, "fp8": True,
         "start": 2500, "pad": 100},
        # one query over a short cache: latency
        {"name": "dense decode 1x600", "op": "dense", "B": 1, "Q": 1, "n": 600, "m": 1, "fp8": False, "ragged": 0},
        # a decode step over long caches
        {"name": "dense decode 16x131072", "op": "dense", "B": 16, "Q": 1, "n": 131072, "m": 1, "fp8": False,
         "ragged": 1000},
        # a short chunk over odd lengths of an m = 2 cache, E4M3 window
        {"name": "dense chunk 3x37 10007", "op": "dense", "B": 3, "Q": 37, "n": 10007, "m": 2, "fp8": True,
         "ragged": 3001},
        # a prefill chunk over everything before it
        {"name": "dense chunk 2048 8192", "op": "dense", "B": 1, "Q": 2048, "n": 8192, "m": 1, "fp8": False,
         "ragged": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "window", "dense"])
    fp8 = rng.random() < 0.5
    if op == "norm_rope":
        T = _log(rng, 1, 8192)
        return {"op": op, "T": T, "fp8": fp8, "weights": rng.random() < 0.6, "pad": rng.randint(0, T // 4),
                "start": _log(rng, 1, 200000) - 1, "gap": rng.choice([0, 8, 512, 1000])}
    if op == "window":
        W, sinks = _log(rng, 1, 2048), rng.choice([0, 1, 4, rng.randint(0, 128)])
        BQ = _log(rng, 1, min(8192, 1_000_000 // (W + sinks + 1)))
        Q = 1 if rng.random() < 0.3 else _log(rng, 1, BQ)
        return {"op": op, "B": max(1, BQ // Q), "Q": Q, "W": W, "sinks": sinks, "fp8": fp8,
                "start": _log(rng, 1, 100000) - 1, "pad": rng.choice([0, rng.randint(0, Q)])}
    n, m = _log(rng, 1, 131072), rng.choice([1, 2])
    BQ = _log(rng, 1, max(1, min(4096, 14_000_000 // n)))
    Q = min(1 if rng.random() < 0.4 else _log(rng, 1, BQ), n * m)
    return {"op": op, "B": max(1, min(BQ // Q, 2_000_000 // n)), "Q": Q, "n": n, "m": m, "fp8": fp8,
            "ragged": rng.choice([0, rng.randint(0, n)])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, fp8, *shape):
    """Window rows of unit root mean square, as stored: bf16, or E4M3 bytes."""
    z = _randn(g, *shape, D)
    z = (z * torch.rsqrt((z * z).mean(-1, keepdim=True))).to(torch.bfloat16)
    return z.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else z


def _table(P):
    """cos and sin of p * THETA^(-2i/64), p < P, as the library's table has them."""
    ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * \
        THETA ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device="cuda") / ROT)
    return torch.stack([ang.cos(), ang.sin()], -1).to(torch.float32).contiguous()


def _window_positions(case):
    """q_pos [B][Q] (-1 behind the last query of a sequence) and the first position of each row buffer."""
    B, Q = case["B"], case["Q"]
    first = [max(0, case["start"] - 37 * b) for b in range(B)]
    live = [max(1, Q - (case["pad"] * b) % Q) if Q > 1 else 1 for b in range(B)]
    pos = np.full((B, Q), -1, np.int64)
    for b in range(B):
        pos[b, :live[b]] = first[b] + np.arange(live[b])
    return pos, np.array([max(0, f - case["W"] + 1) for f in first], np.int64)


def _dense_positions(case):
    """q_pos [B][Q], entries per sequence and the first position of each window buffer: the newest Q tokens of each sequence."""
    B, Q, n, m = case["B"], case["Q"], case["n"], case["m"]
    ns = np.array([max(-(-Q // m), n - (case["ragged"] * b) % n) for b in range(B)], np.int64)
    last = ns * m - 1
    pos = last[:, None] - (Q - 1) + np.arange(Q)[None, :]
    return pos, ns, np.maximum(0, pos[:, 0] - WIN + 1)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm_rope":
        T, gap = case["T"], case["gap"]
        qk = torch.empty(T, H * D + gap, device="cuda", dtype=torch.bfloat16)     # the projections' output
        for a in range(0, T, 2048):
            qk[a:a + 2048] = (2.0 * _randn(g, min(2048, T - a), H * D + gap)).to(torch.bfloat16)
        s["q"] = qk[:, :H * D].unflatten(1, (H, D))
        s["k"] = _randn(g, T, D).to(torch.bfloat16)
        pos = torch.arange(T, device="cuda") + case["start"]
        if case["pad"]:
            pos[torch.randperm(T, generator=g, device="cuda")[:case["pad"]]] = -1
        s["pos"] = pos
        s["slot"] = torch.randperm(T + 5, generator=g, device="cuda")[:T]            # rows of the window buffer
        s["table"] = _table(case["start"] + T)
        s["q_weight"] = 1.0 + 0.2 * _randn(g, D) if case["weights"] else None
        s["k_weight"] = 1.0 + 0.2 * _randn(g, D) if case["weights"] else None
        s["q_out"] = torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16)
        s["rows"] = torch.zeros(T + 5, D, device="cuda", dtype=torch.uint8 if case["fp8"] else torch.bfloat16)
        if own:
            import fp4_kv_cache_csa2_gb300 as csa2
            s["ws"] = csa2.Workspace(csa2.WS_HEADER_BYTES)
        return s
    B, Q = case["B"], case["Q"]
    s["q"] = torch.empty(B, Q, H, D, device="cuda", dtype=torch.bfloat16)
    for b in range(B):
        s["q"][b] = (1.5 * _randn(g, Q, H, D)).to(torch.bfloat16)
    s["out"] = torch.zeros(B, Q, H, D, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros(B, Q, H, device="cuda")
    if case["op"] == "window":
        pos, base = _window_positions(case)
        s["rows"] = _rows(g, case["fp8"], B, case["W"] - 1 + Q)
        s["sinks"] = _rows(g, case["fp8"], B, case["sinks"]) if case["sinks"] else None
        if own:
            import fp4_kv_cache_csa2_gb300 as csa2
            s["ws"] = csa2.Workspace(csa2.window_attn_workspace_size(B, Q, case["W"], case["sinks"]))
    else:
        pos, ns, base = _dense_positions(case)
        cap = -(-case["n"] // 8) * 8
        # entries as the cache write leaves them: 256 bytes of E2M1 pairs, then 32 E4M3 scales
        kv = torch.empty(B, cap, 288, device="cuda", dtype=torch.uint8)
        for b in range(B):
            kv[b, :, :256] = torch.randint(0, 256, (cap, 256), generator=g, device="cuda", dtype=torch.uint8)
            kv[b, :, 256:] = torch.randint(0x28, 0x30, (cap, 32), generator=g, device="cuda", dtype=torch.uint8)
        s["kv"], s["n_entries"] = kv, torch.from_numpy(ns.astype(np.int32)).cuda()
        s["rows"] = _rows(g, case["fp8"], B, WIN - 1 + Q)
        if own:
            import fp4_kv_cache_csa2_gb300 as csa2
            s["cache"] = csa2.Cache(B, cap, case["m"])
            s["cache"].main_kv, s["cache"].n_entries = kv, s["n_entries"]
            s["ws"] = csa2.Workspace(csa2.dense_attn_workspace_size(B, Q, cap))
    s["pos"], s["base"] = torch.from_numpy(pos).cuda(), torch.from_numpy(base).cuda()
    return s


# ------------------------------------------------------------------ the calls and the plain forms
def run(s):
    op = s["case"]["op"]
    if own:
        import fp4_kv_cache_csa2_gb300 as csa2
        if op == "norm_rope":
            csa2.qk_norm_rope(s["pos"], s["table"], s["ws"], q=s["q"], q_weight=s["q_weight"], q_out=s["q_out"],
                              k=s["k"], k_weight=s["k_weight"], rows=s["rows"], k_slot=s["slot"], eps=EPS)
            return {"q": s["q_out"],
                    "rows": s["rows"].view(torch.float8_e4m3fn) if s["case"]["fp8"] else s["rows"]}
        if op == "window":
            csa2.window_attn(s["q"], s["rows"], s["base"], s["pos"], SCALE, s["out"], s["ws"], W=s["case"]["W"],
                             sinks=s["sinks"], lse=s["lse"])
        else:
            csa2.dense_attn(s["cache"], s["q"], s["rows"], s["base"], s["pos"], SCALE, s["out"], s["ws"],
                            max_n=s["cache"].cap, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "norm_rope":
        return _plain_norm_rope(s)
    return _plain_window(s) if op == "window" else _plain_dense(s)


def _normed(x, weight, cs):
    x = x.float()
    y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + EPS)
    if weight is not None:
        y = y * weight
    even, odd = y[..., D - ROT::2], y[..., D - ROT + 1::2]
    c, sn = cs[..., 0], cs[..., 1]
    tail = torch.stack([even * c - odd * sn, even * sn + odd * c], -1).flatten(-2)
    return torch.cat([y[..., :D - ROT], tail], -1)


def _plain_norm_rope(s):
    live = s["pos"] >= 0
    cs = s["table"][s["pos"].clamp(min=0)]
    q = _normed(s["q"], s["q_weight"], cs[:, None]).to(torch.bfloat16)
    k = _normed(s["k"], s["k_weight"], cs)
    k = k.clamp(-448.0, 448.0).to(torch.float8_e4m3fn) if s["case"]["fp8"] else k.to(torch.bfloat16)
    q_out = torch.where(live[:, None, None], q, s["q_out"])
    rows = s["rows"].view(torch.float8_e4m3fn) if s["case"]["fp8"] else s["rows"]
    rows = rows.clone()
    byte = torch.uint8 if s["case"]["fp8"] else torch.bfloat16
    at = s["slot"][:, None].expand(-1, D)
    old = rows.view(byte).gather(0, at)
    rows.view(byte).scatter_(0, at, torch.where(live[:, None], k.view(byte), old))
    return {"q": q_out, "rows": rows}


def _values(rows):
    return rows.view(torch.float8_e4m3fn).float() if rows.dtype == torch.uint8 else rows.float()


def _window_keys(rows, base, pos, W):
    """Keys [B][Q][W][512] of positions pos-W+1 .. pos and which of them are visible."""
    B = rows.shape[0]
    p = pos[..., None] - (W - 1) + torch.arange(W, device=pos.device)
    seen = (p >= 0) & (pos[..., None] >= 0)
    at = (p - base[:, None, None]).clamp(0, rows.shape[1] - 1)
    return _values(rows)[torch.arange(B, device=pos.device)[:, None, None], at], seen


def _softmax_parts(parts):
    """parts: scores, with -inf where masked.  exp(score - max) of each, their sum, and its log."""
    top = torch.stack([p.max(-1).values for p in parts]).max(0).values
    ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = [torch.exp(p - ref[..., None]) for p in parts]
    total = sum(x.sum(-1) for x in e)
    return e, torch.where(total > 0, total, torch.ones_like(total)), ref + torch.log(total)


def _plain_window(s):
    c = s["case"]
    q = s["q"].float()
    keys, seen = _window_keys(s["rows"], s["base"], s["pos"], c["W"])
    parts = [torch.where(seen[:, :, None], torch.matmul(q, keys.transpose(-1, -2)) * SCALE, -math.inf)]
    if s["sinks"] is not None:
        first = _values(s["sinks"])
        old = torch.arange(c["sinks"], device=q.device) < (s["pos"][..., None] - c["W"] + 1)
        sc = torch.matmul(q.flatten(1, 2), first.transpose(-1, -2)).unflatten(1, q.shape[1:3]) * SCALE
        parts.append(torch.where(old[:, :, None], sc, -math.inf))
    e, total, lse = _softmax_parts(parts)
    o = torch.matmul(e[0], keys)
    if s["sinks"] is not None:
        o = o + torch.matmul(e[1].flatten(1, 2), first).unflatten(1, q.shape[1:3])
    return {"out": (o / total[..., None]).to(torch.bfloat16), "lse": lse}


def _dequantised(kv):
    """Entries [..., 288] -> latents [..., 512]: E2M1 codes (even channel in the low nibble) times E4M3 scales."""
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=kv.device)
    values = torch.cat([half, -half])
    codes = kv[..., :256]
    v = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1).flatten(-2)
    scale = kv[..., 256:].contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (32, 16)) * scale[..., None]).flatten(-2)


def _plain_dense(s):
    c = s["case"]
    q = s["q"].float()
    entries = _dequantised(s["kv"])
    near, seen = _window_keys(s["rows"], s["base"], s["pos"], WIN)
    n = entries.shape[1]
    visible = torch.minimum((s["pos"] + 1) // c["m"], s["n_entries"][:, None].long())
    sc = torch.matmul(q.flatten(1, 2), entries.transpose(-1, -2)).unflatten(1, q.shape[1:3]) * SCALE
    sc = torch.where(torch.arange(n, device=q.device) < visible[..., None, None], sc, -math.inf)
    e, total, lse = _softmax_parts(
        [sc, torch.where(seen[:, :, None], torch.matmul(q, near.transpose(-1, -2)) * SCALE, -math.inf)])
    o = torch.matmul(e[0].flatten(1, 2), entries).unflatten(1, q.shape[1:3]) + torch.matmul(e[1], near)
    return {"out": (o / total[..., None]).to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------ the definition in 64 bits
def _wide(rows):
    return rows.view(torch.float8_e4m3fn).double() if rows.dtype == torch.uint8 else rows.double()


def _attend(q, keys):
    """One query's heads [64][512] over keys [n][512], all visible, in 64 bits."""
    if keys.shape[0] == 0:
        return torch.zeros(H, D, dtype=torch.float64, device=q.device), \
            torch.full((H,), -math.inf, dtype=torch.float64, device=q.device)
    logit = torch.einsum("hd,nd->hn", q, keys) / math.sqrt(D)
    return torch.einsum("hn,nd->hd", torch.softmax(logit, -1), keys), torch.logsumexp(logit, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        q_out = torch.zeros(case["T"], H, D, dtype=torch.float64, device="cuda")
        rows = torch.zeros(case["T"] + 5, D, dtype=torch.float64, device="cuda")
        live = (s["pos"] >= 0).nonzero()[:, 0]
        turn = torch.view_as_complex(s["table"][s["pos"][live]].double().contiguous())

        def one(x, weight):
            x = x.double()
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
            x = x if weight is None else x * weight.double()
            z = torch.view_as_complex(x[..., D - ROT:].unflatten(-1, (ROT // 2, 2)).contiguous())
            z = z * (turn[:, None] if x.dim() == 3 else turn)
            x[..., D - ROT:] = torch.view_as_real(z).flatten(-2)
            return x

        q_out[live] = one(s["q"][live], s["q_weight"])
        rows[s["slot"][live]] = one(s["k"][live], s["k_weight"])
        return {"q": q_out, "rows": rows.clamp(-448.0, 448.0) if case["fp8"] else rows}
    B, Q = case["B"], case["Q"]
    out = torch.zeros(B, Q, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    pos, base = s["pos"].tolist(), s["base"].tolist()
    W = case["W"] if case["op"] == "window" else WIN
    for b in range(B):
        rows = _wide(s["rows"][b])
        if case["op"] == "window":
            first = _wide(s["sinks"][b]) if case["sinks"] else rows[:0]
        else:
            magnitude = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
            byte = s["kv"][b, :, :256].long()
            code = torch.empty(byte.shape[0], D, dtype=torch.int64, device="cuda")
            code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
            sign = 1.0 - 2.0 * (code // 8)
            scale = _wide(s["kv"][b, :, 256:].contiguous()).repeat_interleave(16, -1)
            first = magnitude[code % 8] * sign * scale
            n = int(s["n_entries"][b])
        for i in range(Q):
            t = pos[b][i]
            if t < 0:
                continue
            lo = max(0, t - W + 1)
            far = first[:min(case["sinks"], lo)] if case["op"] == "window" else first[:min(n, (t + 1) // case["m"])]
            out[b, i], lse[b, i] = _attend(s["q"][b, i].double(),
                                           torch.cat([far, rows[lo - base[b]:t + 1 - base[b]]]))
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm_rope":
        T = case["T"]
        live = T - case["pad"]
        row = D * (1 if case["fp8"] else 2)
        table = live * ROT * 4
        return {"bytes": live * (2 * H * D * 2 + D * 2 + row) + table + 16 * T, "flops": live * (H + 1) * D * 6}
    B, Q = case["B"], case["Q"]
    row = D * (1 if case["fp8"] else 2)
    if case["op"] == "window":
        pos, base = _window_positions(case)
        W = case["W"]
        lo = np.maximum(0, pos - W + 1)
        keys = np.where(pos >= 0, np.minimum(pos + 1, W) + np.minimum(case["sinks"], lo), 0)
        kv = sum(int(pos[b].max() - base[b] + 1 + min(case["sinks"], lo[b].max())) * row for b in range(B))
    else:
        pos, ns, base = _dense_positions(case)
        entries = np.minimum((pos + 1) // case["m"], ns[:, None])
        keys = np.minimum(pos + 1, WIN) + entries
        kv = int(entries.max(1).sum()) * 288 + sum(int(pos[b].max() - base[b] + 1) * row for b in range(B))
    live = int((pos >= 0).sum())
    return {"bytes": live * H * D * 2 + B * Q * (H * D * 2 + H * 4 + 8) + kv,
            "flops": float(keys.sum()) * H * D * 4}
