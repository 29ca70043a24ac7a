"""Argument checks, workspace arithmetic and the binding's refusals of the 8-bit cache,
the gathered weights and the eviction: everything here returns before any CUDA call."""
import ctypes

import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2

FAKE = 1 << 20                      # never dereferenced: the calls fail on arguments
WS = 1 << 36
BIG = 1 << 30
G = 1 << 32


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_csa2_gb300 import build
    return csa2.load(build.build())


def cache8(**kw):
    a = dict(codes=G, scales=2 * G, cap=64, n_entries=3 * G, m=1)
    a.update(kw)
    return csa2.Cache8Struct(**a)


def cache4(**kw):
    a = dict(main_kv=G, idx_codes=2 * G, idx_scales=20 * G, cap=64, n_entries=3 * G, m=1)
    a.update(kw)
    return csa2.CacheStruct(**a)


def write_args(**kw):
    a = dict(B=2, T=3, x=4 * G, x_stride=512, entry_start=FAKE, n_new=FAKE + 4096)
    a.update(kw)
    return csa2.Cache8WriteArgs(**a)


def attn_args(**kw):
    a = dict(B=2, Q=3, S=200, W=128, scale=0.04, max_n=64, q_pos=FAKE, q=4 * G, swa=5 * G, swa_base_pos=FAKE + 4096,
             out=6 * G, lse=7 * G, swa_fp8=0)
    a.update(kw)
    return csa2.Cache8AttnArgs(**a)


def weights_args(**kw):
    a = dict(B=2, Q=3, scale=0.04, decay=0.9, max_n=64, q_pos=FAKE, q=4 * G, lse=5 * G, prev=6 * G, weights=7 * G)
    a.update(kw)
    return csa2.WeightsArgs(**a)


def evict_args(**kw):
    a = dict(B=2, unit=8, budget=32, n_first=4, n_recent=8, weights=5 * G, to_weights=6 * G, kept=7 * G, n_out=8 * G)
    a.update(kw)
    return csa2.EvictArgs(**a)


BAD_CACHE8 = [(dict(codes=None), 1), (dict(scales=None), 1), (dict(n_entries=None), 1), (dict(codes=G + 8), 1),
              (dict(scales=2 * G + 2), 1), (dict(n_entries=3 * G + 2), 1), (dict(cap=-8), 1), (dict(cap=60), 1),
              (dict(m=3), 2), (dict(cap=1 << 30), 2), (dict(cap=1 << 40), 2)]


@pytest.mark.parametrize("change,want", BAD_CACHE8)
def test_bad_caches_are_refused_by_every_call(lib, change, want):
    c = ctypes.byref(cache8(**change))
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args()), WS, BIG, None) == want
    assert lib.csa2_cache8_attn(c, ctypes.byref(attn_args()), WS, BIG, None) == want
    assert lib.csa2_cache8_attn_weights(c, ctypes.byref(weights_args()), WS, BIG, None) == want
    to = cache8(codes=9 * G, scales=10 * G)
    assert lib.csa2_cache8_evict(c, ctypes.byref(to), ctypes.byref(evict_args()), WS, BIG, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(B=1 << 14, T=(1 << 12) + 1), 2), (dict(x=None), 1), (dict(x=4 * G + 8), 1),
    (dict(entry_start=None), 1), (dict(entry_start=FAKE + 4), 1), (dict(n_new=FAKE + 2), 1), (dict(x_stride=504), 1),
    (dict(x_stride=516), 1), (dict(x_stride=1 << 40), 1), (dict(x=G + 1024), 1), (dict(entry_start=2 * G), 1),
    (dict(n_new=G), 1), (dict(x=G - 1024), 1)])
def test_write_refuses(lib, change, want):
    if "B" in change and change["B"] > 2:
        c = cache8(cap=8)
    else:
        c = cache8()
    assert lib.csa2_cache8_write(ctypes.byref(c), ctypes.byref(write_args(**change)), WS, 256, None) == want


def test_write_workspace_and_nothing_to_do(lib):
    c = ctypes.byref(cache8())
    assert lib.csa2_cache8_write(c, None, WS, 256, None) == 1
    assert lib.csa2_cache8_write(None, ctypes.byref(write_args()), WS, 256, None) == 1
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args()), None, 256, None) == 3
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args()), WS, 255, None) == 3
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args()), WS + 64, 256, None) == 1
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args()), G, 256, None) == 1            # the codes
    assert lib.csa2_cache8_write(c, ctypes.byref(write_args(T=0, x=None)), WS, 256, None) == 0
    over = cache8(scales=G + 4096)                                                            # scales among the codes
    assert lib.csa2_cache8_write(ctypes.byref(over), ctypes.byref(write_args()), WS, 256, None) == 1
    over = cache8(n_entries=G + 4096)
    assert lib.csa2_cache8_write(ctypes.byref(over), ctypes.byref(write_args()), WS, 256, None) == 1


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), 1), (dict(Q=-1), 1), (dict(S=-1), 1), (dict(W=-1), 1), (dict(scale=float("nan")), 1), (dict(swa_fp8=2), 1),
    (dict(max_n=-1), 1), (dict(Q=(1 << 23) + 1), 2), (dict(S=1 << 30), 2), (dict(q=None), 1), (dict(q_pos=None), 1), (dict(swa=None), 1),
    (dict(swa_base_pos=None), 1), (dict(out=None), 1), (dict(out=6 * G + 8), 1), (dict(lse=7 * G + 2), 1),
    (dict(out=4 * G), 1), (dict(out=G), 1), (dict(out=2 * G), 1), (dict(lse=2 * G), 1), (dict(lse=3 * G), 1),
    (dict(out=WS), 1), (dict(lse=6 * G + 64), 1)])
def test_attention_refuses(lib, change, want):
    assert lib.csa2_cache8_attn(ctypes.byref(cache8()), ctypes.byref(attn_args(**change)), WS, BIG, None) == want


def test_attention_workspace(lib):
    c = ctypes.byref(cache8())
    need = csa2.cache8_attn_workspace_size(2, 3, 5000, 128)
    assert need > 256
    assert lib.csa2_cache8_attn(c, ctypes.byref(attn_args(max_n=5000)), WS, need - 1, None) == 3
    assert lib.csa2_cache8_attn(c, ctypes.byref(attn_args(B=0, q=None, out=None)), WS, 256, None) == 0
    assert csa2.cache8_attn_workspace_size(1, 1, 8, -1) == 0 and csa2.cache8_attn_workspace_size(1, 1, -8, 0) == 0
    assert csa2.cache8_attn_workspace_size(6, 1, 5000, 128) == csa2.dense_attn_workspace_size(6, 1, 5000)
    assert csa2.cache8_attn_workspace_size(2, 3, (1 << 63) - 1, 0) <= 256 + 4 * 152 * (2 * 64 + 64 * 512) * 4


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), 1), (dict(Q=-1), 1), (dict(scale=float("inf")), 1), (dict(decay=float("nan")), 1), (dict(max_n=-1), 1),
    (dict(Q=(1 << 23) + 1), 2), (dict(q=None), 1), (dict(q=4 * G + 8), 1), (dict(q_pos=None), 1), (dict(q_pos=FAKE + 4), 1), (dict(lse=None), 1),
    (dict(lse=5 * G + 2), 1), (dict(prev=6 * G + 2), 1), (dict(weights=None), 1), (dict(weights=7 * G + 1), 1),
    (dict(weights=4 * G), 1), (dict(weights=5 * G), 1), (dict(weights=FAKE), 1), (dict(weights=G), 1), (dict(weights=3 * G), 1),
    (dict(weights=WS + 128), 1), (dict(prev=7 * G + 4), 1)])
def test_weights_refuse(lib, change, want):
    a = ctypes.byref(weights_args(**change))
    assert lib.csa2_attn_weights(ctypes.byref(cache4()), a, WS, BIG, None) == want
    assert lib.csa2_cache8_attn_weights(ctypes.byref(cache8()), a, WS, BIG, None) == want


def test_weights_workspace(lib):
    need = csa2.attn_weights_workspace_size(1, 2000, 64)
    assert need > 256 and (need - 256) % (64 * 4) == 0                             # partial sums of the queries' splits
    for call, c in ((lib.csa2_attn_weights, cache4()), (lib.csa2_cache8_attn_weights, cache8())):
        assert call(ctypes.byref(c), ctypes.byref(weights_args(B=1, Q=2000)), WS, need - 1, None) == 3
        assert call(ctypes.byref(c), ctypes.byref(weights_args()), None, need, None) == 3
        assert call(ctypes.byref(c), None, WS, need, None) == 1
        assert call(ctypes.byref(c), ctypes.byref(weights_args(B=0, weights=None)), WS, 4096, None) == 0
    assert lib.csa2_attn_weights(ctypes.byref(cache4(m=3)), ctypes.byref(weights_args()), WS, need, None) == 2
    assert lib.csa2_attn_weights(ctypes.byref(cache4(idx_codes=None, n_entries=3 * G + 2)), ctypes.byref(weights_args()), WS, need, None) == 1
    assert csa2.attn_weights_workspace_size(-1, 1, 8) == 0 and csa2.attn_weights_workspace_size(1, 1, -8) == 0
    most = csa2.attn_weights_workspace_size(1, 2000, (1 << 31) - 1)
    assert all(csa2.attn_weights_workspace_size(1, 2000, n) == most for n in (1 << 31, (1 << 63) - 1))


EVICT = [(dict(B=-1), 1), (dict(unit=0), 1), (dict(unit=4), 1), (dict(budget=0), 1), (dict(budget=-8), 1), (dict(budget=36), 1), (dict(budget=72), 1),
         (dict(n_first=-1), 1), (dict(n_recent=-1), 1), (dict(n_first=33), 1), (dict(n_recent=33), 1), (dict(n_first=9, n_recent=9), 1),
         (dict(n_recent=25, n_first=0), 1), (dict(n_first=1 << 62), 1),
         (dict(weights=None), 1), (dict(weights=5 * G + 8), 1), (dict(to_weights=6 * G + 2), 1), (dict(kept=None), 1), (dict(kept=7 * G + 2), 1),
         (dict(n_out=None), 1), (dict(n_out=8 * G + 2), 1), (dict(to_weights=5 * G), 1), (dict(kept=5 * G), 1), (dict(kept=G), 1),
         (dict(kept=9 * G), 1), (dict(n_out=7 * G), 1), (dict(n_out=9 * G), 1), (dict(to_weights=9 * G), 1), (dict(kept=WS), 1), (dict(kept=3 * G), 1),
         (dict(weights=9 * G), 1), (dict(budget=1 << 32), 2)]


@pytest.mark.parametrize("change,want", EVICT)
def test_evict_refuses(lib, change, want):
    a = ctypes.byref(evict_args(**change))
    to8, to4 = cache8(codes=9 * G, scales=10 * G), cache4(main_kv=9 * G, idx_codes=10 * G, idx_scales=11 * G)
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), ctypes.byref(to8), a, WS, BIG, None) == want
    assert lib.csa2_evict(ctypes.byref(cache4()), ctypes.byref(to4), a, WS, BIG, None) == want


def test_evict_refuses_caches_that_overlap(lib):
    a = ctypes.byref(evict_args())
    for to in (cache8(scales=10 * G), cache8(codes=9 * G), cache8(codes=G + 4096, scales=10 * G), cache8(codes=9 * G, scales=9 * G + 512),
               cache8(codes=9 * G, scales=2 * G + 4), cache8(cap=128), cache8(codes=9 * G, scales=10 * G, cap=24),
               cache8(codes=9 * G + 8, scales=10 * G), cache8(codes=None, scales=10 * G), cache8(codes=9 * G, scales=10 * G, cap=36)):
        assert lib.csa2_cache8_evict(ctypes.byref(cache8()), ctypes.byref(to), a, WS, BIG, None) == 1
    for to in (cache4(main_kv=9 * G), cache4(main_kv=9 * G, idx_codes=10 * G), cache4(cap=128),
               cache4(main_kv=9 * G, idx_codes=10 * G, idx_scales=10 * G + 64)):
        assert lib.csa2_evict(ctypes.byref(cache4()), ctypes.byref(to), a, WS, BIG, None) == 1


def test_evict_workspace_and_units(lib):
    to = cache8(codes=9 * G, scales=10 * G)
    need = csa2.evict_workspace_size(csa2.Cache8(2, 64, 1, device="cpu"), 32, 8)
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), ctypes.byref(to), ctypes.byref(evict_args()), WS, need - 1, None) == 3
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), ctypes.byref(to), ctypes.byref(evict_args()), None, need, None) == 3
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), ctypes.byref(to), ctypes.byref(evict_args(unit=1)), WS, need, None) == 2
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), None, None, WS, need, None) == 1
    assert lib.csa2_evict(ctypes.byref(cache4()), None, None, WS, need, None) == 1
    assert lib.csa2_cache8_evict(ctypes.byref(cache8()), None, ctypes.byref(evict_args(B=0, kept=None)), WS, 2048, None) == 0
    assert lib.csa2_evict_workspace_size(1, 0, 1) == 0 and lib.csa2_evict_workspace_size(1, 12, 8) == 0
    assert lib.csa2_evict_workspace_size(1, 1 << 31, 1) == 0 and lib.csa2_evict_workspace_size(1, 8, 2) == 0


def test_binding_structs_match_the_c_layout(tmp_path):
    from tests.test_library_abi import _c_layout
    for cls, struct in ((csa2.Cache8Struct, "csa2_cache8"), (csa2.Cache8WriteArgs, "csa2_cache8_write_args"),
                        (csa2.Cache8AttnArgs, "csa2_cache8_attn_args"), (csa2.WeightsArgs, "csa2_weights_args"),
                        (csa2.EvictArgs, "csa2_evict_args")):
        names = [f[0] for f in cls._fields_]
        assert _c_layout(tmp_path, struct, names) == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in names], struct


# ------------------------------------------------------------------ the binding's own refusals
class _FakeWs:
    """Stands for a workspace: the binding's own checks come before the call."""
    buf, ptr, nbytes = torch.zeros(1, dtype=torch.uint8), WS, 256


BF16, I64, I32 = torch.bfloat16, torch.int64, torch.int32


def calls(name, **kw):
    c = csa2.Cache8(1, 16, 1, device="cpu")
    q = dict(q=torch.zeros(1, 2, 64, 512, dtype=BF16), q_pos=torch.zeros(1, 2, dtype=I64), scale=0.1, ws=_FakeWs, max_n=16)
    a = {"write": dict(cache=c, x=torch.zeros(1, 3, 512, dtype=BF16), entry_start=torch.zeros(1, dtype=I64), ws=_FakeWs,
                       n_new=torch.zeros(1, dtype=I32)),
         "attn": dict(cache=c, out=torch.zeros(1, 2, 64, 512, dtype=BF16), W=8, swa=torch.zeros(1, 9, 512, dtype=BF16),
                      swa_base_pos=torch.zeros(1, dtype=I64), lse=torch.zeros(1, 2, 64), **q),
         "weights": dict(cache=c, lse=torch.zeros(1, 2, 64), weights=torch.zeros(1, 16), prev=torch.zeros(1, 16), **q),
         "evict": dict(cache=c, weights=torch.zeros(1, 16), kept=torch.zeros(1, 1, dtype=I32), n_out=torch.zeros(1, dtype=I32),
                       ws=_FakeWs, budget=8, unit=8, to=csa2.Cache8(1, 8, 1, device="cpu"), to_weights=torch.zeros(1, 8))}[name]
    a.update(kw)
    return {"write": csa2.cache8_write, "attn": csa2.cache8_attn, "weights": csa2.attn_weights, "evict": csa2.evict}[name](**a)


@pytest.mark.parametrize("call,names", [("write", "x entry_start"), ("attn", "q q_pos out swa swa_base_pos"), ("weights", "q q_pos lse weights"),
                                        ("evict", "weights kept n_out")])
def test_binding_refuses_what_is_missing(call, names):
    for name in names.split():
        with pytest.raises(ValueError, match=f"{name}: missing"):
            calls(call, **{name: None})


@pytest.mark.parametrize("call,name,bad", [
    ("write", "x", torch.zeros(1, 3, 512)), ("write", "x", torch.zeros(1, 3, 256, dtype=BF16)), ("write", "x", torch.zeros(2, 3, 512, dtype=BF16)),
    ("write", "x", torch.zeros(3, 512, dtype=BF16)), ("write", "x", torch.zeros(1, 3, 1024, dtype=BF16)[..., ::2]),
    ("write", "entry_start", torch.zeros(1, dtype=I32)), ("write", "n_new", torch.zeros(1, dtype=I64)), ("write", "n_new", torch.zeros(2, dtype=I32)),
    ("attn", "q", torch.zeros(1, 2, 64, 512, dtype=torch.float16)), ("attn", "q_pos", torch.zeros(2, 2, dtype=I64)),
    ("attn", "out", torch.zeros(1, 2, 64, 512)), ("attn", "lse", torch.zeros(1, 2, 32)), ("attn", "swa", torch.zeros(1, 9, 512)),
    ("attn", "swa_base_pos", torch.zeros(1, dtype=I32)), ("weights", "lse", torch.zeros(1, 2, 64, dtype=torch.float64)),
    ("weights", "prev", torch.zeros(1, 8)), ("weights", "weights", torch.zeros(2, 16)), ("weights", "q", torch.zeros(1, 2, 64, 512)),
    ("evict", "weights", torch.zeros(1, 8)), ("evict", "kept", torch.zeros(1, 8, dtype=I32)), ("evict", "kept", torch.zeros(1, 1, dtype=I64)),
    ("evict", "n_out", torch.zeros(1, dtype=I64)), ("evict", "to_weights", torch.zeros(1, 16)), ("evict", "budget", 12), ("evict", "unit", 2)])
def test_binding_refuses_other_shapes_and_types(call, name, bad):
    with pytest.raises(ValueError, match="budget" if name == "unit" else f"{name}:|{name.split('_')[0]}"):
        calls(call, **{name: bad})


def test_binding_refuses_sequences_strided_apart():
    x = torch.zeros(2, 4, 512, dtype=BF16)[:, :3]                                  # 3 of 4 tokens a sequence: two strides
    with pytest.raises(ValueError, match="x:"):
        calls("write", cache=csa2.Cache8(2, 16, 1, device="cpu"), x=x, entry_start=torch.zeros(2, dtype=I64), n_new=None)


def test_binding_refuses_rows_without_a_window_and_other_caches():
    with pytest.raises(ValueError, match="swa"):
        calls("attn", W=0)
    with pytest.raises(ValueError, match="to:"):
        calls("evict", to=csa2.Cache(1, 8, 1, device="cpu"))
    with pytest.raises(ValueError, match="to:"):
        calls("evict", to=csa2.Cache8(2, 8, 1, device="cpu"))
    for call in ("write", "attn", "weights", "evict"):
        for name, bad in (("codes", torch.zeros(1, 8, 512, dtype=torch.int8)), ("scales", torch.zeros(1, 3)), ("n_entries", torch.zeros(1, dtype=I64)),
                          ("codes", None), ("cap", 12)):
            c = csa2.Cache8(1, 16, 1, device="cpu")
            setattr(c, name, bad)
            with pytest.raises(ValueError, match="cache"):
                calls(call, cache=c)


def test_a_workspace_on_the_host_is_refused():
    for call in ("write", "attn", "weights", "evict"):
        with pytest.raises(ValueError, match="ws: the workspace is not on a CUDA device"):
            calls(call)


def test_the_split_of_pairs_follows_the_number_of_sequences(lib):
    """Lengths are not known on the host: the longest's work is divided as for lengths spread evenly below it (several
    sequences), or as it is (one)."""
    part = 64 * (2 + 512) * 4                                # a partial state
    for (B, Q, n, W), split in {(4, 37, 10000, 128): 2, (3, 37, 10007, 128): 2, (7, 16, 5300, 128): 2, (16, 8, 2000, 128): 1,
                                (2, 128, 3000, 128): 1, (3, 8, 30000, 128): 6, (1, 148, 10000, 128): 1}.items():
        want = 256 + (-(-B * Q * split * part // 256) * 256 if split > 1 else 0)
        assert csa2.cache8_attn_workspace_size(B, Q, n, W) == want, (B, Q, n, W)


def test_which_kernel_the_attention_takes(lib):
    """The sizes of the GPU tests of either kernel (tests/test_gpu_cache8.py, tests/test_gpu_cache8_edges.py)."""
    def plan(B, Q, max_n, W):
        split = ctypes.c_int(0)
        return lib.csa2_test_cache8_attn_plan(B, Q, max_n, W, ctypes.byref(split)), split.value

    for call in [(1, 152, 1300, 0), (2, 76, 1441, 130), (4, 37, 1600, 99), (1, 151, 1300, 200), (1, 152, 1300, 64), (1, 152, 1300, 16),
                 (1, 152, 1300, 40), (1, 152, 1300, 128), (1, 300, 1300, 200), (1, 152, 500, 20), (2, 76, 400, 0)]:
        assert plan(*call) == (1, 1), call                   # pairs, undivided
    for call in [(1, 60, 2999, 128), (2, 31, 2999, 64), (1, 60, 3000, 0), (1, 60, 1300, 20), (1, 60, 2000, 20), (1, 60, 1 << 40, 20)]:
        assert plan(*call)[0] == 1 and plan(*call)[1] > 1, call
    for call in [(1, 1, 200, 0), (1, 1, 3000, 0), (16, 1, 131072, 128), (1, 2, 200, 0), (1, 4, 600, 0), (3, 2, 1000, 130), (1, 60, 1, 20)]:
        assert plan(*call)[0] == 0, call
    assert plan(1, 0, 64, 0)[0] == 0 and plan(-1, 1, 64, 0)[0] == plan(1, 1, -1, 0)[0] == plan(1, 1, 1, -1)[0] == -1
    assert plan(1 << 13, 1 << 12, 64, 0)[0] == -1 and lib.csa2_test_cache8_attn_plan(1, 1, 64, 0, None) == -1
