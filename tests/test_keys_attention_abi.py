"""Argument checks and workspace arithmetic of the norm and rotation of queries
and window keys, the window attention and the dense attention: everything here
returns before any CUDA call."""
import ctypes

import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2

FAKE = 1 << 20                      # never dereferenced: the calls fail on arguments
WS = 1 << 36
PART = (2 * 64 + 64 * 512) * 4


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_csa2_gb300 import build
    return csa2.load(build.build())


def qk_args(**kw):
    T = kw.get("T", 4)
    a = dict(T=T, pos=FAKE, rope_cs=FAKE, rope_P=64, eps=1e-6, rows_fp8=0, q=1 << 32, q_stride=32768, q_weight=None,
             q_out=2 << 32, k=3 << 32, k_stride=512, k_weight=None, rows=4 << 32, n_rows=8, k_slot=None)
    a.update(kw)
    return csa2.QkArgs(**a)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(rope_P=-1), 1), (dict(n_rows=-1), 1), (dict(T=(1 << 26) + 1), 2),
    (dict(eps=float("nan")), 1), (dict(eps=-1e-6), 1), (dict(rows_fp8=2), 1),
    (dict(pos=None), 1), (dict(pos=FAKE + 4), 1), (dict(rope_cs=None), 1), (dict(rope_cs=FAKE + 8), 1),
    (dict(q_out=None), 1), (dict(q=(1 << 32) + 8), 1), (dict(q_weight=FAKE + 4), 1),
    (dict(q_stride=32760), 1), (dict(q_stride=32772), 1), (dict(k_stride=504), 1), (dict(k_stride=1 << 40), 1),
    (dict(rows=None), 1), (dict(rows=(4 << 32) + 8), 1), (dict(k_slot=FAKE + 4), 1),
    (dict(q_out=(1 << 32) + 16), 1),                                   # overlaps q
    (dict(q_out=1 << 32, q_stride=32776), 1),                          # in place needs dense tokens
    (dict(rows=3 << 32), 1),                                           # overlaps k
    (dict(rows=(2 << 32) + 65536), 1), (dict(k=(2 << 32) + 65536), 1),  # overlap q_out
    (dict(rows=(1 << 32) + 65536), 1),                                 # overlaps q
])
def test_norm_rope_refuses(lib, change, want):
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args(**change)), WS, 256, None) == want


@pytest.mark.parametrize("out", ["q_out", "rows"])
@pytest.mark.parametrize("name,last", [("pos", 4 * 8), ("rope_cs", 64 * 256), ("q_weight", 2048), ("k_weight", 2048),
                                       ("k_slot", 4 * 8), ("ws", 256)])
def test_norm_rope_refuses_outputs_over_its_small_inputs(lib, out, name, last):
    at = (8 << 32) + 4096
    ws = at if name == "ws" else WS
    kw = {} if name == "ws" else {name: at}
    size = 4 * 65536 if out == "q_out" else 8 * 1024
    for addr in (at, at + last - 16, at - size + 16):
        assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args(**kw, **{out: addr})), ws, 256, None) == 1, addr - at


def test_norm_rope_nothing_to_do_and_workspace(lib):
    assert lib.csa2_qk_norm_rope(None, WS, 256, None) == 1
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args()), None, 0, None) == 3
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args()), WS + 128, 256, None) == 1
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args()), WS, 255, None) == 3
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args(T=0, pos=None)), WS, 256, None) == 0
    assert lib.csa2_qk_norm_rope(ctypes.byref(qk_args(q=None, k=None)), WS, 256, None) == 0


def window_args(**kw):
    a = dict(B=2, Q=3, S=200, W=128, n_sink=4, scale=0.04, q_pos=FAKE, q=1 << 32, rows=2 << 32, swa_base_pos=FAKE + 4096,
             sinks=3 << 32, out=4 << 32, lse=5 << 32, rows_fp8=0)
    a.update(kw)
    return csa2.WindowArgs(**a)


def dense_args(**kw):
    a = dict(B=2, Q=3, S=200, scale=0.04, max_n=64, q_pos=FAKE, q=1 << 32, swa=2 << 32, swa_base_pos=FAKE + 4096,
             out=4 << 32, lse=5 << 32, swa_fp8=0)
    a.update(kw)
    return csa2.DenseArgs(**a)


CACHE = csa2.CacheStruct(6 << 32, 7 << 32, 8 << 32, 64, 9 << 32, 1)


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), 1), (dict(Q=-1), 1), (dict(S=-1), 1), (dict(scale=float("inf")), 1), (dict(rows_fp8=2), 1),
    (dict(B=1 << 13, Q=(1 << 11) + 1), 2), (dict(B=1 << 16, Q=1, S=1 << 15), 2),
    (dict(q=None), 1), (dict(q=(1 << 32) + 8), 1), (dict(q_pos=None), 1), (dict(q_pos=FAKE + 4), 1),
    (dict(swa_base_pos=None), 1), (dict(swa_base_pos=FAKE + 2), 1), (dict(rows=None), 1), (dict(rows=(2 << 32) + 8), 1),
    (dict(out=None), 1), (dict(out=(4 << 32) + 2), 1), (dict(lse=(5 << 32) + 2), 1),
    (dict(out=1 << 32), 1), (dict(out=(2 << 32) + 1024), 1), (dict(lse=(4 << 32) + 4), 1), (dict(lse=1 << 32), 1),
    (dict(out=FAKE), 1), (dict(lse=FAKE + 4096), 1), (dict(out=WS), 1),
])
def test_attention_calls_refuse(lib, change, want):
    need = 1 << 30
    assert lib.csa2_window_attn(ctypes.byref(window_args(**change)), WS, need, None) == want
    renamed = {{"rows": "swa", "rows_fp8": "swa_fp8"}.get(k, k): v for k, v in change.items()}
    assert lib.csa2_dense_attn(ctypes.byref(CACHE), ctypes.byref(dense_args(**renamed)), WS, need, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(W=0), 1), (dict(W=-5), 1), (dict(n_sink=-1), 1), (dict(sinks=None), 1), (dict(sinks=(3 << 32) + 8), 1),
    (dict(n_sink=1 << 30), 2), (dict(out=3 << 32), 1)])
def test_window_refuses(lib, change, want):
    assert lib.csa2_window_attn(ctypes.byref(window_args(**change)), WS, 1 << 30, None) == want


def test_dense_refuses(lib):
    def call(cache=CACHE, ws=WS, n=1 << 30, **kw):
        return lib.csa2_dense_attn(ctypes.byref(cache) if cache else None, ctypes.byref(dense_args(**kw)), ws, n, None)
    assert call(cache=None) == 1
    assert lib.csa2_dense_attn(ctypes.byref(CACHE), None, WS, 1 << 30, None) == 1
    assert call(max_n=-1) == 1
    assert call(cache=csa2.CacheStruct(6 << 32, 7 << 32, 8 << 32, 60, 9 << 32, 1)) == 1        # cap % 8
    assert call(cache=csa2.CacheStruct(6 << 32, 7 << 32, 8 << 32, 64, 9 << 32, 3)) == 2        # m
    assert call(out=6 << 32) == 1 and call(lse=9 << 32) == 1                                   # the cache itself
    assert call(ws=None) == 3 and call(n=csa2.dense_attn_workspace_size(2, 3, 64) - 1) == 3
    assert lib.csa2_window_attn(None, WS, 1 << 30, None) == 1
    need = csa2.window_attn_workspace_size(2, 3, 128, 4)
    assert lib.csa2_window_attn(ctypes.byref(window_args()), WS, need - 1, None) == 3


def test_nothing_to_do(lib):
    none = dict(B=0, q=None, q_pos=None, out=None)
    assert lib.csa2_window_attn(ctypes.byref(window_args(rows=None, sinks=None, **none)), WS, 256, None) == 0
    assert lib.csa2_dense_attn(ctypes.byref(CACHE), ctypes.byref(dense_args(swa=None, **none)), WS, 256, None) == 0


def test_workspace_sizes(lib):
    assert csa2.dense_attn_workspace_size(-1, 1, 8) == 0 and csa2.window_attn_workspace_size(1, 1, 0, 0) == 0
    # many queries fill the GPU by themselves: no partial states
    assert csa2.dense_attn_workspace_size(1, 4096, 8192) == 256
    assert csa2.window_attn_workspace_size(64, 64, 1024, 0) == 256
    # one key run cannot be divided
    assert csa2.window_attn_workspace_size(1, 1, 128, 0) == 256
    # a long cache and one query: a state per SM at most
    one = csa2.dense_attn_workspace_size(1, 1, 1 << 20) - 256
    assert one % PART == 0 and 64 * PART <= one <= 152 * PART
    # however long the window or the cache, at most four states an SM
    for b in (1, 3, 16, 100, 300, 600):
        for n in (csa2.dense_attn_workspace_size(b, 1, 1 << 31), csa2.window_attn_workspace_size(b, 1, (1 << 31) - 1, 0)):
            assert n - 256 <= 4 * 152 * PART


@pytest.mark.parametrize("B,Q", [(1, 1), (3, 7), (152, 1), (600, 1), (4096, 4096)])
def test_the_largest_max_n(lib, B, Q):
    """However many entries a call names, its workspace is that of the most a cache can hold."""
    most = csa2.dense_attn_workspace_size(B, Q, (1 << 31) - 1)
    assert 256 <= most <= 256 + 4 * 152 * PART
    for n in (1 << 31, 1 << 40, 1 << 62, (1 << 63) - 1):
        assert csa2.dense_attn_workspace_size(B, Q, n) == most


def test_binding_structs_match_the_c_layout(tmp_path):
    from tests.test_library_abi import _c_layout
    for cls, struct in ((csa2.QkArgs, "csa2_qk_args"), (csa2.WindowArgs, "csa2_window_args"),
                        (csa2.DenseArgs, "csa2_dense_args")):
        names = [f[0] for f in cls._fields_]
        c = _c_layout(tmp_path, struct, names)
        assert c == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in names], struct


class _FakeWs:
    """Stands for a workspace: the binding's own checks come before the call."""
    buf, ptr, nbytes = torch.zeros(1, dtype=torch.uint8), WS, 256


def test_binding_refuses_shapes_types_and_strides():
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    pos, cs = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError, match="pos"):
        csa2.qk_norm_rope(pos.int(), cs, _FakeWs, q=q, q_out=q)
    with pytest.raises(ValueError, match="q:"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q[:, :32], q_out=q)
    with pytest.raises(ValueError, match="strides"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q.transpose(0, 1).contiguous().transpose(0, 1), q_out=q)
    with pytest.raises(ValueError, match="q_out"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q, q_out=q.float())
    with pytest.raises(ValueError, match="q_weight"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q, q_out=q, q_weight=torch.ones(64))
    rows, base = torch.zeros(1, 130, 512, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    p1, q1 = torch.zeros(1, 2, dtype=torch.int64), q[None]
    with pytest.raises(ValueError, match="sinks"):       # sinks of another type than the rows
        csa2.window_attn(q1, rows, base, p1, 0.1, torch.empty_like(q1), _FakeWs, W=8,
                         sinks=torch.zeros(1, 4, 512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="swa_base_pos"):
        csa2.window_attn(q1, rows, base.repeat(2), p1, 0.1, torch.empty_like(q1), _FakeWs, W=8)
    with pytest.raises(ValueError, match="lse"):
        csa2.window_attn(q1, rows, base, p1, 0.1, torch.empty_like(q1), _FakeWs, W=8, lse=torch.zeros(1, 2, 32))
    with pytest.raises(ValueError, match="sequences"):
        csa2.dense_attn(csa2.Cache(2, 8, 1, device="cpu"), q1, rows, base, p1, 0.1, torch.empty_like(q1), _FakeWs, max_n=8)


def test_binding_refuses_types_of_the_right_size():
    """A type of the same width would be read as another number."""
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    pos, cs = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError, match="q:"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q.half(), q_out=q)
    with pytest.raises(ValueError, match="q_out"):
        csa2.qk_norm_rope(pos, cs, _FakeWs, q=q, q_out=q.half())
    with pytest.raises(ValueError, match="pos"):
        csa2.qk_norm_rope(pos.double(), cs, _FakeWs, q=q, q_out=q)
    with pytest.raises(ValueError, match="rope_cs"):
        csa2.qk_norm_rope(pos, cs.int(), _FakeWs, q=q, q_out=q)
    k, rows = torch.zeros(2, 512, dtype=torch.bfloat16), torch.zeros(2, 512)
    for wrong in (torch.float8_e5m2, torch.bool, torch.float16):
        with pytest.raises(ValueError, match="rows"):
            csa2.qk_norm_rope(pos, cs, _FakeWs, k=k, rows=rows.to(wrong))
    base, p1, q1 = torch.zeros(1, dtype=torch.int64), torch.zeros(1, 2, dtype=torch.int64), q[None]
    r1 = torch.zeros(1, 130, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="lse"):
        csa2.window_attn(q1, r1, base, p1, 0.1, torch.empty_like(q1), _FakeWs, W=8,
                         lse=torch.zeros(1, 2, 64, dtype=torch.int32))
    with pytest.raises(ValueError, match="out"):
        csa2.dense_attn(csa2.Cache(1, 8, 1, device="cpu"), q1, r1, base, p1, 0.1, q1.half(), _FakeWs, max_n=8)
