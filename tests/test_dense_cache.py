"""What the dense attention asks of a cache: entries and their numbers, no index keys."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2

WS = 1 << 36                        # never dereferenced: the calls return before any CUDA call


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_csa2_gb300 import build
    return csa2.load(build.build())


def dense(lib, cache, **kw):
    a = dict(B=0, Q=3, S=200, scale=0.04, max_n=64, q_pos=None, q=None, swa=None, swa_base_pos=None, out=None, lse=None,
             swa_fp8=0)
    a.update(kw)
    return lib.csa2_dense_attn(ctypes.byref(cache), ctypes.byref(csa2.DenseArgs(**a)), WS, 1 << 30, None)


def test_the_index_keys_may_be_left_out(lib):
    for codes, scales in ((None, None), (7 << 32, None), ((7 << 32) + 1, (8 << 32) + 1)):
        assert dense(lib, csa2.CacheStruct(6 << 32, codes, scales, 64, 9 << 32, 1)) == 0
    # and nothing else
    assert dense(lib, csa2.CacheStruct(None, None, None, 64, 9 << 32, 1)) == 1
    assert dense(lib, csa2.CacheStruct((6 << 32) + 8, None, None, 64, 9 << 32, 1)) == 1
    assert dense(lib, csa2.CacheStruct(6 << 32, None, None, 64, None, 1)) == 1
    assert dense(lib, csa2.CacheStruct(6 << 32, None, None, 64, (9 << 32) + 2, 1)) == 1
    assert dense(lib, csa2.CacheStruct(6 << 32, None, None, 60, 9 << 32, 1)) == 1
    assert dense(lib, csa2.CacheStruct(6 << 32, None, None, 64, 9 << 32, 3)) == 2


def test_calls_that_select_still_want_them(lib):
    for codes, scales in ((None, 8 << 32), (7 << 32, None), (None, None)):
        c = csa2.CacheStruct(6 << 32, codes, scales, 64, 9 << 32, 1)
        assert lib.csa2_index_score(ctypes.byref(c), 1 << 20, 1 << 20, 1 << 20, None, 0, 1 << 20, 1, 1, 64, WS, 1 << 20,
                                    None) == 1
        assert lib.csa2_decode(ctypes.byref(c), ctypes.byref(csa2.DecodeArgs()), WS, 1 << 20, None) == 1


def test_a_cache_without_index_keys():
    c = csa2.Cache(3, 12, 2, device="cpu", index=False)
    assert c.idx_codes is None and c.idx_scales is None and c.main_kv.shape == (3, 16, 288)
    for s in (c.struct(), c.sequence(1).struct()):
        assert s.idx_codes is None and s.idx_scales is None and s.cap == 16 and s.m == 2
    assert c.sequence(1).struct().main_kv == c.main_kv.data_ptr() + 16 * 288
    full = csa2.Cache(1, 8, 1, device="cpu").struct()
    assert full.idx_codes and full.idx_scales


@pytest.mark.gpu
def test_dense_attention_over_a_cache_without_index_keys():
    g = torch.Generator().manual_seed(3)
    n = 300
    kv = torch.randint(0, 256, (2, 304, 288), generator=g, dtype=torch.uint8)
    kv[..., 256:] = 0x30
    q = torch.randn(2, 3, 64, 512, generator=g).bfloat16().cuda()
    rows = torch.randn(2, 130, 512, generator=g).bfloat16().cuda()
    pos = torch.from_numpy(n - 3 + np.arange(3)).expand(2, 3).contiguous().cuda()
    base = torch.full((2,), n - 130, dtype=torch.int64, device="cuda")
    ws = csa2.Workspace(csa2.dense_attn_workspace_size(2, 3, n))
    outs = []
    for index in (True, False):
        cache = csa2.Cache(2, 304, 1, index=index)
        cache.main_kv.copy_(kv)
        cache.n_entries.fill_(n)
        outs.append(torch.zeros_like(q))
        csa2.dense_attn(cache, q, rows, base, pos, 0.04, outs[-1], ws, max_n=n)
        csa2.dense_attn(cache.sequence(1), q[1:], rows[1:], base[1:], pos[1:], 0.04, outs[-1][1:], ws, max_n=n)
    assert ws.sync_status()[0] == 0
    assert torch.equal(outs[0], outs[1]) and outs[0].abs().sum() > 0
