"""Refusals of the binding's norm and rotation, window attention and dense attention: arguments that
are missing or have another number of axes.  Nothing here reaches the library."""
import pytest
import torch

import fp4_kv_cache_csa2_gb300 as csa2


class _FakeWs:
    """Stands for a workspace: the binding's own checks come before the call."""
    buf, ptr, nbytes = torch.zeros(1, dtype=torch.uint8), 1 << 36, 256


BF16, I64 = torch.bfloat16, torch.int64


def norm_args(**kw):
    a = dict(pos=torch.zeros(2, dtype=I64), rope_cs=torch.zeros(4, 32, 2), ws=_FakeWs, q=torch.zeros(2, 64, 512, dtype=BF16),
             q_out=torch.zeros(2, 64, 512, dtype=BF16), k=torch.zeros(2, 512, dtype=BF16), rows=torch.zeros(5, 512, dtype=BF16))
    a.update(kw)
    return a


def attn_args(name, **kw):
    a = dict(q=torch.zeros(1, 2, 64, 512, dtype=BF16), swa_base_pos=torch.zeros(1, dtype=I64),
             q_pos=torch.zeros(1, 2, dtype=I64), scale=0.1, out=torch.zeros(1, 2, 64, 512, dtype=BF16), ws=_FakeWs)
    if name == "window":
        a.update(rows=torch.zeros(1, 9, 512, dtype=BF16), W=8, sinks=torch.zeros(1, 3, 512, dtype=BF16))
    else:
        a.update(cache=csa2.Cache(1, 8, 1, device="cpu"), swa=torch.zeros(1, 9, 512, dtype=BF16), max_n=8)
    a.update(kw)
    return a


@pytest.mark.parametrize("name", ["pos", "rope_cs", "q_out", "rows"])
def test_norm_refuses_what_is_missing(name):
    with pytest.raises(ValueError, match=f"{name}: missing"):
        csa2.qk_norm_rope(**norm_args(**{name: None}))


@pytest.mark.parametrize("name,shape", [("pos", (1, 2)), ("pos", ()), ("rope_cs", (4, 64)), ("q", (64, 512)), ("q", ()),
                                        ("k", (1, 2, 512)), ("rows", ()), ("rows", (5, 511)), ("q_out", (2, 64 * 512))])
def test_norm_refuses_other_axes(name, shape):
    old = norm_args()[name]
    with pytest.raises(ValueError, match=f"{name}:"):
        csa2.qk_norm_rope(**norm_args(**{name: torch.zeros(shape, dtype=old.dtype)}))


@pytest.mark.parametrize("call,names", [("window", ["q", "rows", "swa_base_pos", "q_pos", "out"]),
                                        ("dense", ["q", "swa", "swa_base_pos", "q_pos", "out"])])
def test_attentions_refuse_what_is_missing_or_has_other_axes(call, names):
    fn = csa2.window_attn if call == "window" else csa2.dense_attn
    for name in names:
        with pytest.raises(ValueError, match=f"{name}: missing"):
            fn(**attn_args(call, **{name: None}))
        old = attn_args(call)[name]
        for other in (old.flatten()[0], old.flatten(), old[None]):
            if other.shape == old.shape:
                continue
            with pytest.raises(ValueError, match=f"{name}:"):
                fn(**attn_args(call, **{name: other}))
    if call == "window":
        with pytest.raises(ValueError, match="sinks:"):
            fn(**attn_args(call, sinks=torch.zeros(3, dtype=BF16)))


def test_a_workspace_on_the_host_is_refused():
    """Everything in host memory agrees with itself: no call may take it to the GPU."""
    for call in (lambda: csa2.qk_norm_rope(**norm_args()), lambda: csa2.window_attn(**attn_args("window")),
                 lambda: csa2.dense_attn(**attn_args("dense"))):
        with pytest.raises(ValueError, match="ws: the workspace is not on a CUDA device"):
            call()


def test_the_current_stream_without_torchs_own_shortcut(monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream if index == 3 else None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 40 + index, raising=False)
    assert csa2._current_stream(3) == 43
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert csa2._current_stream(3) == 77


def test_dense_refuses_a_cache_that_is_not_as_it_says():
    """The tensors of a cache are the caller's to replace: entries of another size or type, fewer than `cap`,
    strided ones, and numbers of entries in 64 bits or of another batch."""
    def call(**kw):
        cache = csa2.Cache(1, 8, 1, device="cpu")
        for name, value in kw.items():
            setattr(cache, name, value)
        return csa2.dense_attn(**attn_args("dense", cache=cache))
    u8 = torch.uint8
    for bad in (torch.zeros(1, 8, 280, dtype=u8), torch.zeros(1, 7, 288, dtype=u8), torch.zeros(2, 8, 288, dtype=u8),
                torch.zeros(1, 8, 288), torch.zeros(1, 16, 288, dtype=u8)[:, ::2], torch.zeros(8, 288, dtype=u8), None):
        with pytest.raises(ValueError, match="cache.main_kv"):
            call(main_kv=bad)
    with pytest.raises(ValueError, match="cache.main_kv"):
        call(cap=16)
    for bad in (torch.zeros(1, dtype=I64), torch.zeros(2, dtype=torch.int32), torch.zeros(1), None):
        with pytest.raises(ValueError, match="cache.n_entries"):
            call(n_entries=bad)
