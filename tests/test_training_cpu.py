"""Argument checks of the training operators' C entries, on the CPU: nothing is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    from nvfp4_bit_quantized_gb300 import _lib
    return _lib


FAR = 0x10000


def test_layer_norm_rejects_bad_arguments(lib):
    L = lib.lib()
    good = dict(x=FAR, xt=1, rows=4, cols=64, ldx=64, res=None, ldr=0, w=FAR, b=None, wt=0, eps=1e-5, y=FAR, yt=1, ldy=64,
                h=None, ldh=0, mean=FAR, rstd=FAR)

    def fwd(**kw):
        return L.nvfp4_layer_norm_forward(*{**good, **kw}.values(), None)
    for kw, want in [(dict(xt=3), lib.ERR_INVALID_ARG), (dict(yt=-1), lib.ERR_INVALID_ARG), (dict(wt=2), lib.ERR_INVALID_ARG),
                     (dict(cols=0), lib.ERR_SHAPE), (dict(rows=-1), lib.ERR_SHAPE), (dict(ldx=63), lib.ERR_SHAPE),
                     (dict(ldy=63), lib.ERR_SHAPE), (dict(eps=-1.0), lib.ERR_INVALID_ARG),
                     (dict(eps=float("inf")), lib.ERR_INVALID_ARG), (dict(eps=float("nan")), lib.ERR_INVALID_ARG),
                     (dict(x=None), lib.ERR_INVALID_ARG), (dict(w=None), lib.ERR_INVALID_ARG),
                     (dict(mean=None), lib.ERR_INVALID_ARG), (dict(res=FAR, ldr=64), lib.ERR_INVALID_ARG),
                     (dict(res=FAR, ldr=63, h=FAR, ldh=64), lib.ERR_SHAPE), (dict(x=FAR + 1), lib.ERR_ALIGNMENT),
                     (dict(w=FAR + 2), lib.ERR_ALIGNMENT), (dict(rows=0, x=None), lib.OK)]:
        assert fwd(**kw) == want, kw
    size = L.nvfp4_layer_norm_backward_workspace_bytes(4, 64)
    assert size > 0 and L.nvfp4_layer_norm_backward_workspace_bytes(4, 0) == 0
    good = dict(dy=FAR, yt=1, lddy=64, x=FAR, xt=1, rows=4, cols=64, ldx=64, w=FAR, wt=0, mean=FAR, rstd=FAR, dh=None, lddh=0,
                dx=FAR, lddx=64, dw=FAR, db=None, ws=FAR, n=size)

    def bwd(**kw):
        return L.nvfp4_layer_norm_backward(*{**good, **kw}.values(), None)
    for kw, want in [(dict(xt=9), lib.ERR_INVALID_ARG), (dict(cols=0), lib.ERR_SHAPE), (dict(lddy=1), lib.ERR_SHAPE),
                     (dict(lddx=1), lib.ERR_SHAPE), (dict(dh=FAR, lddh=3), lib.ERR_SHAPE), (dict(dw=None), lib.ERR_INVALID_ARG),
                     (dict(rstd=None), lib.ERR_INVALID_ARG), (dict(dw=FAR + 2), lib.ERR_ALIGNMENT),
                     (dict(ws=None), lib.ERR_WORKSPACE), (dict(n=size - 1), lib.ERR_WORKSPACE),
                     (dict(ws=FAR + 4), lib.ERR_WORKSPACE)]:
        assert bwd(**kw) == want, kw


def test_attention_rejects_bad_arguments(lib):
    L, ref = lib.lib(), ctypes.byref

    def shape(**kw):
        a = dict(tq=8, tk=8, heads=4, kv_heads=2, dim=64, causal=1, scale=0.125, nseq=1, cu_q=None, cu_k=None)
        return lib.AttentionShapeC(*{**a, **kw}.values())

    def heads(data=FAR, ts=512, hs=64):
        return lib.HeadsC(data, ts, hs)

    def fwd(s, q=None, lse=FAR):
        q = heads() if q is None else q
        return L.nvfp4_attention_forward(ref(s), ref(q), ref(heads()), ref(heads()), ref(heads()), lse, None, None)

    def bwd(s, ws=FAR, n=1 << 30):
        h = ref(heads())
        return L.nvfp4_attention_backward(ref(s), h, h, h, h, h, FAR, h, h, h, ws, n, None, None)
    for kw, want in [(dict(tq=-1), lib.ERR_SHAPE), (dict(heads=3), lib.ERR_SHAPE), (dict(kv_heads=0), lib.ERR_SHAPE),
                     (dict(dim=60), lib.ERR_SHAPE), (dict(dim=136), lib.ERR_SHAPE), (dict(dim=0), lib.ERR_SHAPE),
                     (dict(nseq=0), lib.ERR_INVALID_ARG), (dict(nseq=2), lib.ERR_INVALID_ARG),
                     (dict(cu_q=FAR), lib.ERR_INVALID_ARG), (dict(cu_q=FAR, cu_k=FAR + 2), lib.ERR_ALIGNMENT),
                     (dict(scale=float("nan")), lib.ERR_INVALID_ARG)]:
        assert fwd(shape(**kw)) == want, kw
        assert bwd(shape(**kw)) == want, kw
        assert L.nvfp4_attention_backward_workspace_bytes(ref(shape(**kw))) == 0
    assert fwd(shape(), heads(None)) == lib.ERR_INVALID_ARG
    assert fwd(shape(), heads(FAR + 8)) == lib.ERR_ALIGNMENT
    assert fwd(shape(), heads(ts=260)) == lib.ERR_ALIGNMENT
    assert fwd(shape(), heads(hs=68)) == lib.ERR_ALIGNMENT
    assert fwd(shape(), heads(hs=0)) == lib.ERR_SHAPE
    assert fwd(shape(), heads(ts=32)) == lib.ERR_SHAPE
    assert fwd(shape(), lse=None) == lib.ERR_INVALID_ARG
    assert fwd(shape(tq=0), heads(None)) == lib.OK
    need = L.nvfp4_attention_backward_workspace_bytes(ref(shape()))
    assert need >= 4 * 8 * 4
    assert bwd(shape(), ws=None) == lib.ERR_WORKSPACE
    assert bwd(shape(), n=need - 1) == lib.ERR_WORKSPACE
    assert bwd(shape(), ws=FAR + 4) == lib.ERR_WORKSPACE


def test_adamw_rejects_bad_arguments(lib):
    L = lib.lib()

    def call(t=None, count=1, **kw):
        a = dict(param=FAR, grad=FAR, m=FAR, v=FAR, ms=FAR, vs=FAR, n=100, pt=0, gt=1, wd=0.1, id=0)
        h = dict(bits=8, round=1, step=1, lr=0.1, b1=0.9, b2=0.95, eps=1e-8, seed=1)
        tensor = (lib.AdamWTensorC * 1)(lib.AdamWTensorC(*{**a, **(t or {})}.values()))
        hp = lib.AdamWParams(*{**h, **kw}.values())
        return L.nvfp4_adamw_step(tensor, count, ctypes.byref(hp), None, None, None)
    for t, kw, want in [({}, dict(bits=16), lib.ERR_INVALID_ARG), ({}, dict(round=2), lib.ERR_INVALID_ARG),
                        ({}, dict(step=0), lib.ERR_INVALID_ARG), ({}, dict(step=2**32), lib.ERR_INVALID_ARG),
                        ({}, dict(b1=1.0), lib.ERR_INVALID_ARG), ({}, dict(b2=-0.1), lib.ERR_INVALID_ARG),
                        ({}, dict(eps=-1.0), lib.ERR_INVALID_ARG), ({}, dict(lr=float("inf")), lib.ERR_INVALID_ARG),
                        (dict(n=-1), {}, lib.ERR_SHAPE), (dict(pt=2), {}, lib.ERR_INVALID_ARG),
                        (dict(gt=-1), {}, lib.ERR_INVALID_ARG), (dict(id=-1), {}, lib.ERR_INVALID_ARG),
                        (dict(wd=float("nan")), {}, lib.ERR_INVALID_ARG), (dict(param=None), {}, lib.ERR_INVALID_ARG),
                        (dict(ms=None), {}, lib.ERR_INVALID_ARG), (dict(param=FAR + 2), {}, lib.ERR_ALIGNMENT),
                        (dict(m=FAR + 1), dict(bits=32), lib.ERR_ALIGNMENT), (dict(vs=FAR + 1), {}, lib.ERR_ALIGNMENT),
                        (dict(n=0, param=None), {}, lib.OK), (dict(grad=None), {}, lib.OK)]:
        assert call(t, **kw) == want, (t, kw)
    assert call(count=0) == lib.OK and call(count=-1) == lib.ERR_INVALID_ARG
    assert L.nvfp4_adamw_step(None, 1, None, None, None, None) == lib.ERR_INVALID_ARG


def test_attention_forward_rejects_a_bad_workspace(lib):
    L, ref = lib.lib(), ctypes.byref
    s = lib.AttentionShapeC(8, 8, 4, 2, 64, 1, 0.125, 1, None, None)
    h = lib.HeadsC(FAR, 512, 64)
    need = L.nvfp4_attention_forward_workspace_bytes(ref(s))
    assert need > 0
    assert L.nvfp4_attention_forward_workspace_bytes(ref(lib.AttentionShapeC(8, 8, 4, 3, 64, 1, 0.125, 1, None, None))) == 0
    for ws, n in ((FAR + 4, need), (FAR, need - 1)):
        assert L.nvfp4_attention_forward_ws(ref(s), ref(h), ref(h), ref(h), ref(h), FAR, ws, n, None, None) == lib.ERR_WORKSPACE


class FakeBuffer:
    def __init__(self, n, **kw):
        self.n = n

    def numel(self):
        return self.n


@pytest.fixture
def workspaces(monkeypatch):
    """api._workspace with the device's part replaced; returns what sets whether the stream is captured."""
    import torch
    from nvfp4_bit_quantized_gb300 import api
    state = {"capturing": False, "stream": 5}
    monkeypatch.setattr(torch, "empty", FakeBuffer)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(api, "_stream", lambda: state["stream"])
    api._ws.clear()
    yield api, state
    api._ws.clear()


def test_a_captured_call_has_scratch_memory_of_its_own(workspaces):
    """A kept buffer is replaced when it grows; what a graph's launches point to must be neither kept nor replaced."""
    api, state = workspaces
    kept = api._workspace(1000)
    assert api._workspace(1 << 16) is kept and api._workspace(1, (0, 5)) is kept
    state["capturing"] = True
    a, b = api._workspace(1000), api._workspace(1000, (0, 5))
    assert kept is not a and kept is not b and a is not b and a.numel() >= 1000
    state["capturing"] = False
    assert api._workspace(1000) is kept
    larger = api._workspace(1 << 20)
    assert larger is not kept and larger is not a and api._workspace(1000) is larger
    state["stream"] = 6
    assert api._workspace(1000) is not larger


def test_threads_do_not_share_scratch_memory(workspaces):
    """Two threads' calls on one stream: their launches may alternate, so what one call leaves for its later launches must not
    lie where the other's does."""
    import threading
    api, _ = workspaces
    mine, theirs = api._workspace(1000), []
    t = threading.Thread(target=lambda: theirs.extend(api._workspace(1000) for _ in range(2)))
    t.start()
    t.join()
    assert theirs[0] is theirs[1] and theirs[0] is not mine and api._workspace(1000) is mine


def test_attention_rejects_more_tiles_than_its_counters_hold(lib):
    """The counter of tiles x heads runs up to three grids past the last one, in 32 bits."""
    L, ref, h = lib.lib(), ctypes.byref, ctypes.byref(lib.HeadsC(FAR, 512, 64))
    for nseq, heads, ok in ((2 ** 25 - 1, 64, False), (2 ** 25 - 1024, 64, False), (2 ** 25 - 1025, 64, True), (2 ** 31 - 200, 1, False)):
        s = lib.AttentionShapeC(8, 8, heads, 1, 64, 1, 0.125, nseq, FAR, FAR)
        for size in (L.nvfp4_attention_backward_workspace_bytes, L.nvfp4_attention_forward_workspace_bytes):
            assert (size(ref(s)) > 0) == ok, (nseq, heads)
        if not ok:
            assert L.nvfp4_attention_forward(ref(s), h, h, h, h, FAR, None, None) == lib.ERR_SHAPE
            assert L.nvfp4_attention_backward(ref(s), h, h, h, h, h, FAR, h, h, h, FAR, 1 << 40, None, None) == lib.ERR_SHAPE
