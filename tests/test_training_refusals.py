"""Refusals of the training entry points without a GPU: bad arguments come back as codes before
anything is enqueued (C ABI), and the binding refuses tensors of the wrong shape, type or place."""

import ctypes
import os

import pytest
import torch

from conftest import ROOT

LIB = os.path.join(ROOT, "draft_verification_04_amd", "libspecverify.so")


@pytest.fixture(scope="module")
def sv():
    if not os.path.exists(LIB):
        pytest.fail("libspecverify.so is not built (run __graft_entry__.build())")
    import draft_verification_04_amd as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def p():
    # a host buffer standing in for device pointers: 16-byte but never 256-byte aligned, so that as a
    # workspace it is refused and nothing is launched
    buf = (ctypes.c_uint8 * 1024)()
    ptr = ctypes.c_void_p(((ctypes.addressof(buf) + 255) & ~255) + 16)
    ptr.keep = buf
    return ptr


def _off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_teacher_topk(sv, p):
    lib = sv.load_library()
    ws = lib.spec_teacher_workspace_size(2, 4, 100, 8)
    assert ws > 0 and ws % 256 == 0
    assert lib.spec_teacher_workspace_size(0, 4, 100, 8) == 0 and lib.spec_teacher_workspace_size(2, 4, 100, 257) == 0

    def call(B=2, G=4, V=100, dt=1, t=p, K=8, T=p, i=p, v=p, w=p, wsb=ws):
        return lib.spec_teacher_topk(B, G, V, dt, t, K, None, T, i, v, None, None, w, wsb, None)
    for bad in (dict(B=0), dict(G=0), dict(G=65), dict(V=0), dict(V=524289), dict(dt=0, V=262145), dict(dt=2),
                dict(t=None), dict(t=_off(p, 2)), dict(K=0), dict(K=257), dict(T=None), dict(i=None), dict(v=None)):
        assert call(**bad) == 1, bad
    assert call(w=None) == 2 and call(wsb=ws - 1) == 2 and call() == 2


def test_teacher_workspace_holds_either_type(sv):
    """The size does not name the storage type: it covers the segments of both (and their lists, where
    a row is cut into several)."""
    lib = sv.load_library()
    for V in (1, 7, 8191, 16384, 16385, 32768, 32769, 262144, 262145, 524288):
        a, b = (lib.spec_teacher_workspace_size(3, 2, V, K) for K in (1, 256))
        assert 0 < a <= b


def test_distill(sv, p):
    lib = sv.load_library()
    ws = lib.spec_distill_workspace_size(2, 4, 100, 8)
    assert ws > 0 and ws % 256 == 0

    def fwd(B=2, G=4, V=100, dt=1, x=p, K=8, i=p, v=p, mode=0, T=p, lo=p, sav=p, w=p, wsb=ws):
        return lib.spec_distill_loss(B, G, V, dt, x, K, i, v, None, mode, None, T, lo, sav, None, w, wsb, None)
    for bad in (dict(B=0), dict(G=65), dict(V=524289), dict(dt=5), dict(x=None), dict(x=_off(p, 4)), dict(K=0),
                dict(K=257), dict(i=None), dict(v=None), dict(mode=2), dict(mode=-1), dict(T=None), dict(lo=None),
                dict(sav=None)):
        assert fwd(**bad) == 1, bad
    assert fwd(w=None) == 2 and fwd(wsb=ws - 1) == 2 and fwd() == 2

    def bwd(B=2, G=4, V=100, dt=1, x=p, K=8, i=p, v=p, mode=0, T=p, sav=p, g=p, o=p):
        return lib.spec_distill_loss_backward(B, G, V, dt, x, K, i, v, mode, T, sav, g, o, None)
    for bad in (dict(B=0), dict(K=0), dict(mode=2), dict(x=None), dict(i=None), dict(v=None), dict(T=None),
                dict(sav=None), dict(g=None), dict(o=None), dict(o=_off(p, 8)), dict(x=_off(p, 8)),
                dict(dt=0, V=262145)):
        assert bwd(**bad) == 1, bad
    # 2^24 requests of 64 positions pass the dispatch packet's 32-bit work-item count
    assert bwd(B=1 << 24, G=64) == 3


def test_head_xent(sv, p):
    lib = sv.load_library()
    ws = lib.spec_head_xent_workspace_size(10, 100, 64, 1)
    wb = lib.spec_head_xent_backward_workspace_size(10, 100, 64, 1)
    assert ws > 0 and ws % 256 == 0 and wb > 0 and wb % 256 == 0
    assert lib.spec_head_xent_workspace_size(10, 100, 60, 1) == 0            # 120-byte rows
    assert lib.spec_head_xent_workspace_size(10, 100, 60, 0) > 0             # 240-byte rows
    assert lib.spec_head_xent_backward_workspace_size(0, 100, 64, 1) == 0

    def fwd(N=10, V=100, d=64, dt=1, h=p, W=p, y=p, lo=p, ls=p, w=p, wsb=ws):
        return lib.spec_head_xent(N, V, d, dt, h, W, y, lo, ls, None, w, wsb, None)

    def bwd(N=10, V=100, d=64, dt=1, h=p, W=p, y=p, ls=p, g=p, gh=p, gw=p, w=p, wsb=wb):
        return lib.spec_head_xent_backward(N, V, d, dt, h, W, y, ls, g, gh, gw, w, wsb, None)
    for f in (fwd, bwd):
        for bad in (dict(N=0), dict(N=(1 << 20) + 1), dict(V=0), dict(V=524289), dict(d=0), dict(d=60),
                    dict(d=16392), dict(dt=2), dict(h=None), dict(h=_off(p, 8)), dict(W=None), dict(W=_off(p, 8)),
                    dict(y=None), dict(ls=None)):
            assert f(**bad) == 1, bad
        assert f(w=None) == 2 and f(wsb=255) == 2 and f() == 2
    assert fwd(lo=None) == 1 and bwd(g=None) == 1 and bwd(gh=None, gw=None) == 1
    assert bwd(gh=_off(p, 4)) == 1 and bwd(gw=_off(p, 4)) == 1


def test_binding_refuses_before_the_device(sv):
    f = torch.zeros
    with pytest.raises(ValueError, match="target"):
        sv.teacher_topk(f(2, 3), 4)
    with pytest.raises(TypeError, match="K"):
        sv.teacher_topk(f(2, 3, 4), 2.0)
    with pytest.raises(ValueError, match="temperature"):
        sv.teacher_topk(f(2, 3, 4), 2, temperature=f(3))
    with pytest.raises(TypeError, match="CUDA"):
        sv.teacher_topk(f(2, 3, 4), 2)
    with pytest.raises(ValueError, match="ids"):
        sv.distill_loss(f(2, 3, 4), f(2, 2, 4), f(2, 2, 4))
    with pytest.raises(ValueError, match="values"):
        sv.distill_loss(f(2, 3, 4), f(2, 3, 4), f(2, 3, 5))
    with pytest.raises(TypeError, match="CUDA"):
        sv.distill_loss(f(2, 3, 4), f(2, 3, 4, dtype=torch.int32), f(2, 3, 4))
    with pytest.raises(ValueError, match="weight"):
        sv.head_xent(f(2, 8), f(5, 16), f(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="labels"):
        sv.head_xent(f(2, 8), f(5, 8), f(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        sv.head_xent(f(2, 8), f(5, 8), f(2, dtype=torch.int32))
