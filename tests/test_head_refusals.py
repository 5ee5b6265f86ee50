"""Refusals of the head's entry points without a GPU: bad arguments come back as codes before anything is enqueued
(C ABI), and the binding refuses tensors of the wrong shape, type or place."""

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


class Places:
    """Addresses standing in for device pointers, far apart: every call here is refused before one is looked at."""

    def __init__(self):
        self.n = 0

    def __call__(self, off=0):
        self.n += 1
        return ctypes.c_void_p((1 << 40) + (self.n << 32) + off)


@pytest.fixture
def p():
    return Places()


def _at(a, n):
    return ctypes.c_void_p(a.value + n)


# Each of these calls has one thing wrong with it; none is ever right, so that nothing is launched.

def test_norm(sv, p):
    lib = sv.load_library()
    x, r, w, h, y, c, s, t = (p() for _ in range(8))

    def call(N=3, d=64, dt=1, x=x, r=r, w=w, eps=1e-6, h=h, y=y, c=None, s=None, t=t):
        return lib.spec_head_norm(N, d, dt, x, r, w, eps, h, y, c, s, t, None)
    for bad in (dict(N=0), dict(N=(1 << 20) + 1), dict(d=0), dict(d=16385), dict(dt=2), dict(x=None), dict(w=None),
                dict(x=_at(x, 8)), dict(r=_at(r, 2)), dict(w=_at(w, 4)), dict(h=_at(h, 8)), dict(y=_at(y, 8)),
                dict(h=None), dict(y=None), dict(y=y, c=c, s=s), dict(y=None, c=c), dict(y=None, s=s),
                dict(y=None, c=_at(c, 8), s=s), dict(y=None, c=c, s=s, d=40),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(h=_at(x, 64)), dict(h=_at(x, -64)), dict(y=_at(r, 128)), dict(h=w), dict(y=w), dict(y=h),
                dict(t=x), dict(t=y), dict(y=None, c=x, s=s), dict(y=None, c=c, s=r), dict(y=None, c=c, s=c),
                dict(y=None, c=h, s=s)):
        assert call(**bad) == 1, bad


def test_norm_backward(sv, p):
    lib = sv.load_library()
    gy, h, w, t, gh, gx, gw, ws = (p() for _ in range(8))
    need = lib.spec_head_norm_backward_workspace_size(3, 64)
    assert need > 0 and need % 256 == 0 and lib.spec_head_norm_backward_workspace_size(0, 64) == 0
    assert lib.spec_head_norm_backward_workspace_size(3, 16385) == 0

    def call(N=3, d=64, dt=1, gy=gy, h=h, w=w, t=t, gh=gh, gx=gx, gw=gw, ws=ws, n=need):
        return lib.spec_head_norm_backward(N, d, dt, gy, h, w, t, gh, gx, gw, ws, n, None)
    for bad in (dict(N=0), dict(d=0), dict(d=16385), dict(dt=2), dict(gy=None), dict(h=None), dict(w=None),
                dict(t=None), dict(gx=None), dict(gy=_at(gy, 8)), dict(h=_at(h, 8)), dict(gh=_at(gh, 8)),
                dict(gx=_at(gx, 8)), dict(gw=_at(gw, 8)), dict(w=_at(w, 8)), dict(gx=_at(gy, 64)), dict(gx=_at(h, -16)),
                dict(gx=w), dict(gx=t), dict(gx=gw), dict(gw=gy), dict(gw=h), dict(gw=w), dict(gw=t), dict(gw=gh)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 2 and call(n=need - 1) == 2 and call(ws=_at(ws, 16)) == 2


def test_quantize_and_logits(sv, p):
    lib = sv.load_library()
    w, c, s, x, sx, z = (p() for _ in range(6))

    def quant(V=5, d=64, dt=1, w=w, c=c, s=s):
        return lib.spec_head_quantize(V, d, dt, w, c, s, None)
    for bad in (dict(V=0), dict(V=524289), dict(d=0), dict(d=8), dict(d=40), dict(d=16400), dict(dt=2), dict(w=None),
                dict(c=None), dict(s=None), dict(w=_at(w, 8)), dict(c=_at(c, 8)), dict(c=w), dict(s=w), dict(s=c),
                dict(c=_at(w, 512))):
        assert quant(**bad) == 1, bad

    def logits(N=3, V=5, d=64, dt=1, x=x, sx=sx, w=w, s=s, z=z):
        return lib.spec_head_logits(N, V, d, dt, x, sx, w, s, z, None)
    for bad in (dict(N=0), dict(N=(1 << 20) + 1), dict(V=0), dict(V=524289), dict(d=8), dict(d=40), dict(d=16400),
                dict(dt=2), dict(x=None), dict(sx=None), dict(w=None), dict(s=None), dict(z=None), dict(x=_at(x, 8)),
                dict(w=_at(w, 8)), dict(z=_at(z, 8)), dict(z=x), dict(z=sx), dict(z=w), dict(z=s), dict(x=_at(z, 16))):
        assert logits(**bad) == 1, bad


def test_adjust(sv, p):
    lib = sv.load_library()
    z, x, L, H, hl, pl, r, f, q, bo, bt, bv, m, mi, o, st = (p() for _ in range(16))

    def call(B=2, R=4, V=100, dt=1, z=z, G=3, x=x, L=L, H=H, nH=10, hl=hl, pl=pl, r=r, f=f, q=q, bo=bo, bt=bt, bv=bv,
             nb=5, m=m, M=2, mi=mi, o=o, st=st):
        return lib.spec_adjust_logits(B, R, V, dt, z, G, x, L, H, nH, hl, pl, r, f, q, bo, bt, bv, nb, m, M, mi, o, st,
                                      None)
    for bad in (dict(B=0), dict(R=0, G=0), dict(R=5), dict(R=2), dict(G=-1), dict(G=65, R=65), dict(V=0),
                dict(V=524289), dict(V=262145, dt=0), dict(dt=2), dict(z=None), dict(z=_at(z, 8)), dict(o=None),
                dict(o=_at(o, 8)), dict(x=None), dict(H=None), dict(nH=0), dict(nH=(1 << 28) + 1),
                dict(H=None, nH=0), dict(H=None, nH=0, hl=None), dict(H=None, nH=10, hl=None, pl=None),
                dict(bo=None), dict(bt=None), dict(bv=None), dict(bo=None, bt=None, bv=None), dict(nb=-1),
                dict(m=None), dict(m=None, M=0), dict(M=0), dict(mi=None, M=1),
                dict(o=_at(z, 16)), dict(o=_at(z, -16)), dict(o=x), dict(o=L), dict(o=H), dict(o=hl), dict(o=pl), dict(o=r),
                dict(o=f), dict(o=q), dict(o=bo), dict(o=bt), dict(o=bv), dict(o=m), dict(o=mi), dict(st=o), dict(st=z),
                dict(st=H), dict(st=L), dict(st=m)):
        assert call(**bad) == 1, bad
    # 2^31 - 1 requests of 64 slices pass the dispatch packet's 32-bit work-item count
    far = [ctypes.c_void_p(k << 52) for k in range(1, 4)]
    assert lib.spec_adjust_logits((1 << 31) - 1, 1, 524288, 1, far[0], 0, None, None, None, 0, None, None, None, None,
                                  None, None, None, None, 0, None, 0, None, far[1], far[2], None) == 3
    # so do 2^22 requests of one slice each, where long histories make it a slice of 1024 threads
    far = [ctypes.c_void_p(k << 52) for k in range(1, 6)]
    assert lib.spec_adjust_logits(1 << 22, 1, 4096, 1, far[0], 0, None, None, far[3], 9000, None, None, far[4], None,
                                  None, None, None, None, 0, None, 0, None, far[1], far[2], None) == 3


def test_binding_refuses_before_the_device(sv):
    f = torch.zeros
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    c8 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="x must be"):
        sv.head_norm(f(3), f(3))
    with pytest.raises(ValueError, match="weight"):
        sv.head_norm(f(2, 3), f(4))
    with pytest.raises(ValueError, match="residual"):
        sv.head_norm(f(2, 3), f(3), f(3, 2))
    with pytest.raises(TypeError, match="CUDA"):
        sv.head_norm(f(2, 3), f(3))
    with pytest.raises(ValueError, match="rstd"):
        sv.head_norm_backward(f(2, 3), f(2, 3), f(3), f(3))
    with pytest.raises(ValueError, match="grad_h"):
        sv.head_norm_backward(f(2, 3), f(2, 3), f(3), f(2), f(2, 4))
    with pytest.raises(TypeError, match="CUDA"):
        sv.head_norm_backward(f(2, 3), f(2, 3), f(3), f(2))
    with pytest.raises(ValueError, match="weight"):
        sv.head_quantize(f(3))
    with pytest.raises(TypeError, match="CUDA"):
        sv.head_quantize(f(3, 16))
    with pytest.raises(ValueError, match="weight_codes"):
        sv.head_logits(c8(2, 16), f(2, 1), c8(3, 32), f(1, 1))
    with pytest.raises(ValueError, match="scales"):
        sv.head_logits(c8(2, 144), f(2, 1), c8(3, 144), f(1, 2))
    with pytest.raises(ValueError, match="weight_scales"):
        sv.head_logits(c8(2, 144), f(2, 2), c8(129, 144), f(1, 2))
    with pytest.raises(TypeError, match="logits are"):
        sv.head_logits(c8(2, 16), f(2, 1), c8(3, 16), f(1, 1), dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA"):
        sv.head_logits(c8(2, 16), f(2, 1), c8(3, 16), f(1, 1))
    z = f(2, 4, 50)
    for kw, match in ((dict(draft_tokens=i(2, 5)), "rows"), (dict(draft_tokens=None), "rows"),
                      (dict(draft_tokens=i(3, 3)), "draft_tokens"), (dict(lengths=i(3)), "lengths"),
                      (dict(history=i(3, 9)), "history"), (dict(history_len=i(2)), "history"),
                      (dict(repetition=f(3)), "repetition"), (dict(bias=(i(2), i(4), f(4))), "offsets"),
                      (dict(bias=(i(3), i(4), f(5))), "values"), (dict(mask=i(2, 4, 1)), "mask"),
                      (dict(mask=i(2, 3, 2)), "mask"), (dict(mask_index=i(2)), "mask"), (dict(out=f(2, 4, 51)), "out"),
                      (dict(status=i(3)), "status")):
        with pytest.raises(ValueError, match=match):
            sv.adjust_logits(z, **dict(dict(draft_tokens=i(2, 3)), **kw))
    with pytest.raises(TypeError, match="CUDA"):
        sv.adjust_logits(z, i(2, 3))
