"""Training calls that would be answered wrongly are refused: sizes that do not fit the C ABI's int32 (ctypes
would pass their low 32 bits on), and gradients that would overwrite what the call still reads."""

import ctypes

import pytest
import torch

import draft_verification_04_amd as sv

BIG = (1 << 32) + 8


def _meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused():
    i32 = torch.int32
    small = torch.zeros(2, 3, 4)
    calls = [
        ("K", lambda: sv.teacher_topk(small, BIG)),
        ("K", lambda: sv.teacher_topk(small, -BIG)),
        ("V", lambda: sv.teacher_topk(_meta(2, 3, BIG), 4)),
        ("B", lambda: sv.teacher_topk(_meta(BIG, 3, 4), 4)),
        ("V", lambda: sv.distill_loss(_meta(2, 3, BIG), _meta(2, 3, 4, dtype=i32), _meta(2, 3, 4))),
        ("K", lambda: sv.distill_loss(small, _meta(2, 3, BIG, dtype=i32), _meta(2, 3, BIG))),
        ("K", lambda: sv.distill_loss_backward(small, _meta(2, 3, BIG, dtype=i32), _meta(2, 3, BIG),
                                               _meta(2, 3, 8, dtype=torch.float64), _meta(2, 3))),
        ("N", lambda: sv.head_xent(_meta(BIG, 8), _meta(5, 8), _meta(BIG, dtype=i32))),
        ("V", lambda: sv.head_xent(_meta(2, 8), _meta(BIG, 8), _meta(2, dtype=i32))),
        ("d", lambda: sv.head_xent_backward(_meta(2, BIG), _meta(5, BIG), _meta(2, dtype=i32), _meta(2), _meta(2))),
    ]
    for name, call in calls:
        with pytest.raises(ValueError, match=f"^{name} = "):
            call()


def test_gradients_over_inputs_are_refused():
    """The buffer is host memory: every call below is refused before anything is enqueued."""
    lib = sv.load_library()
    N, V, d, dt = 4, 16, 64, 1                       # hidden 512 bytes, weight 2048
    ws = lib.spec_head_xent_backward_workspace_size(N, V, d, dt)
    buf = (ctypes.c_uint8 * (ws + 16384))()
    base = (ctypes.addressof(buf) + 255) & ~255
    at = lambda n: ctypes.c_void_p(base + n)
    where = dict(h=0, W=512, y=2560, ls=2576, g=2592, gh=3328, gw=4096)
    work = at(8192)

    def call(**moved):
        w = {**where, **moved}
        return lib.spec_head_xent_backward(N, V, d, dt, at(w["h"]), at(w["W"]), at(w["y"]), at(w["ls"]), at(w["g"]),
                                           at(w["gh"]), at(w["gw"]), work, ws, None)
    for moved in (dict(gh=0), dict(gh=256), dict(gh=2048), dict(gw=512), dict(gw=0), dict(gw=1024), dict(gh=2544),
                  dict(gh=2560), dict(gw=2576), dict(gh=4608), dict(gw=3584)):
        assert call(**moved) == 1, moved

    B, G, V, K = 2, 2, 64, 4                         # logits 512 bytes, the list 64 + 64, saved 256
    where2 = dict(x=0, i=512, v=576, T=640, sv=656, g=912)

    def back(o):
        w = {k: at(n) for k, n in where2.items()}
        return lib.spec_distill_loss_backward(B, G, V, dt, w["x"], K, w["i"], w["v"], 0, w["T"], w["sv"], w["g"], at(o),
                                              None)
    for o in (16, 256, 496, 512, 576, 640, 656, 896, 912):
        assert back(o) == 1, o
