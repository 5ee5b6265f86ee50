"""Sizes that do not fit the C ABI's int32 are refused by the binding (ctypes would pass their low 32 bits on)."""

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
