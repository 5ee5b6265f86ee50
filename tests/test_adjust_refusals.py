"""The binding of spec_adjust_logits refuses arrays that the call could not be told apart from none."""

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


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("index", [False, True])
def test_no_masks(sv, index):
    """A mask array of no masks (its address is NULL) is not the same as no mask: without an index every request needs
    one, with an index there is none to name."""
    kw = dict(mask_index=_i(2) - 1) if index else {}
    with pytest.raises(ValueError, match="mask"):
        sv.adjust_logits(torch.zeros(2, 4, 50), _i(2, 3), mask=_i(0, 4, 2), **kw)


@pytest.mark.parametrize("kw", [dict(history_len=_i(3)), dict(prompt_len=_i(2, 1)), dict(history_len=[0, 0])])
def test_lengths_of_a_history_of_no_tokens(sv, kw):
    """They are checked like any others, though there is nothing to read."""
    with pytest.raises(ValueError, match=next(iter(kw))):
        sv.adjust_logits(torch.zeros(2, 4, 50), _i(2, 3), history=_i(2, 0), **kw)
