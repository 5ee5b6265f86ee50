"""Pins of the oracle of the head's operators: torch's own conversions and autograd, closed forms, small cases by
hand."""

import math

import numpy as np
import pytest
import torch

import oracle


def test_e4m3_is_torchs_conversion():
    rng = np.random.default_rng(1)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)].double()
    assert np.array_equal(oracle.e4m3(every.numpy()), every.numpy())            # its own numbers
    s = torch.sort(every).values.unique()
    mid = ((s[1:] + s[:-1]) / 2).numpy()                                        # ties go to the even code
    x = np.concatenate([mid, rng.normal(0, 30, 4000).astype(np.float32), rng.normal(0, 0.01, 4000).astype(np.float32)])
    x = x[np.abs(x) <= 448]
    ref = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3(x), ref)


def test_quantize_blocks():
    x = np.zeros((3, 130))
    x[0, 5], x[1, 128], x[2, 129] = -896.0, 7.0, 3.5
    o = oracle.quantize(x, 1)
    assert o["scales"][0].tolist() == [2.0, 2.0 ** -100 / 448] and o["scales"][1, 1] == 7.0 / 448
    assert o["codes"][0, 5] == -448 and o["codes"][1, 128] == 448 and o["codes"][2, 129] == 448
    o = oracle.quantize(x, 128)
    assert o["scales"].tolist() == [[2.0, 7.0 / 448]] and o["codes"][2, 129] == 224


def test_norm_and_its_gradients_match_autograd():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, res, w, gy, gh = r(5, 33), r(5, 33), r(33), r(5, 33), r(5, 33)
    x.requires_grad_(), res.requires_grad_(), w.requires_grad_()
    h = x + res
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-3) * w
    o = oracle.head_norm(x.detach().numpy(), w.detach().numpy(), res.detach().numpy(), 1e-3)
    assert np.allclose(o["y"], y.detach().numpy(), rtol=0, atol=1e-12)
    ((y * gy).sum() + (h * gh).sum()).backward()
    b = oracle.head_norm_grad(gy.numpy(), o["h"], w.detach().numpy(), o["rstd"], gh.numpy())
    for t in (x, res):
        assert np.allclose(b["grad_x"], t.grad.numpy(), rtol=0, atol=1e-12)
    assert np.allclose(b["grad_weight"], w.grad.numpy(), rtol=0, atol=1e-12)


def test_head_logits_by_hand():
    x, w = np.ones((1, 130)), np.ones((129, 130))
    o = oracle.head_logits(x, [[2.0, 3.0]], w, [[1.0, 10.0], [0.5, 0.25]])
    assert o["logits"].tolist()[0] == [2 * 128 + 3 * 10 * 2] * 128 + [128 + 0.75 * 2]


def test_adjust_by_hand():
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    z = torch.tensor([[[1.0, -1.0, 2.0, 4.0, 0.0, 8.0, -3.0]] * 3])
    o = oracle.adjust_logits(z, i([2, 3]), None, i([0, 6, -1, 3, 3, 9]), i(5), i(2), torch.tensor([2.0]),
                             torch.tensor([0.5]), torch.tensor([0.25]),
                             (i(0, 3), i(4, 5, 5), torch.tensor([1.5, 7.0, -math.inf])), i([[0x7f]] * 3))
    # tokens 0 and 6 in the prompt, 3 twice in the output; 5 is banned by the last of its two entries
    row = [0.5, -1.0, 2.0, 2.0 - 1.0 - 0.25, 1.5, -math.inf, -6.0]
    assert o["logits"][0, 0].tolist() == row and o["status"].tolist() == [0]
    row[2] = 1.0 - 0.5 - 0.25                                   # behind the first draft
    assert o["logits"][0, 1].tolist() == row
    row[3] = 2.0 - 1.5 - 0.25                                   # and the second
    assert o["logits"][0, 2].tolist() == row
    o = oracle.adjust_logits(z, i([2, 3]), None, None, mask=i([[0x7f], [0], [0x55]]))
    assert np.isneginf(o["logits"][0, 1]).all() and o["logits"][0, 2, ::2].tolist() == [1, 2, 0, -3]
    assert np.isneginf(o["logits"][0, 2, 1::2]).all()


@pytest.mark.parametrize("kw, bit", [
    (dict(lengths=[3]), 8), (dict(lengths=[-1]), 8), (dict(history_len=[7]), 8), (dict(prompt_len=[7]), 8),
    (dict(repetition=[0.0]), 512), (dict(repetition=[math.nan]), 512), (dict(frequency=[math.inf]), 512),
    (dict(history=[[0, 0, 0, 0, 0, 7]]), 1), (dict(history=[[0, 0, 0, 0, 0, -2]]), 1), (dict(draft_tokens=[[7, 0]]), 1),
    (dict(bias=([0, 2], [0], [1.0])), 256), (dict(bias=([1, 0], [0], [1.0])), 256),
    (dict(bias=([0, 1], [7], [1.0])), 1), (dict(mask_index=[1]), 1024), (dict(mask_index=[-2]), 1024)])
def test_adjust_status(kw, bit):
    z = torch.zeros((1, 3, 7))
    base = dict(draft_tokens=[[2, 3]], lengths=None, history=[[0, 1, 2, 3, 4, 5]], history_len=None, prompt_len=None,
                repetition=[1.1], frequency=[0.0], presence=[0.0], mask=[[[0]] * 3], mask_index=[-1], bias=None)
    base.update(kw)
    f = ("repetition", "frequency", "presence")
    t = {k: None if v is None or k == "bias" else torch.tensor(v, dtype=torch.float32 if k in f else torch.int32)
         for k, v in base.items()}
    if base["bias"]:
        o, i, v = base["bias"]
        t["bias"] = (torch.tensor(o, dtype=torch.int32), torch.tensor(i, dtype=torch.int32), torch.tensor(v))
    o = oracle.adjust_logits(z, t.pop("draft_tokens"), t.pop("lengths"), **t)
    assert o["status"].tolist() == [bit]
    assert (o["logits"] == 0).all()
