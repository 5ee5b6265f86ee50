"""Pins of the training oracle (DSpark paper, §3.3): closed forms, other libraries' functions and
finite differences."""

import math

import numpy as np
import pytest
import scipy.special
import torch

import oracle


def _rows(seed, B=3, G=2, V=60):
    rng = np.random.default_rng(seed)
    t = rng.normal(0, 2, (B, G + 1, V)).astype(np.float32)
    d = (t[:, :G] + rng.normal(0, 0.7, (B, G, V))).astype(np.float32)
    return rng, t, d


def test_teacher_list_order_ties_and_missing_entries():
    z = np.full((1, 2, 6), -np.inf, dtype=np.float32)
    z[0, 0] = [1.0, 3.0, 3.0, -np.inf, 0.0, 3.0]
    o = oracle.teacher_topk(z, 4)
    assert o["ids"][0, 0].tolist() == [1, 2, 5, 0] and o["values"][0, 0].tolist() == [3, 3, 3, 1]
    o = oracle.teacher_topk(z, 8)
    assert o["ids"][0, 0].tolist() == [1, 2, 5, 0, 4, -1, -1, -1]
    assert np.isneginf(o["values"][0, 0, 5:]).all()
    assert math.isclose(o["lse"][0, 0], scipy.special.logsumexp([1, 3, 3, 0, 3]), abs_tol=1e-14)


def test_teacher_lse_with_temperature_lengths_and_status():
    rng, t, _ = _rows(1, B=5)
    t[3, 1, 7] = np.nan
    T = np.array([0.7, 1.3, 1.0, 1.0, 0.0], dtype=np.float32)
    o = oracle.teacher_topk(t, 3, [2, 1, 0, 2, 2], T)
    assert o["status"].tolist() == [0, 0, 0, 4, 2]
    assert np.allclose(o["lse"][0], scipy.special.logsumexp(t[0, :2].astype(np.float64) / float(T[0]), axis=-1),
                       rtol=0, atol=1e-13)
    assert np.isneginf(o["lse"][1, 1]) and (o["ids"][2] == -1).all() and np.isnan(o["values"][3]).all()


def test_kl_over_the_whole_vocabulary_matches_torch():
    rng, t, d = _rows(2)
    B, G, V = d.shape
    tt = oracle.teacher_topk(t, V)
    o = oracle.distill_loss(d, tt["ids"], tt["values"])
    ref = torch.nn.functional.kl_div(torch.log_softmax(torch.tensor(d, dtype=torch.float64), -1),
                                     torch.log_softmax(torch.tensor(t[:, :G], dtype=torch.float64), -1),
                                     reduction="none", log_target=True).sum(-1).numpy()
    assert np.allclose(o["loss"], ref, rtol=0, atol=1e-12)
    o = oracle.distill_loss(d, tt["ids"], tt["values"], tt["lse"])     # no token outside: no tail
    assert np.allclose(o["loss"], ref, rtol=0, atol=1e-12)


def test_tv_is_one_minus_the_overlap_mass():
    rng, t, d = _rows(3)
    T = np.array([0.6, 1.0, 1.7], dtype=np.float32)
    tt = oracle.teacher_topk(t, d.shape[2], None, T)
    o = oracle.distill_loss(d, tt["ids"], tt["values"], None, "tv", None, T)
    assert np.allclose(o["loss"], 1.0 - oracle.overlap_mass(t, d, None, T)["overlap"], rtol=0, atol=1e-12)


def test_rows_of_one_huge_value_are_uniform():
    """Every logit at the lowest fp32 value (a row that a mask leaves empty): q = 1/V, p = 1/K."""
    V, K = 50, 8
    d = np.full((1, 1, V), np.finfo(np.float32).min)
    ids, vals = np.arange(K).reshape(1, 1, K), np.full((1, 1, K), np.finfo(np.float32).min)
    kl = oracle.distill_loss(d, ids, vals, grad_loss=np.ones((1, 1)))
    assert abs(kl["loss"][0, 0] - np.log(V / K)) < 1e-14
    want = np.full(V, 1 / V)
    want[:K] -= 1 / K
    assert np.abs(kl["grad"][0, 0] - want).max() < 1e-15
    tv = oracle.distill_loss(d, ids, vals, mode="tv")
    assert abs(tv["loss"][0, 0] - (1 - K / V)) < 1e-14


def test_the_tail_is_one_bucket():
    """With the tail kept the loss is that of the distributions over K + 1 outcomes."""
    rng, t, d = _rows(4, B=1, G=1)
    tt = oracle.teacher_topk(t, 5)
    p = scipy.special.softmax(t[0, 0].astype(np.float64))
    q = scipy.special.softmax(d[0, 0].astype(np.float64))
    at = tt["ids"][0, 0]
    pb, qb = np.append(p[at], 1 - p[at].sum()), np.append(q[at], 1 - q[at].sum())
    kl = oracle.distill_loss(d, tt["ids"], tt["values"], tt["lse"])["loss"][0, 0]
    tv = oracle.distill_loss(d, tt["ids"], tt["values"], tt["lse"], "tv")["loss"][0, 0]
    assert math.isclose(kl, (pb * np.log(pb / qb)).sum(), abs_tol=1e-12)
    assert math.isclose(tv, 0.5 * np.abs(pb - qb).sum(), abs_tol=1e-12)


@pytest.mark.parametrize("mode", ["kl", "tv"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(mode, tail):
    rng, t, d = _rows(5, B=2, G=2, V=17)
    d = d.astype(np.float64)
    T = np.array([0.8, 1.4])
    tt = oracle.teacher_topk(t, 5, None, T)
    w = rng.normal(0, 1, (2, 2))

    def f(x):
        return (w * oracle.distill_loss(x, tt["ids"], tt["values"], tt["lse"] if tail else None, mode, None,
                                        T)["loss"]).sum()
    o = oracle.distill_loss(d, tt["ids"], tt["values"], tt["lse"] if tail else None, mode, None, T, w)
    assert o["margin"].min() > 1e-3          # no kink within a step of 1e-5
    h = 1e-5
    for _ in range(40):
        at = tuple(int(rng.integers(n)) for n in d.shape)
        x = d.copy()
        x[at] += h
        y = d.copy()
        y[at] -= h
        assert math.isclose((f(x) - f(y)) / (2 * h), o["grad"][at], abs_tol=1e-8)


def test_distill_status_and_empty_rows():
    rng, t, d = _rows(6, B=6, G=2, V=9)
    tt = oracle.teacher_topk(t, 3)
    ids, vals = tt["ids"].copy(), tt["values"].copy()
    ids[0, 0] = -1                     # nothing named: the row is not read
    d[0, 0, 2] = np.nan
    ids[1, 1, 0] = 9
    ids[2, 0, 1] = ids[2, 0, 0]
    d[3, 1, 4] = np.inf
    vals[4, 0, 2] = np.nan
    o = oracle.distill_loss(d, ids, vals, grad_loss=np.ones((6, 2)))
    assert o["status"].tolist() == [0, 1, 256, 4, 4, 0]
    assert o["loss"][0, 0] == 0 and (o["grad"][0, 0] == 0).all() and o["loss"][0, 1] > 0
    assert np.isnan(o["loss"][1:5]).all() and (o["grad"][1:5] == 0).all()


def test_head_xent_against_torch_and_differences():
    rng = np.random.default_rng(7)
    N, V, d = 9, 13, 6
    h, w = rng.normal(0, 1, (N, d)), rng.normal(0, 1, (V, d))
    y = rng.integers(0, V, N)
    y[2] = -1
    g = rng.normal(0, 1, N)
    o = oracle.head_xent(h, w, y, g)
    H = torch.tensor(h, requires_grad=True)
    W = torch.tensor(w, requires_grad=True)
    loss = torch.nn.functional.cross_entropy(H @ W.t(), torch.tensor(y), ignore_index=-1, reduction="none")
    (loss * torch.tensor(g)).sum().backward()
    assert np.allclose(o["loss"], loss.detach().numpy(), rtol=0, atol=1e-13)
    assert np.allclose(o["grad_hidden"], H.grad.numpy(), rtol=0, atol=1e-13)
    assert np.allclose(o["grad_weight"], W.grad.numpy(), rtol=0, atol=1e-13)
    e = 1e-6
    for _ in range(20):
        at = (int(rng.integers(V)), int(rng.integers(d)))
        wp, wm = w.copy(), w.copy()
        wp[at] += e
        wm[at] -= e
        diff = (np.dot(g, oracle.head_xent(h, wp, y)["loss"]) - np.dot(g, oracle.head_xent(h, wm, y)["loss"])) / (2 * e)
        assert math.isclose(diff, o["grad_weight"][at], abs_tol=1e-7)


def test_head_xent_bad_rows_add_nothing():
    rng = np.random.default_rng(8)
    h, w = rng.normal(0, 1, (5, 4)), rng.normal(0, 1, (7, 4))
    h[1] = np.inf
    h[4, 0] = np.nan
    y = np.array([3, 2, 7, -2, -1])
    o = oracle.head_xent(h, w, y, np.ones(5))
    assert o["status"].tolist() == [0, 4, 1, 1, 0]
    assert np.isnan(o["loss"][1:4]).all() and o["loss"][4] == 0 and np.isnan(o["lse"][4])
    only = oracle.head_xent(h[:1], w, y[:1], np.ones(1))
    assert np.allclose(o["grad_weight"], only["grad_weight"]) and (o["grad_hidden"][1:] == 0).all()
