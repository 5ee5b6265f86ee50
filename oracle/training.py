"""Oracle: the drafter's training operators (fp64, CPU).

Test infrastructure only (see the package docstring).

DSpark paper, §3.3: the drafter is trained on the target's distributions with
a cross entropy and a total variation loss per block position.  Three
operators are restated here, each from its formula:

  * `teacher_topk`    -- the K largest logits of each target row (value
    descending, equal values by id ascending, -inf never listed) and
    ln sum_v exp(z_v / T) over the whole row;
  * `distill_loss`    -- KL(p || q) or the total variation distance of a
    teacher's list p from q = softmax(z / T), and its gradient.  Without
    teacher_lse p is the softmax over the list; with it p_e = exp(v_e / T -
    lse) and the rest r_t = max(0, 1 - sum p) is one bucket against q's mass
    outside the list.  The gradient goes through the softmax, dz = q (dq -
    sum q dq), from the derivatives with respect to q: -p_e/q_e in the list
    and -r_t/r_s outside it (KL), -[p_e > q_e] and -[r_t > r_s] (TV);
  * `head_xent`       -- cross entropy of softmax(H W^T) against labels
    (-1: the row is left out), and its gradients.

A request (a row, for `head_xent`) with bad data gets a status and NaN
outputs; its gradient rows are zero.
"""

import numpy as np

from .verification import (
    STATUS_BAD_LENGTH,
    STATUS_BAD_TEMPERATURE,
    STATUS_BAD_TOKEN,
    STATUS_NONFINITE,
    _as_np,
    _bad_rows,
)

STATUS_BAD_LIST = 256


def _lse(x):
    """ln sum exp over the last axis (-inf for a row of -inf)."""
    m = np.max(x, axis=-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        return np.log(np.exp(x - m).sum(axis=-1)) + m[..., 0]


def _log_softmax(x, total=None):
    """x - ln sum exp(total), total = x by default, for sums whose logarithm is lost beside the values:
    the largest value is taken off first."""
    total = x if total is None else total
    m = np.max(total)
    with np.errstate(divide="ignore", invalid="ignore"):
        return (x - m) - np.log(np.exp(total - m).sum())


def _request_status(L, G, T):
    if L < 0 or L > G:
        return STATUS_BAD_LENGTH
    return 0 if np.isfinite(T) and T > 0.0 else STATUS_BAD_TEMPERATURE


def teacher_topk(target, K, lengths=None, temperature=None):
    """ids [B, G, K], values [B, G, K], lse [B, G], status [B] for target [B, G+1, V]."""
    B, G, V = target.shape[0], target.shape[1] - 1, target.shape[2]
    Ls = np.full(B, G, dtype=np.int64) if lengths is None else _as_np(lengths).astype(np.int64)
    Ts = np.ones(B) if temperature is None else _as_np(temperature).astype(np.float64)
    ids = np.full((B, G, K), -1, dtype=np.int64)
    vals = np.full((B, G, K), -np.inf)
    lse = np.full((B, G), -np.inf)
    status = np.zeros(B, dtype=np.int64)
    for i in range(B):
        L, T = int(Ls[i]), float(Ts[i])
        st = _request_status(L, G, T)
        if st == 0 and L > 0:
            z = _as_np(target[i, :L]).astype(np.float64)
            if _bad_rows(z).any():
                st = STATUS_NONFINITE
            else:
                for k in range(L):
                    order = np.argsort(-z[k], kind="stable")[:K]
                    order = order[z[k, order] > -np.inf]
                    ids[i, k, :len(order)] = order
                    vals[i, k, :len(order)] = z[k, order]
                lse[i, :L] = _lse(z / T)
        status[i] = st
        if st:
            ids[i], vals[i], lse[i] = -1, np.nan, np.nan
    return dict(ids=ids, values=vals, lse=lse, status=status)


def distill_loss(draft, ids, values, teacher_lse=None, mode="kl", lengths=None, temperature=None, grad_loss=None):
    """loss [B, G], status [B], margin [B, G] and, with grad_loss [B, G], grad [B, G, V].

    margin: the smallest relative distance |p - q| / q of the pairs a total variation loss compares
    (its derivative jumps where p = q); inf for KL.
    """
    B, G, V = draft.shape
    ids, values = _as_np(ids).astype(np.int64), _as_np(values).astype(np.float64)
    Ls = np.full(B, G, dtype=np.int64) if lengths is None else _as_np(lengths).astype(np.int64)
    Ts = np.ones(B) if temperature is None else _as_np(temperature).astype(np.float64)
    tl = None if teacher_lse is None else _as_np(teacher_lse).astype(np.float64)
    loss = np.zeros((B, G))
    status = np.zeros(B, dtype=np.int64)
    margin = np.full((B, G), np.inf)
    grad = None if grad_loss is None else np.zeros((B, G, V))
    qs = np.zeros((B, G, V))
    for i in range(B):
        L, T = int(Ls[i]), float(Ts[i])
        st = _request_status(L, G, T)
        for k in range(L if st == 0 else 0):
            used = (ids[i, k] != -1) & ~(values[i, k] == -np.inf)
            if not used.any():
                continue
            at, v = ids[i, k][used], values[i, k][used]
            if ((at < 0) | (at >= V)).any():
                st |= STATUS_BAD_TOKEN
            inside = at[(at >= 0) & (at < V)]
            if len(set(inside.tolist())) < len(inside):
                st |= STATUS_BAD_LIST
            z = _as_np(draft[i, k]).astype(np.float64)
            bad = bool(_bad_rows(z[None])[0]) or not (v[(at >= 0) & (at < V)] < np.inf).all()
            if bad or (tl is not None and not np.isfinite(tl[i, k])):
                st |= STATUS_NONFINITE
            if st:
                continue
            lq = _log_softmax(z / T)
            outside = np.ones(V, dtype=bool)
            outside[at] = False
            zo = z[outside] / T
            lo = -np.inf
            if (zo > -np.inf).any():   # both sums against the outside's largest value, then that value's own share
                lo = _log_softmax(zo.max(), z / T) - _log_softmax(zo.max(), zo)
            lp = _log_softmax(v / T) if tl is None else v / T - tl[i, k]
            p, q, rs = np.exp(lp), np.exp(lq), np.exp(lo)
            rt = max(0.0, 1.0 - p.sum()) if tl is not None and outside.any() else 0.0
            qs[i, k] = q
            with np.errstate(divide="ignore", invalid="ignore"):
                if mode == "kl":
                    t = np.where(p > 0, p * (lp - lq[at]), 0.0).sum()
                    if rt > 0:
                        t += rt * (np.log(rt) - lo)
                    # q dq per token and its sum, without dividing by q
                    qdq = np.zeros(V)
                    if rt > 0:
                        qdq[outside] = -rt * np.where(q[outside] > 0, np.exp(lq[outside] - lo), 0.0)
                    qdq[at] = -p
                else:
                    up, tup = p > q[at], rt > rs
                    t = np.where(up, p - q[at], 0.0).sum() + max(rt - rs, 0.0)
                    qdq = np.where(outside, -q * tup, 0.0)
                    qdq[at] = np.where(up, -q[at], 0.0)
                    pairs = np.abs(p - q[at]) / q[at]
                    margin[i, k] = min(pairs.min(), abs(rt - rs) / rs if rt > 0 and rs > 0 else np.inf)
            loss[i, k] = t
            if grad is not None:
                grad[i, k] = (qdq - q * qdq.sum()) * (float(_as_np(grad_loss)[i, k]) / T)
        status[i] = st
        if st:
            loss[i] = np.nan
            if grad is not None:
                grad[i] = 0.0
    return dict(loss=loss, status=status, margin=margin, grad=grad, q=qs)


def head_xent(hidden, weight, labels, grad_loss=None):
    """loss, lse, status [N]; with grad_loss [N] also grad_hidden, grad_weight, p [N, V] and g [N, V]
    (the gradient with respect to the logits)."""
    h, w = _as_np(hidden).astype(np.float64), _as_np(weight).astype(np.float64)
    y = _as_np(labels).astype(np.int64)
    N, V = len(y), w.shape[0]
    with np.errstate(invalid="ignore", over="ignore"):
        z = h @ w.T
    bad = _bad_rows(z)
    lse = np.full(N, np.nan)
    lse[~bad] = _lse(z[~bad])
    status = np.where((y < -1) | (y >= V), STATUS_BAD_TOKEN, 0) | np.where(bad & (y != -1), STATUS_NONFINITE, 0)
    rows = np.flatnonzero((y >= 0) & (status == 0))
    loss = np.where(status != 0, np.nan, 0.0)
    loss[rows] = lse[rows] - z[rows, y[rows]]
    out = dict(loss=loss, lse=lse, status=status)
    if grad_loss is not None:
        p = np.zeros((N, V))
        p[rows] = np.exp(z[rows] - lse[rows, None])
        g = p.copy()
        g[rows, y[rows]] -= 1.0
        g *= np.where(np.isin(np.arange(N), rows), _as_np(grad_loss).astype(np.float64), 0.0)[:, None]
        out.update(grad_hidden=np.zeros_like(h), grad_weight=np.zeros_like(w), p=p, g=g)
        out["grad_hidden"][rows] = g[rows] @ w
        out["grad_weight"] = g[rows].T @ h[rows]
    return out
