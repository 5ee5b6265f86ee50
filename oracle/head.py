"""Oracle: from the last hidden state to the logits (fp64, CPU).

Test infrastructure only (see the package docstring).

  * `head_norm`, `head_norm_grad` -- h = x + residual, y = h / sqrt(mean(h^2) + eps) * w, and its gradients at the
    stored h, from the formula (through the mean as well as through h);
  * `e4m3`            -- the nearest number of 4 exponent and 3 mantissa bits (bias 7, no infinities, largest 448),
    ties to even;
  * `quantize`        -- codes (as the numbers they stand for) and scales, max(amax, 2^-100) / 448 for each block of
    `rows` x 128;
  * `head_logits`     -- the product of two such arrays;
  * `adjust_logits`   -- repetition, frequency and presence penalties, biases and masks, row by row of a block.
"""

import numpy as np

from .verification import STATUS_BAD_LENGTH, STATUS_BAD_TOKEN
from .training import STATUS_BAD_LIST

STATUS_BAD_PENALTY = 512
STATUS_BAD_MASK = 1024


def _as_np(t):
    """As fp64 (exact for every type that comes in, the 8-bit ones among them)."""
    return t.detach().cpu().float().double().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def head_norm(x, w, residual=None, eps=1e-6):
    h = _as_np(x) + (0.0 if residual is None else _as_np(residual))
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return dict(h=h, rstd=rstd, y=h * rstd[:, None] * _as_np(w))


def head_norm_grad(grad_y, h, w, rstd, grad_h=None):
    gy, h, w, rstd = (_as_np(t) for t in (grad_y, h, w, rstd))
    xh = h * rstd[:, None]
    g = gy * w
    gx = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return dict(grad_x=gx + (0.0 if grad_h is None else _as_np(grad_h)), grad_weight=(gy * xh).sum(axis=0))


def e4m3_step(q):
    """The distance between neighbouring numbers at q's exponent (2^-9 below 2^-6)."""
    a = np.maximum(np.abs(q), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(a)) - 3.0)


def e4m3(q):
    step = e4m3_step(q)
    return np.clip(np.round(q / step) * step, -448.0, 448.0)   # np.round: ties to even


def _spread(s, rows, n, d):
    return np.repeat(np.repeat(s, rows, 0)[:n], 128, 1)[:, :d]


def quantize(x, rows):
    """dict(q: the quotients before rounding, codes, scales)."""
    x = _as_np(x)
    n, d = x.shape
    nb, gb = -(-n // rows), -(-d // 128)
    s = np.empty((nb, gb))
    for i in range(nb):
        for g in range(gb):
            s[i, g] = max(np.abs(x[i * rows:(i + 1) * rows, g * 128:(g + 1) * 128]).max(), 2.0 ** -100) / 448.0
    q = x / _spread(s, rows, n, d)
    return dict(q=q, codes=e4m3(q), scales=s)


def head_logits(codes, scales, weight_codes, weight_scales):
    """dict(logits, mass: the sum of the terms' magnitudes)."""
    x, w = _as_np(codes), _as_np(weight_codes)
    x = x * _spread(_as_np(scales), 1, *x.shape)
    w = w * _spread(_as_np(weight_scales), 128, *w.shape)
    return dict(logits=x @ w.T, mass=np.abs(x) @ np.abs(w).T)


def adjust_logits(logits, draft_tokens=None, lengths=None, history=None, history_len=None, prompt_len=None,
                  repetition=None, frequency=None, presence=None, bias=None, mask=None, mask_index=None):
    """dict(logits (rows that are not adjusted as they came), status, mass: what the rounding is relative to,
    touched [B, R, V]: the values that a token's penalty, bias or mask reaches)."""
    z = _as_np(logits).copy()
    B, R, V = z.shape
    G = 0 if draft_tokens is None else draft_tokens.shape[1]
    ints = lambda t: None if t is None else t.cpu().numpy().astype(np.int64)
    x, L, hist, hl, pl = (ints(t) for t in (draft_tokens, lengths, history, history_len, prompt_len))
    H = 0 if hist is None else hist.shape[1]
    one = lambda t, k, b: k if t is None else float(_as_np(t)[b])
    offs, btok, bval = (None, None, None) if bias is None else (ints(bias[0]), ints(bias[1]), _as_np(bias[2]))
    words = None if mask is None else mask.cpu().numpy().view(np.uint32)
    status = np.zeros(B, dtype=np.int32)
    mass, touched = np.abs(z), np.zeros(z.shape, dtype=bool)
    for b in range(B):
        n = G if L is None else int(L[b])
        st = 0
        live = n + R - G
        if n < 0 or n > G:
            st, live = st | STATUS_BAD_LENGTH, 0
        h1 = H if hl is None else int(hl[b])
        p1 = 0 if pl is None else int(pl[b])
        if not (0 <= p1 <= h1 <= H):
            st, h1, p1 = st | STATUS_BAD_LENGTH, 0, 0
        rep, freq, pres = one(repetition, 1.0, b), one(frequency, 0.0, b), one(presence, 0.0, b)
        if not (0.0 < rep < np.inf and np.isfinite(freq) and np.isfinite(pres)):
            st |= STATUS_BAD_PENALTY
        penal = rep != 1.0 or freq != 0.0 or pres != 0.0
        line = hist[b, :h1] if penal and live > 0 and h1 else np.zeros(0, dtype=np.int64)
        drafts = x[b, :max(min(live - 1, G), 0)] if penal and G else np.zeros(0, dtype=np.int64)
        if (line < -1).any() or (line >= V).any() or (drafts < 0).any() or (drafts >= V).any():
            st |= STATUS_BAD_TOKEN
        add = np.zeros(V)
        biased = np.zeros(V, dtype=bool)
        if bias is not None:
            lo, hi = int(offs[b]), int(offs[b + 1])
            if lo < 0 or hi < lo or hi > len(btok):
                st |= STATUS_BAD_LIST
            elif live > 0:
                if ((btok[lo:hi] < 0) | (btok[lo:hi] >= V)).any():
                    st |= STATUS_BAD_TOKEN
                else:
                    for t, v in zip(btok[lo:hi], bval[lo:hi]):
                        add[t], biased[t] = v, True
        m = -1 if words is None else (b if mask_index is None else int(mask_index[b]))
        if m < -1 or (words is not None and m >= len(words)):
            st |= STATUS_BAD_MASK
        status[b] = st
        if st:
            continue
        count = np.zeros(V)
        prompt = np.zeros(V, dtype=bool)
        prompt[line[:p1][line[:p1] >= 0]] = True
        np.add.at(count, line[p1:][line[p1:] >= 0], 1.0)
        for k in range(live):
            if k and penal:
                count[drafts[k - 1]] += 1.0
            r = z[b, k]
            seen = prompt | (count > 0)
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(seen, np.where(r > 0, r / rep, r * rep), r)
                size = np.abs(s) + np.abs(freq * count) + np.abs(pres) + np.abs(add)
                s = np.where(seen, s - freq * count - pres * (count > 0), s)
                s = np.where(biased, s + add, s)
            on = np.ones(V, dtype=bool)
            if m >= 0:
                on = (words[m, k][np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1 == 1
            z[b, k] = np.where(on, s, -np.inf)
            mass[b, k] = np.maximum(mass[b, k], size)
            touched[b, k] = seen | biased | ~on
    return dict(logits=z, status=status, mass=mass, touched=touched)
