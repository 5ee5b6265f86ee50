"""Edges of the drafter's training operators that ordinary rows do not reach (u = 2^-24, half a step of
fp32; a term, a sum and a difference each bounded where it is tested)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import oracle

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import draft_verification_04_amd as m
    m.load_library()
    return m


def _np(t):
    t = t.detach().cpu()
    return (t.double() if t.is_floating_point() else t).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,g", [(1e-38, 10.0), (2.0 ** -100, 2.0 ** 35), (1.0, 2.0 ** 127)])
def test_distill_gradient_with_factors_past_fp32(sv, dtype, T, g):
    """grad_loss / T past fp32's largest value: tokens without mass still get 0, values in range stay right and
    only those past the type's range are infinite.  Outside the list 2^10 equal logits share the draft's mass."""
    V, K = 5000, 3
    z = torch.full((1, 2, V), -1.0, device=DEV)
    z[0, :, 1000:1000 + 2 ** 10] = 1.0
    z[0, 1, 7] = 1.0                         # row 1: a listed token among them
    d = z.to(DT[dtype])
    ids = torch.tensor([[[7, 8, 9]] * 2], dtype=torch.int32, device=DEV)
    vals = torch.tensor([[[0.5, 0.25, -1.0]] * 2], device=DEV)
    temp = torch.tensor([T], device=DEV)
    w = torch.tensor([[g, -g]], device=DEV)
    ref = oracle.distill_loss(d, ids, vals, None, "kl", None, temp, w)
    f = sv.distill_loss(d, ids, vals, None, sv.SPEC_DISTILL_KL, None, temp)
    grad = sv.distill_loss_backward(d, ids, vals, f["saved"], w, sv.SPEC_DISTILL_KL, temp)
    torch.cuda.synchronize()
    got, want = _np(grad), ref["grad"]
    big = np.abs(want) > float(torch.finfo(DT[dtype]).max)
    assert (np.abs(want[0, 0, 1000:2024]) > 1e30).all() and not big[0, 0, 1000:2024].any()
    assert np.isinf(got[big]).all() and (np.sign(got[big]) == np.sign(want[big])).all()
    # q: 700 u (its sum and exponent), one rounding to the type; q below 2^-126 counts as 0
    eps = torch.finfo(DT[dtype]).eps
    scale = g / float(temp[0])
    tol = 700 * U * ref["q"] * scale + eps / 2 * (1 + 2 ** -10) * np.abs(want) + 2.0 ** -126 * scale + 1e-37
    assert (np.abs(got - want)[~big] <= tol[~big]).all()
    if T < 1e-20:
        assert (got[0, :, :1000][:, 10:] == 0).all()


def _lse_of(sv, z, T):
    """spec_teacher_topk's normalisers of the rows z [B, V] (one position a request: 512 requests or more are walked
    whole, a workgroup a row)."""
    t = torch.stack([z, z], 1).contiguous()
    o = sv.teacher_topk(t, 1, None, T)
    torch.cuda.synchronize()
    assert not o["status"].any()
    return _np(o["lse"])[:, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_normaliser_of_a_value_far_above_the_first_chunk(sv, dtype):
    """One token stands 20 to 69 nats above the row's first 64 KB, which the exponents are taken against.  Its
    own term is nearly all of the sum: an exponent below 64 is rounded by 2^-19 at most (22 u of its term), the
    scale's rounding leaves 2 binary orders of itself (1.4 u) and exp2 an ulp (2 u); a larger one is summed against
    the row's largest value, where this term is exactly 1.  Half a step of the result besides."""
    rng = np.random.default_rng(17)
    B, V = 512, 50021
    T = torch.from_numpy(rng.uniform(0.6, 1.4, B).astype(np.float32))
    top = torch.from_numpy(rng.uniform(-2, 2, B).astype(np.float32)).to(torch.bfloat16)
    low = (top.float() - torch.from_numpy(rng.uniform(20, 69, B).astype(np.float32)) * T).to(torch.bfloat16)
    z = low.to(DEV)[:, None].repeat(1, V)
    z[:, 50000] = top.to(DEV)
    got = _lse_of(sv, z.to(DT[dtype]), T.to(DEV))
    t = _np(T)
    want = np.logaddexp(_np(top) / t, _np(low) / t + np.log(V - 1))
    err = np.abs(got - want) / U
    assert (err <= 26 + np.abs(want)).all(), (err.max(), int(err.argmax()))


def test_normaliser_of_rows_summed_again(sv):
    """Rows whose first 64 KB are masked have no reference and are summed a second time: 256 equal terms per
    thread and the row's largest.  They are added in pairs, then vector by vector: 3 + 33 roundings, an ulp of
    exp2 (2 u), 3 u of the exponent, half a step of the result."""
    rng = np.random.default_rng(18)
    B, V, first = 512, 163840, 32768
    T = torch.from_numpy(rng.uniform(0.6, 1.4, B).astype(np.float32))
    v = torch.from_numpy(rng.uniform(-0.25, 0, B).astype(np.float32)).to(torch.bfloat16)
    z = v.to(DEV)[:, None].repeat(1, V)
    z[:, :first] = -float("inf")
    z[:, V - 1] = 0.0
    got = _lse_of(sv, z, T.to(DEV))
    x = _np(v) / _np(T)
    want = np.log(1.0 + (V - first - 1) * np.exp(x))
    err = np.abs(got - want) / U
    assert (err <= 38 + 3 * np.abs(x) + np.abs(want)).all(), (err.max(), int(err.argmax()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,K", [(500, 256), (520, 64), (531, 65), (1000, 65), (1000, 119), (1100, 152), (1500, 129),
                                 (1500, 200), (1800, 193), (2047, 256), (2060, 256), (1025, 256), (263, 256)])
def test_lists_of_rows_without_a_bound(sv, dtype, V, K):
    """Short rows with long lists: too few full waves to take a bound from, every value is a candidate."""
    rng = np.random.default_rng(V + K)
    B, G = 5, 3
    t = torch.from_numpy(rng.normal(0, 3, (B, G + 1, V)).astype(np.float32))
    t[1] = torch.arange(V) / 64.0                      # rising
    t[2] = torch.from_numpy(rng.integers(-2, 3, (G + 1, V)).astype(np.float32))
    t[3, :, rng.random(V) < 0.5] = -np.inf
    t = t.to(DT[dtype]).to(DEV)
    print(f"lists {V} {K} {dtype}", flush=True)
    got = sv.teacher_topk(t, K)
    torch.cuda.synchronize()
    ref = oracle.teacher_topk(t, K)
    assert (_np(got["ids"]) == ref["ids"]).all() and np.array_equal(_np(got["values"]), ref["values"])
    assert (np.abs(_np(got["lse"]) - ref["lse"]) <= U * (110 + np.abs(ref["lse"]))).all()


@pytest.mark.parametrize("N,V,d", [(60, 500, 64), (200, 1000, 208), (300, 2500, 1208), (1100, 3000, 1104)])
def test_label_entries_of_the_head_gradients_are_rounded_once(sv, N, V, d):
    """Hidden states and weights of one value per row, each in a column of its own: every entry of both gradients
    is one entry of G times one factor.  A label's entry of G takes part unrounded, so its products carry
    half a step of bf16, the others' half a step of G besides.  (z is exact; lse is off by 310 u + u |lse|, the
    exponential by 310 u, u = 2^-24, and the fp32 products and sums by 8 u.)"""
    g = torch.Generator().manual_seed(N)
    a = (torch.randn(N, generator=g) * 1.5).to(torch.bfloat16)
    b = (torch.randn(min(V, d), generator=g) * 1.5).to(torch.bfloat16)
    h, w = torch.zeros((N, d), dtype=torch.bfloat16), torch.zeros((V, d), dtype=torch.bfloat16)
    h[torch.arange(N), torch.arange(N)] = a
    w[torch.arange(len(b)), torch.arange(len(b))] = b
    y = (torch.arange(N) * 7 + 3) % 50
    gl = torch.randn(N, generator=g)
    H, W, Y, L = h.to(DEV), w.to(DEV), y.to(torch.int32).to(DEV), gl.to(DEV)
    f = sv.head_xent(H, W, Y)
    out = sv.head_xent_backward(H, W, Y, f["lse"], L)
    torch.cuda.synchronize()
    z = np.zeros((N, V))
    z[np.arange(N), np.arange(N)] = _np(a) * _np(b)[:N]
    lse = np.log(np.exp(z).sum(1, keepdims=True))
    p, hot = np.exp(z - lse), np.eye(V)[y.numpy()]
    G, scale = (p - hot) * _np(gl)[:, None], np.abs(_np(gl))[:, None]
    e32 = p * scale * U * (620 + 2 * np.abs(lse)) + 8 * U * np.abs(G)
    half = 2.0 ** -8 * (1 + 2 ** -10)
    rounded = _np(torch.from_numpy(G).to(torch.bfloat16))
    n = len(b)
    for name, got, x, e, k, label in (
            ("grad_hidden", _np(out["grad_hidden"])[:, :n], G[:, :n], e32[:, :n], _np(b)[None], hot[:, :n]),
            ("grad_weight", _np(out["grad_weight"])[:, :N], G.T, e32.T, _np(a)[None], hot.T)):
        want, label = x * k, label.astype(bool)
        once = e * np.abs(k) + half * np.abs(want) + 1e-37
        err = np.abs(got - want)
        assert (err <= once + ~label * half * np.abs(want)).all(), name
        # the bound tells them apart: of the label's entries, G rounded before the product passes it
        twice = _np(torch.from_numpy((rounded[:, :n] if name == "grad_hidden" else rounded.T) * k).to(torch.bfloat16))
        assert (np.abs(twice - want) > once)[label].any(), name
    assert not _np(out["grad_hidden"])[:, n:].any() and not _np(out["grad_weight"])[:, N:].any()


@pytest.mark.parametrize("mode", ["kl", "tv"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradients_against_differences(sv, mode, tail):
    """Central differences of step e = 2^-4 on rows where teacher and draft stand well apart, so that no p = q lies
    within a step and the entries looked at are several times the difference's own error: the losses are off by
    400 u each (u = 2^-24), so the quotient by 400 u / e, and by e^2 / 6 times a third derivative, at most
    1 / (8 T^3) of a sum of probabilities, 1 / (10 T^3) of a logarithm of one and, with a tail, of a second."""
    B, G, V, K, e = 3, 2, 40, 6, 2.0 ** -4
    rng = np.random.default_rng(5)
    d = np.zeros((B, G, V), dtype=np.float32)
    ids = np.zeros((B, G, K), dtype=np.int32)
    vals = np.tile(np.arange(4.0, 1.0, -0.5, dtype=np.float32), (B, G, 1))
    far = np.zeros((B, G), dtype=np.int64)
    for i in range(B):
        for k in range(G):
            at = rng.permutation(V)
            ids[i, k], far[i, k] = at[:K], at[K]
            d[i, k, at[:K]] = vals[i, k, ::-1]      # the list's logits the other way round
            d[i, k, at[K]] = 2.5                    # and a token outside it
    T = np.array([0.75, 1.0, 1.25], dtype=np.float32)
    lse = np.log(np.exp(vals / T[:, None, None].astype(np.float64)).sum(2)) + 0.1
    c = lambda x: torch.from_numpy(x).to(DEV)
    D, ID, VA, TE, W = c(d), c(ids), c(vals), c(T), torch.ones((B, G), device=DEV)
    LS = c(lse.astype(np.float32)) if tail else None
    m = sv.SPEC_DISTILL_KL if mode == "kl" else sv.SPEC_DISTILL_TV
    f = sv.distill_loss(D, ID, VA, LS, m, None, TE)
    grad = _np(sv.distill_loss_backward(D, ID, VA, f["saved"], W, m, TE))
    loss = lambda x: sv.distill_loss(x, ID, VA, LS, m, None, TE)["loss"]
    seen = 0
    same = np.ones((B, G), dtype=bool)
    for j in range(K + 1):
        at = c(np.concatenate([ids, far[..., None].astype(np.int32)], 2)[..., j:j + 1].astype(np.int64))
        x, y = (D.scatter_add(2, at, torch.full(at.shape, s * e, device=DEV)) for s in (1, -1))
        if mode == "tv":
            assert min(oracle.distill_loss(t, ID, VA, LS, "tv", None, TE)["margin"].min() for t in (x, y)) > 440 * U
            # rows whose comparisons all fall the same way on both sides (each q is monotone in between)
            sides = [_sides(t, ids, vals, lse if tail else None, T) for t in (_np(x), _np(y))]
            same = (sides[0] == sides[1]).all(axis=2)
        diff = (_np(loss(x)) - _np(loss(y))) / (2 * e)
        g = np.take_along_axis(grad, at.cpu().numpy(), 2)[..., 0]
        third = (0.125 if mode == "tv" else 0.2) / T[:, None].astype(np.float64) ** 3
        tol = 400 * U * (1 + np.abs(_np(f["loss"]))) / e + e * e / 6 * third + 1e-6
        assert (np.abs(diff - g) <= tol)[same].all(), (j, np.abs(diff - g).max())
        seen += (np.abs(g) > 8 * tol)[same].sum()
    assert seen >= 3 * B * G, seen


def _sides(x, ids, vals, lse, T):
    t = T[:, None, None].astype(np.float64)
    q = np.exp(x / t)
    q /= q.sum(2, keepdims=True)
    p = np.exp(vals / t)
    p /= p.sum(2, keepdims=True) if lse is None else np.exp(lse)[..., None]
    s = np.take_along_axis(q, ids.astype(np.int64), 2)
    return np.concatenate([p > s, (1 - p.sum(2, keepdims=True)) > (1 - s.sum(2, keepdims=True))], 2)


def test_losses_from_an_autograd_function(sv):
    """As documented: the calls come back detached where an input requires a gradient, and train through a
    torch.autograd.Function that makes both of them."""
    class Xent(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w, y):
            o = sv.head_xent(h, w, y)
            ctx.save_for_backward(h, w, y, o["lse"])
            return o["loss"]

        @staticmethod
        def backward(ctx, g):
            h, w, y, lse = ctx.saved_tensors
            o = sv.head_xent_backward(h, w, y, lse, g.contiguous())
            return o["grad_hidden"], o["grad_weight"], None

    class Distill(torch.autograd.Function):
        @staticmethod
        def forward(ctx, d, ids, vals):
            o = sv.distill_loss(d, ids, vals)
            ctx.save_for_backward(d, ids, vals, o["saved"])
            return o["loss"]

        @staticmethod
        def backward(ctx, g):
            d, ids, vals, saved = ctx.saved_tensors
            return sv.distill_loss_backward(d, ids, vals, saved, g.contiguous()), None, None

    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    h = torch.randn((30, 64), generator=g, device=DEV, requires_grad=True)
    w = torch.randn((400, 64), generator=g, device=DEV, requires_grad=True)
    y = torch.randint(400, (30,), generator=g, device=DEV).to(torch.int32)
    d = torch.randn((2, 3, 500), generator=g, device=DEV, requires_grad=True)
    t = sv.teacher_topk(torch.randn((2, 4, 500), generator=g, device=DEV), 8)
    o, f = sv.head_xent(h, w, y), sv.distill_loss(d, t["ids"], t["values"])
    assert not any(x.requires_grad for x in (*o.values(), *f.values()))
    c, e = torch.rand((30,), generator=g, device=DEV), torch.rand((2, 3), generator=g, device=DEV)
    ((Xent.apply(h, w, y) * c).sum() + (Distill.apply(d, t["ids"], t["values"]) * e).sum()).backward()
    b = sv.head_xent_backward(h, w, y, o["lse"], c)
    torch.cuda.synchronize()
    assert torch.equal(h.grad, b["grad_hidden"]) and torch.equal(w.grad, b["grad_weight"])
    assert torch.equal(d.grad, sv.distill_loss_backward(d, t["ids"], t["values"], f["saved"], e))
    assert not b["grad_hidden"].requires_grad


def test_head_fp32_sums_of_long_rows(sv):
    """Sums of equal terms, whose roundings all fall the same way.  A product is rounded 256 times at most in its
    block and once per block of 256 (and once as a product): 256 + k / 256 + 2 roundings, not k."""
    g = torch.Generator().manual_seed(3)
    N, V, d = 64, 40, 16384
    a, b = torch.rand(N, generator=g) + 0.5, (torch.rand(V, generator=g) - 0.3) * (3.0 / d)
    h, w = a[:, None].repeat(1, d).contiguous().to(DEV), b[:, None].repeat(1, d).contiguous().to(DEV)
    y = (torch.arange(N) % V).to(torch.int32).to(DEV)
    o = sv.head_xent(h, w, y)
    torch.cuda.synchronize()
    z = d * np.outer(_np(a), _np(b))
    lse = np.log(np.exp(z).sum(1))
    loss = lse - z[np.arange(N), np.arange(N) % V]
    dz = (256 + d / 256 + 2) * U * np.abs(z).max(1)
    assert (np.abs(_np(o["lse"]) - lse) <= dz + U * (310 + np.abs(lse))).all()
    assert (np.abs(_np(o["loss"]) - loss) <= 2 * dz + U * (310 + np.abs(lse) + np.abs(loss))).all()
    # grad_weight: as many equal rows
    N, V, d = 8192, 6, 8
    a, b = torch.rand(d, generator=g) + 0.5, torch.randn((V, d), generator=g)
    h, w = a.repeat(N, 1).contiguous().to(DEV), b.to(DEV)
    y = torch.full((N,), 2, dtype=torch.int32, device=DEV)
    gl = torch.full((N,), 0.7, device=DEV)
    o = sv.head_xent(h, w, y)
    gw = sv.head_xent_backward(h, w, y, o["lse"], gl, need_hidden=False)["grad_weight"]
    torch.cuda.synchronize()
    z = _np(b) @ _np(a)
    lse = np.log(np.exp(z).sum())
    p = np.exp(z - lse)
    G = p.copy()
    G[2] -= 1.0
    G *= float(gl[0])
    want = N * np.outer(G, _np(a))
    dz = (d + 2) * U * (np.abs(_np(b)) @ np.abs(_np(a)))
    eG = p * 0.7 * (2 * dz + dz.max() + U * (620 + np.abs(lse))) * 1.01 + 4 * U * np.abs(G)
    tol = N * np.outer(eG, _np(a)) + (256 + N / 256 + 2) * U * np.abs(want)
    assert (np.abs(_np(gw) - want) <= tol).all()
