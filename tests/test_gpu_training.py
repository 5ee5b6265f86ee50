"""GPU parity of the drafter's training operators with the fp64 oracle.

Tolerances (u = 2^-24, half a step of fp32):
  exponentials and sums: a term exp((z - m) / T) carries at most 1 ulp (2 u) of exp2 and 3 u x of its
    exponent, x = |z - m| / T (a rounded difference or scale, and one multiply-add); a thread adds its
    vectors in pairs (3 levels) and at most 40 of them and a scalar one after the other in fp32, a term's
    sum is rounded at most 44 < 65 times, and the rest is fp64.  The sum is off by at most
    u (65 + 2 + 3 E[x]) relative, and E[x] <= ln V + 1 over a softmax of V terms: u (67 + 3 * 14.2) < 110 u
    for every V <= 2^19 + 1.
  lse: 110 u + u |lse| for the final rounding.
  distillation losses: they depend on sums over the row through one normaliser and the tail's
    logarithm, each weighed by at most 1: 220 u + u |loss|; 400 u covers both and the margins of the
    fp64 list terms.
  distillation gradient: q b - c with q off by 110 u relative (3 u x of its own exponent: x e^-x <= 0.37,
    so 1.2 u absolute is covered by q's factor below where x is small and by q itself where x is large:
    x <= 104 before q is 0 in fp32, 312 u), a and b off by 220 u: 700 u q |g| / T, plus half a step of the
    storage type.
  head logits: products of d terms in fp32: dz = (d + 2) u sum_k |h_k w_k| bounds every order.
    lse: max dz + (256 + 2 + 6 + 3 * 14.2) u (a strip adds at most 128 * 2 terms in fp32, and its sum is
    scaled at most 3 times on its way to the row's, the exponents of all adding up to x) < max dz + 310 u,
    + u |lse|.  G: p (2 dz + dlse + 310 u) |g| + half a step of the type times |G| (its rounding for the
    product); the products' sums: |G| |W| (terms + 16) u, and half a step for the result.
"""

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


def _dist_inputs(seed, B, G, V, dtype, ragged=True, masked=0.0):
    rng = np.random.default_rng(seed)
    t = torch.from_numpy(rng.normal(0, 2.5, (B, G + 1, V)).astype(np.float32))
    t.scatter_add_(2, torch.from_numpy(rng.integers(0, V, (B, G + 1, 1))), torch.full((B, G + 1, 1), 6.0))
    d = t[:, :G] + torch.from_numpy(rng.normal(0, 0.6, (B, G, V)).astype(np.float32))
    if masked:
        m = torch.from_numpy(rng.random((B, 1, V)) < masked)
        m[:, :, 0] = False
        t[m.expand_as(t)] = -np.inf
        d[m.expand_as(d)] = -np.inf
    L = torch.from_numpy(rng.integers(0, G + 1, B).astype(np.int32)) if ragged else None
    T = torch.from_numpy(rng.uniform(0.6, 1.4, B).astype(np.float32))
    w = torch.from_numpy(rng.normal(0, 1, (B, G)).astype(np.float32))
    c = lambda x: None if x is None else x.to(DEV)
    return c(t.to(DT[dtype])), c(d.to(DT[dtype])), c(L), c(T), c(w)


def _check_teacher(got, ref):
    assert (_np(got["status"]) == ref["status"]).all()
    assert (_np(got["ids"]) == ref["ids"]).all()
    assert np.array_equal(_np(got["values"]), ref["values"], equal_nan=True)
    l, r = _np(got["lse"]), ref["lse"]
    fin = np.isfinite(r)
    assert np.array_equal(l[~fin], r[~fin], equal_nan=True)
    err = np.abs(l[fin] - r[fin])
    assert (err <= U * (110 + np.abs(r[fin]))).all(), err.max()


SHAPES = [(1, 1, 1), (2, 3, 5), (3, 2, 15), (2, 4, 64), (4, 3, 257), (1, 4, 1000), (2, 2, 3001), (2, 2, 4097),
          (2, 2, 20011), (2, 1, 32768), (1, 2, 32783), (2, 2, 151936), (1, 1, 262143)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_teacher_topk(sv, shape, dtype):
    B, G, V = shape
    t, _, L, T, _ = _dist_inputs(V, B, G, V, dtype, ragged=B > 1)
    for K in (1, 8, 64, 256):
        print(f"teacher {shape} {dtype} K={K}", flush=True)
        got = sv.teacher_topk(t, K, L, T)
        torch.cuda.synchronize()
        _check_teacher(got, oracle.teacher_topk(t, K, L, T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "few", "rising", "falling", "masked", "one", "zeros"])
def test_teacher_topk_of_ties_and_orders(sv, kind, dtype):
    """Rows whose values make the segment's bound useless (ties, sorted rows) or nearly empty."""
    B, G, V = 2, 2, 40007
    rng = np.random.default_rng(5)
    z = np.zeros((B, G + 1, V), dtype=np.float32)
    if kind == "two":
        z[..., rng.integers(0, V, 300)] = 1.0
    elif kind == "few":
        z[:] = rng.integers(-3, 4, z.shape)
    elif kind == "rising":
        z[:] = np.arange(V) / 64.0
    elif kind == "falling":
        z[:] = -np.arange(V) / 64.0
    elif kind == "masked":
        z[:] = -np.inf
        z[..., ::97] = rng.normal(0, 1, z[..., ::97].shape)
    elif kind == "one":
        z[:] = -np.inf
        z[..., V - 1] = -5.0
    elif kind == "zeros":
        z[..., ::2] = -0.0
    t = torch.from_numpy(z).to(DT[dtype]).to(DEV)
    for K in (1, 50, 256):
        print(f"teacher {kind} {dtype} K={K}", flush=True)
        got = sv.teacher_topk(t, K)
        torch.cuda.synchronize()
        _check_teacher(got, oracle.teacher_topk(t, K))


def test_teacher_topk_status(sv):
    t, _, _, T, _ = _dist_inputs(9, 9, 3, 9001, "f32", ragged=False)
    L = torch.tensor([3, 2, 0, 3, 3, 4, -1, 3, 2], dtype=torch.int32, device=DEV)
    t[0, 2, 9000] = float("nan")
    t[1, 2, 5] = float("nan")          # past the length: not read
    t[2] = float("nan")                # length 0: not read
    t[3, 1, 4444] = float("inf")
    t[4, 0] = -float("inf")
    T[7] = 0.0
    T[8] = float("nan")
    got = sv.teacher_topk(t, 20, L, T)
    torch.cuda.synchronize()
    ref = oracle.teacher_topk(t, 20, L, T)
    assert ref["status"].tolist() == [4, 0, 0, 4, 4, 8, 8, 2, 2]
    _check_teacher(got, ref)


def _check_distill(sv, draft, ids, vals, tlse, mode, L, T, w, in_place=False, far_tail=False):
    name = "kl" if mode == sv.SPEC_DISTILL_KL else "tv"
    ref = oracle.distill_loss(draft, ids, vals, tlse, name, L, T, w)
    # no pair so near p = q that rounding could pick the other side: q is off by 110 u, r_s (one sum
    # over another) by 220 u.  (Of one token, p = q = 1: q b - c is 1 - 1 or 0 - 0, 0 on either side.)
    if name == "tv" and draft.shape[2] > 1:
        assert ref["margin"].min() > 440 * U
    got = sv.distill_loss(draft, ids, vals, tlse, mode, L, T)
    keep = draft.clone()
    grad = sv.distill_loss_backward(draft, ids, vals, got["saved"], w, mode, T, in_place=in_place)
    torch.cuda.synchronize()
    assert in_place or torch.equal(keep.view(torch.uint8), draft.view(torch.uint8))
    assert (_np(got["status"]) == ref["status"]).all(), (_np(got["status"]), ref["status"])
    l, r = _np(got["loss"]), ref["loss"]
    fin = np.isfinite(r)
    assert np.array_equal(l[~fin], r[~fin], equal_nan=True)
    err = np.abs(l[fin] - r[fin])
    assert (err <= U * (400 + np.abs(r[fin]))).all(), err.max()
    Td = np.ones(draft.shape[0]) if T is None else _np(T)
    with np.errstate(invalid="ignore", divide="ignore"):
        scale = np.where(np.isfinite(Td) & (Td > 0), np.abs(_np(w)).T / Td, 0.0).T[..., None]
    eps = torch.finfo(draft.dtype).eps
    tol = 700 * U * ref["q"] * scale + eps / 2 * (1 + 2 ** -10) * np.abs(ref["grad"]) + 1e-37
    if far_tail:
        # r_t large beside r_s: outside the list the gradient is (q / r_s) (b r_s - r_t), its second factor
        # fp64 and no longer about r_s.  q / r_s is off by 110 u (its sum) and 3 u x, x <= 104 before it is
        # 0 in fp32: 422 u < 700 u of the gradient.
        outside = torch.ones(draft.shape, dtype=torch.bool)
        outside.scatter_(2, ids.cpu().long(), False)
        tol += 700 * U * np.abs(ref["grad"]) * outside.numpy()
    err = np.abs(_np(grad) - ref["grad"])
    assert (err <= tol).all(), (np.argwhere(err > tol)[:5], err.max())
    return got, grad, ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_distill_loss_and_gradient(sv, shape, dtype):
    B, G, V = shape
    t, d, L, T, w = _dist_inputs(V + 1, B, G, V, dtype, ragged=B > 1)
    for K, mode, tail in ((1, 0, True), (7, 1, False), (64, 0, False), (256, 1, True), (200, 0, True)):
        print(f"distill {shape} {dtype} K={K} mode={mode} tail={tail}", flush=True)
        o = sv.teacher_topk(t, K, L, T)
        _check_distill(sv, d.clone(), o["ids"], o["values"], o["lse"] if tail else None, mode, L, T, w,
                       in_place=mode == 1)


@pytest.mark.parametrize("mode", [0, 1])
def test_distill_masked_vocabulary(sv, mode):
    """Both sides mask four fifths of the vocabulary with -inf."""
    t, d, L, T, w = _dist_inputs(77, 3, 3, 5003, "bf16", masked=0.8)
    o = sv.teacher_topk(t, 40, L, T)
    _, grad, _ = _check_distill(sv, d, o["ids"], o["values"], o["lse"], mode, L, T, w)
    assert (grad[torch.isinf(d)] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_far_tail(sv, dtype):
    """The draft puts nearly nothing outside the list (down to exp(-200) of it): the tail's mass is
    summed on its own, so its logarithm and the gradient's share stay exact."""
    B, G, V, K = 3, 2, 4099, 16
    rng = np.random.default_rng(3)
    d = rng.normal(0, 1, (B, G, V)).astype(np.float32)
    ids = np.stack([[rng.permutation(V)[:K] for _ in range(G)] for _ in range(B)]).astype(np.int32)
    for i, lift in enumerate((10.0, 60.0, 200.0)):
        for k in range(G):
            d[i, k, ids[i, k]] += lift
    vals = rng.normal(0, 1, (B, G, K)).astype(np.float32)
    c = lambda x: torch.from_numpy(x).to(DEV)
    d = c(d).to(DT[dtype])
    lse = torch.logsumexp(c(vals).double(), 2).float() + 0.25     # a tail of 1 - e^-0.25
    w = c(rng.normal(0, 1, (B, G)).astype(np.float32))
    B_ids, B_vals = c(ids), c(vals)
    ref = oracle.distill_loss(d, B_ids, B_vals, lse, "kl", None, None, w)
    got = sv.distill_loss(d, B_ids, B_vals, lse)
    grad = sv.distill_loss_backward(d, B_ids, B_vals, got["saved"], w)
    torch.cuda.synchronize()
    assert (np.abs(_np(got["loss"]) - ref["loss"]) <= U * (400 + np.abs(ref["loss"]))).all()
    # outside the list the gradient is -r_t times a softmax over the outside tokens, exact to 700 u of it
    eps = torch.finfo(DT[dtype]).eps
    err = np.abs(_np(grad) - ref["grad"])
    assert (err <= (700 * U + eps / 2 * (1 + 2 ** -10)) * np.abs(ref["grad"]) + 1e-37 +
            700 * U * ref["q"] * np.abs(_np(w))[..., None]).all()


def test_distill_status_and_empty_rows(sv):
    t, d, _, T, w = _dist_inputs(11, 12, 3, 20011, "bf16", ragged=False)
    o = sv.teacher_topk(t, 30, None, T)
    ids, vals, lse = o["ids"].clone(), o["values"].clone(), o["lse"].clone()
    L = torch.tensor([3, 3, 3, 3, 3, 3, 2, 3, 4, 3, 3, 0], dtype=torch.int32, device=DEV)
    ids[0, 1] = -1                     # a row without an entry: not read
    d[0, 1, 100] = float("nan")
    vals[1, 0] = -float("inf")         # the same, named but without mass
    ids[2, 2, 5] = 20011
    ids[3, 0, 29] = -2
    ids[4, 1, 7] = ids[4, 1, 3]
    vals[5, 1, 2] = float("nan")
    d[6, 2] = float("nan")             # past the length
    d[7, 0, 20010] = float("inf")
    T[9] = 0.0
    d[10, 1] = -float("inf")
    for mode in (0, 1):
        _, _, ref = _check_distill(sv, d, ids, vals, None, mode, L, T, w)
        assert ref["status"].tolist() == [0, 0, 1, 1, 256, 4, 0, 4, 8, 2, 4, 0]
    lse[11, 0] = float("nan")          # length 0: not looked at
    lse[0, 1] = float("nan")           # the row without an entry
    lse[6, 1] = float("inf")
    _, _, ref = _check_distill(sv, d, ids, vals, lse, 0, L, T, w)
    assert ref["status"].tolist() == [0, 0, 1, 1, 256, 4, 4, 4, 8, 2, 4, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_walked_whole(sv, dtype):
    """Rows of several chunks, one workgroup each (512 rows or more): values that rise with the token id
    (each chunk's bound is passed by the next one's), ties, and ordinary rows."""
    B, G, V = 64, 8, 50021
    t, d, L, T, w = _dist_inputs(71, B, G, V, dtype)
    t[0] = (torch.arange(V, device=DEV) / 64.0).to(t.dtype)
    t[1] = 1.5
    t[2] = torch.where(torch.arange(V, device=DEV) % 7 == 0, 2.0, -1.0).to(t.dtype)
    t[3] = -float("inf")
    t[3, :, V - 1] = 0.25
    t[4, :, V // 2:] += 200.0        # past the first chunk's reference by more than fp32 holds
    d[4, :, V // 2:] += 200.0
    L[:5] = torch.tensor([8, 3, 5, 8, 8], dtype=torch.int32)
    for K, tail in ((16, True), (256, False)):
        print(f"whole rows {dtype} K={K}", flush=True)
        o = sv.teacher_topk(t, K, L, T)
        torch.cuda.synchronize()
        _check_teacher(o, oracle.teacher_topk(t, K, L, T))
        _check_distill(sv, d, o["ids"], o["values"], o["lse"] if tail else None, 0, L, T, w)


def test_many_requests_with_lengths(sv):
    """Up to 4096 requests the live rows are found by a prefix sum, beyond that rows keep their places."""
    for B in (513, 4096, 4097):
        t, d, L, T, w = _dist_inputs(B, B, 2, 130, "bf16")
        L[5], T[7] = 3, 0.0
        print(f"requests {B}", flush=True)
        o = sv.teacher_topk(t, 9, L, T)
        torch.cuda.synchronize()
        _check_teacher(o, oracle.teacher_topk(t, 9, L, T))
        _check_distill(sv, d, o["ids"], o["values"], None, 0, L, T, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_of_the_lowest_value(sv, dtype):
    """Masked tokens at the type's lowest finite value have no mass; a row of nothing else is uniform."""
    low = torch.finfo(DT[dtype]).min
    t, d, L, T, w = _dist_inputs(81, 4, 3, 9001, dtype, ragged=False)
    m = torch.arange(9001, device=DEV) % 3 != 0
    t[:, :, m] = low
    d[:, :, m] = low
    t[2, 1], d[2, 1] = low, low
    T[2] = 1.25                      # low / T is finite
    for K in (20, 256):
        print(f"lowest {dtype} K={K}", flush=True)
        o = sv.teacher_topk(t, K, L, T)
        torch.cuda.synchronize()
        _check_teacher(o, oracle.teacher_topk(t, K, L, T))
        _check_distill(sv, d, o["ids"], o["values"], None, 0, L, T, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_temperatures(sv, dtype):
    """Temperatures towards 0 (the argmax) and towards infinity (uniform).  (KL: at both ends p = q.)"""
    t, d, _, T, w = _dist_inputs(83, 5, 2, 4099, dtype, ragged=False)
    T = torch.tensor([1e-30, 1e-4, 1e-2, 1e4, 1e30], device=DEV)
    o = sv.teacher_topk(t, 33, None, T)
    torch.cuda.synchronize()
    _check_teacher(o, oracle.teacher_topk(t, 33, None, T))
    _check_distill(sv, d, o["ids"], o["values"], None, 0, None, T, w)
    c = slice(1, 4)
    _check_distill(sv, d[c].clone(), o["ids"][c].clone(), o["values"][c].clone(),
                   o["lse"][c].clone(), 0, None, T[c].clone(), w[c].clone(), far_tail=True)


def test_offsets_past_32_bits(sv):
    """Logits of more than 4 GiB: the last request's rows, behind requests without work."""
    B, G, V = 130, 64, 262143
    lt, ld, _, _, lw = _dist_inputs(91, 1, G, V, "bf16", ragged=False)
    t = torch.zeros((B, G + 1, V), dtype=torch.bfloat16, device=DEV)
    d = torch.zeros((B, G, V), dtype=torch.bfloat16, device=DEV)
    t[-1], d[-1] = lt[0], ld[0]
    assert t.numel() * 2 > 2 ** 32 and d.numel() * 2 > 2 ** 32
    L = torch.zeros(B, dtype=torch.int32, device=DEV)
    L[-1] = 5
    w = lw.expand(B, G).contiguous()
    print("past 32 bits", flush=True)
    o = sv.teacher_topk(t, 12, L)
    f = sv.distill_loss(d, o["ids"], o["values"], o["lse"], 0, L)
    g = sv.distill_loss_backward(d, o["ids"], o["values"], f["saved"], w)
    torch.cuda.synchronize()
    one = {k: v[-1:] for k, v in o.items()}
    _check_teacher(one, oracle.teacher_topk(lt, 12, L[-1:], None))
    assert (o["ids"][:-1] == -1).all() and (f["loss"][:-1] == 0).all()
    ref = oracle.distill_loss(ld, one["ids"], one["values"], one["lse"], "kl", L[-1:], None, lw)
    assert (np.abs(_np(f["loss"][-1:]) - ref["loss"]) <= U * (400 + np.abs(ref["loss"]))).all()
    tol = 700 * U * ref["q"] * np.abs(_np(lw))[..., None] + 2.0 ** -8 * (1 + 2 ** -10) * np.abs(ref["grad"]) + 1e-37
    assert (np.abs(_np(g[-1:]) - ref["grad"]) <= tol).all()
    assert not g[:-1].any()


def test_distill_list_in_any_order_and_unused_entries(sv):
    """The list may come in any order with unused entries in between: the loss and gradient are those
    of the sorted list (the list terms are summed in fp64 in another order: 64 terms of 2^-53)."""
    t, d, L, T, w = _dist_inputs(13, 3, 4, 10007, "f32")
    o = sv.teacher_topk(t, 40, L, T)
    perm = torch.randperm(64, generator=torch.Generator().manual_seed(1)).to(DEV)
    ids = torch.nn.functional.pad(o["ids"], (0, 24), value=-1)[..., perm].contiguous()
    vals = torch.nn.functional.pad(o["values"], (0, 24), value=float("nan"))[..., perm].contiguous()
    for mode in (0, 1):
        a = sv.distill_loss(d, o["ids"], o["values"], o["lse"], mode, L, T)
        b = sv.distill_loss(d, ids, vals, o["lse"], mode, L, T)
        ga = sv.distill_loss_backward(d, o["ids"], o["values"], a["saved"], w, mode, T)
        gb = sv.distill_loss_backward(d, ids, vals, b["saved"], w, mode, T)
        torch.cuda.synchronize()
        assert torch.allclose(a["loss"], b["loss"], rtol=4 * U, atol=2.0 ** -40)
        assert torch.allclose(ga, gb, rtol=4 * U, atol=2.0 ** -40)


def _head_inputs(seed, N, V, d, dtype, ignored=0.1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.randn((N, d), generator=g, device=DEV).to(DT[dtype])
    w = (torch.randn((V, d), generator=g, device=DEV) * (3.0 / d ** 0.5)).to(DT[dtype])
    y = torch.randint(V, (N,), generator=g, device=DEV)
    y[torch.rand((N,), generator=g, device=DEV) < ignored] = -1
    return h, w, y.to(torch.int32), torch.randn((N,), generator=g, device=DEV)


def _check_head(sv, h, w, y, gl):
    got = sv.head_xent(h, w, y)
    b = sv.head_xent_backward(h, w, y, got["lse"], gl)
    torch.cuda.synchronize()
    ref = oracle.head_xent(h, w, y, gl)
    H, W = _np(h), _np(w)
    N, d = H.shape
    V = W.shape[0]
    eps = torch.finfo(h.dtype).eps
    assert (_np(got["status"]) == ref["status"]).all()
    rows = np.flatnonzero((ref["status"] == 0) & ~np.isnan(ref["lse"]))
    assert (np.isnan(_np(got["lse"])) == np.isnan(ref["lse"])).all()
    assert np.isnan(_np(got["loss"])[ref["status"] != 0]).all()
    dz = np.zeros((N, V))
    fin = np.flatnonzero(np.isfinite(H).all(axis=1))
    dz[fin] = (d + 2) * U * (np.abs(H[fin]) @ np.abs(W).T)
    dlse = dz.max(axis=1) + 310 * U + U * np.abs(np.nan_to_num(ref["lse"]))
    assert (np.abs(_np(got["lse"]) - ref["lse"])[rows] <= dlse[rows]).all()
    err = np.abs(_np(got["loss"]) - ref["loss"])[rows]
    assert (err <= (dlse + dz.max(axis=1))[rows] + U * np.abs(ref["loss"][rows])).all()
    G, p = np.abs(ref["g"]), ref["p"] * np.abs(_np(gl))[:, None]
    eG = p * (2 * dz + dlse[:, None] + 310 * U) * 1.01 + (eps / 2 * 1.01 + 4 * U) * G + 1e-38
    eG[ref["g"].any(axis=1) == 0] = 0.0
    live = G.any(axis=1)
    Hs = np.where(live[:, None], np.abs(np.nan_to_num(H, posinf=0, neginf=0)), 0.0)
    th = eG @ np.abs(W) + (V + 16) * U * (G @ np.abs(W)) + eps / 2 * 1.01 * np.abs(ref["grad_hidden"]) + 1e-37
    tw = eG.T @ Hs + (N + 16) * U * (G.T @ Hs) + eps / 2 * 1.01 * np.abs(ref["grad_weight"]) + 1e-37
    for name, tol in (("grad_hidden", th), ("grad_weight", tw)):
        err = np.abs(_np(b[name]) - ref[name])
        assert (err <= tol).all(), (name, np.argwhere(~(err <= tol))[:5], np.nanmax(err))
    return got, b, ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(1, 1, 8), (1, 7, 16), (3, 257, 8), (5, 100, 72), (16, 1000, 256), (63, 129, 264),
                                   (64, 5000, 64), (65, 255, 136), (129, 1025, 128), (300, 3001, 40),
                                   (257, 513, 1000), (1, 20011, 512), (130, 256, 24), (348, 717, 3064),
                                   (200, 3000, 640)])
def test_head_xent(sv, N, V, d, dtype):
    print(f"head {N} {V} {d} {dtype}", flush=True)
    _check_head(sv, *_head_inputs(N + V + d, N, V, d, dtype))


@pytest.mark.parametrize("dtype,N,V,d", [("bf16", 1025, 16500, 1000), ("f32", 1030, 16600, 500),
                                         ("bf16", 1025, 70001, 64)])
def test_head_xent_large_tiles_and_pieces(sv, dtype, N, V, d):
    """The 256 x 256 tiles of every product, and (the last) a vocabulary in two pieces."""
    print(f"head {N} {V} {d} {dtype}", flush=True)
    _check_head(sv, *_head_inputs(4, N, V, d, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_xent_bad_rows(sv, dtype):
    """Bad labels, rows left out and rows with no finite normaliser add nothing to the gradients, also
    where their hidden states are infinite."""
    h, w, y, gl = _head_inputs(21, 140, 700, 64, dtype)
    y[0], y[1], y[2], y[3] = 700, -2, -1, 5
    h[2] = float("inf")
    h[3, 7] = float("nan")
    h[4] = float("inf")
    y[4] = 3
    got, b, ref = _check_head(sv, h, w, y, gl)
    assert ref["status"][:5].tolist() == [1, 1, 0, 4, 4]
    assert (b["grad_hidden"][:5] == 0).all() and torch.isfinite(b["grad_weight"]).all()
    y[:] = -1
    got = sv.head_xent(h, w, y)
    b = sv.head_xent_backward(h, w, y, got["lse"], gl)
    torch.cuda.synchronize()
    assert (got["loss"] == 0).all() and (got["status"] == 0).all()
    assert (b["grad_hidden"] == 0).all() and (b["grad_weight"] == 0).all()


def test_head_xent_one_gradient_only(sv):
    h, w, y, gl = _head_inputs(22, 200, 900, 128, "bf16")
    lse = sv.head_xent(h, w, y)["lse"]
    both = sv.head_xent_backward(h, w, y, lse, gl)
    a = sv.head_xent_backward(h, w, y, lse, gl, need_weight=False)
    b = sv.head_xent_backward(h, w, y, lse, gl, need_hidden=False)
    torch.cuda.synchronize()
    assert set(a) == {"grad_hidden"} and set(b) == {"grad_weight"}
    assert torch.equal(a["grad_hidden"], both["grad_hidden"]) and torch.equal(b["grad_weight"], both["grad_weight"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_xent_one_label_for_many_rows(sv, dtype):
    """Every row names one of two tokens: the sums of a token's row of grad_weight run over all rows."""
    h, w, y, gl = _head_inputs(23, 2100, 300, 1032, dtype)
    y[:] = 7
    y[1030:1040] = 299
    y[2050] = -1
    h[3, 5] = float("inf")
    _check_head(sv, h, w, y, gl)


@pytest.mark.parametrize("dtype,V,d", [("bf16", 300001, 16), ("f32", 5001, 8200), ("f32", 40001, 1000)])
def test_head_xent_pieces_for_one_gradient(sv, dtype, V, d):
    """A vocabulary in pieces for few rows, and each gradient alone."""
    print(f"head pieces {V} {d} {dtype}", flush=True)
    h, w, y, gl = _head_inputs(24, 5, V, d, dtype)
    y[:3] = torch.tensor([V - 1, 0, V // 2])
    _, both, _ = _check_head(sv, h, w, y, gl)
    lse = sv.head_xent(h, w, y)["lse"]
    a = sv.head_xent_backward(h, w, y, lse, gl, need_weight=False)
    b = sv.head_xent_backward(h, w, y, lse, gl, need_hidden=False)
    torch.cuda.synchronize()
    assert torch.equal(a["grad_hidden"], both["grad_hidden"]) and torch.equal(b["grad_weight"], both["grad_weight"])


def test_head_xent_offsets_past_32_bits(sv):
    """A head of more than 4 GiB, zero but for a few rows: with z = 0 for V - 3 tokens the loss, lse and
    gradients follow in closed form.  The rows hold small integers times powers of two, so the logits are
    exact (no rounding in fp32) and only the softmax rounds."""
    N, V, d = 3, 262143, 16384
    W = torch.zeros((V, d), dtype=torch.bfloat16, device=DEV)
    h = torch.zeros((N, d), dtype=torch.bfloat16, device=DEV)
    assert W.numel() * 2 > 2 ** 32
    toks = [0, V - 2, V - 1]
    for n, v in enumerate(toks):
        W[v, n::4] = 0.5
        h[n, n::4] = 2.0 ** -8
        h[n, (n + 1) % 3::4] = 2.0 ** -9
    y = torch.tensor([V - 1, V - 2, V - 1], dtype=torch.int32, device=DEV)
    gl = torch.tensor([1.0, -0.5, 2.0], device=DEV)
    print("head past 32 bits", flush=True)
    got = sv.head_xent(h, W, y)
    b = sv.head_xent_backward(h, W, y, got["lse"], gl)
    torch.cuda.synchronize()
    H, Z = _np(h), np.zeros((N, 3))
    Ws = _np(W[toks])
    Z = H @ Ws.T
    lse = np.log(np.exp(Z).sum(1) + (V - 3))
    p = np.exp(Z - lse[:, None])
    hot = np.array([[int(y[n]) == v for v in toks] for n in range(N)], dtype=float)
    assert (np.abs(_np(got["lse"]) - lse) <= U * (310 + lse)).all()
    assert (np.abs(_np(got["loss"]) - (lse - (Z * hot).sum(1))) <= U * (310 + 2 * lse + np.abs(Z).max())).all()
    Gm = (p - hot) * _np(gl)[:, None]
    # G: p off by (dlse + 310 u) of itself, half a step of bf16 in the product; half a step for the result
    eG = (620 + lse.max()) * U * p * np.abs(_np(gl))[:, None] * 1.01 + (2.0 ** -8 * 1.01 + 4 * U) * np.abs(Gm)
    gh, gw = Gm @ Ws, Gm.T @ H
    th = eG @ np.abs(Ws) + 2.0 ** -8 * 1.01 * np.abs(gh) + 16 * U * (np.abs(Gm) @ np.abs(Ws))
    tw = eG.T @ np.abs(H) + 2.0 ** -8 * 1.01 * np.abs(gw) + 16 * U * (np.abs(Gm).T @ np.abs(H))
    assert (np.abs(_np(b["grad_hidden"]) - gh) <= th).all()
    assert (np.abs(_np(b["grad_weight"][toks]) - gw) <= tw).all()
    # every other token: p0 = 1 / sum of the row, the same row for all of them
    g0 = (np.exp(-lse) * _np(gl)) @ H
    rest = b["grad_weight"][1:V - 2]
    assert torch.equal(rest.min(0).values, rest.max(0).values)
    t0 = (np.exp(-lse) * np.abs(_np(gl))) @ np.abs(H) * (2.0 ** -8 * 1.01 + 700 * U) + 2.0 ** -8 * 1.01 * np.abs(g0)
    assert (np.abs(_np(rest[0]) - g0) <= t0).all()


def test_gradients_against_differences(sv):
    """Central differences of the losses in fp32 (step e): the losses are off by at most 400 u each, so
    the quotient by 400 u / e, and by e^2 / 6 times a third derivative of at most 6 |g| / T^3."""
    t, d, _, T, w = _dist_inputs(31, 2, 2, 40, "f32", ragged=False)
    o = sv.teacher_topk(t, 6, None, T)
    e = 2.0 ** -6
    rng = np.random.default_rng(2)
    for mode in (0, 1):
        f = sv.distill_loss(d, o["ids"], o["values"], o["lse"], mode, None, T)
        grad = sv.distill_loss_backward(d, o["ids"], o["values"], f["saved"], w, mode, T)
        for _ in range(12):
            i, k, v = int(rng.integers(2)), int(rng.integers(2)), int(rng.integers(40))
            s = []
            margins = []
            for sign in (1, -1):
                x = d.clone()
                x[i, k, v] += sign * e
                s.append(float(sv.distill_loss(x, o["ids"], o["values"], o["lse"], mode, None, T)["loss"][i, k]))
                margins.append(oracle.distill_loss(x, o["ids"], o["values"], o["lse"], "tv", None, T)["margin"][i, k])
            if mode == 1 and min(margins) < 0.1:
                continue                # a kink may lie inside the step
            g, Ti = float(w[i, k]), float(T[i])
            diff = (s[0] - s[1]) / (2 * e) * g
            assert abs(diff - float(grad[i, k, v])) <= abs(g) * (400 * U / e + e * e / Ti ** 3 + 1e-6)


def test_streams_devices_and_given_buffers(sv):
    """A side stream, outputs and workspaces of the caller, and two calls at once on two streams."""
    t, d, L, T, w = _dist_inputs(41, 8, 4, 30011, "bf16")
    h, W, y, gl = _head_inputs(42, 300, 2000, 128, "bf16")

    def step(stream=None):
        o = sv.teacher_topk(t, 32, L, T, stream=stream)
        f = sv.distill_loss(d, o["ids"], o["values"], o["lse"], 0, L, T, stream=stream)
        g = sv.distill_loss_backward(d, o["ids"], o["values"], f["saved"], w, 0, T, stream=stream)
        x = sv.head_xent(h, W, y, stream=stream)
        b = sv.head_xent_backward(h, W, y, x["lse"], gl, stream=stream)
        return [o["ids"], o["lse"], f["loss"], g, x["loss"], b["grad_hidden"], b["grad_weight"]]
    ref = step()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [step(x) for x in s]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(ref, g):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    lib = sv.load_library()
    n = lib.spec_head_xent_backward_workspace_size(300, 2000, 128, 1)
    guard = torch.full((n + 512,), 7, dtype=torch.uint8, device=DEV)
    out = dict(grad_hidden=torch.empty_like(h), grad_weight=torch.empty_like(W))
    lse = sv.head_xent(h, W, y)["lse"]
    sv.head_xent_backward(h, W, y, lse, gl, out=out, workspace=guard[:n])
    torch.cuda.synchronize()
    assert (guard[n:] == 7).all()
    assert torch.equal(out["grad_hidden"], ref[5]) and torch.equal(out["grad_weight"], ref[6])
    with pytest.raises(ValueError, match="too small"):
        sv.head_xent_backward(h, W, y, lse, gl, workspace=guard[:n - 1])


def test_captured_step_replays(sv):
    """A training step on given buffers recorded into a HIP graph and replayed three times with other
    work between: every replay equals the eager step bit for bit."""
    t, d, L, T, w = _dist_inputs(51, 6, 3, 40009, "bf16")
    h, W, y, gl = _head_inputs(52, 200, 3000, 96, "bf16")
    s = torch.cuda.Stream()

    def step():
        o = sv.teacher_topk(t, 24, L, T)
        f = sv.distill_loss(d, o["ids"], o["values"], None, 1, L, T)
        g = sv.distill_loss_backward(d, o["ids"], o["values"], f["saved"], w, 1, T)
        x = sv.head_xent(h, W, y)
        b = sv.head_xent_backward(h, W, y, x["lse"], gl)
        return [o["ids"], o["values"], o["lse"], f["loss"], g, x["loss"], b["grad_hidden"], b["grad_weight"]]
    with torch.cuda.stream(s):
        ref = [x.clone() for x in step()]
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for rep in range(3):
        for x in got:
            x.fill_(-7)
        sv.head_xent(h, W, y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        print(f"graph replay {rep}", flush=True)
        for a, b in zip(ref, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_training_step_of_a_markov_drafter(sv):
    """The operators as a drafter's training uses them: the target's rows become lists once; the draft's
    logits are those of the head over [h ; W1[x_prev]] against [W | W2t] (DSpark paper, Eq. 5); the
    distillation gradient flows to them, the cross entropy to the head from the hidden states, and
    both agree with the oracle on the very same tensors.  With the lists of the draft itself the
    distillation loss and its gradient vanish."""
    B, G, V, d, r = 6, 4, 1500, 48, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(61)
    hid = torch.randn((B * G, d), generator=g, device=DEV)
    W1 = torch.randn((V, r), generator=g, device=DEV)
    head = torch.cat([torch.randn((V, d), generator=g, device=DEV) * 0.4,
                      torch.randn((V, r), generator=g, device=DEV) * 0.2], 1).to(torch.bfloat16)
    x = torch.randint(V, (B, G + 1), generator=g, device=DEV)
    rows = torch.cat([hid, W1[x[:, :-1].reshape(-1)]], 1).to(torch.bfloat16)
    labels = x[:, 1:].reshape(-1).to(torch.int32).contiguous()
    weight = torch.exp(-torch.arange(G, device=DEV).float() / G).expand(B, G).contiguous()
    _check_head(sv, rows, head, labels, (0.1 * weight).reshape(-1).contiguous())
    draft = (rows.float() @ head.float().t()).view(B, G, V).to(torch.bfloat16)
    target = torch.cat([draft.float() + 0.5 * torch.randn((B, G, V), generator=g, device=DEV),
                        torch.zeros((B, 1, V), device=DEV)], 1).to(torch.bfloat16)
    o = sv.teacher_topk(target, 64)
    _check_distill(sv, draft, o["ids"], o["values"], None, sv.SPEC_DISTILL_TV, None, None, 0.9 * weight)
    same = sv.teacher_topk(torch.cat([draft, draft[:, :1]], 1), 64)
    f = sv.distill_loss(draft, same["ids"], same["values"], same["lse"])
    gr = sv.distill_loss_backward(draft, same["ids"], same["values"], f["saved"], weight)
    torch.cuda.synchronize()
    assert float(f["loss"].abs().max()) <= 400 * U * 2
    assert float(gr.float().abs().max()) <= 700 * U * 2
