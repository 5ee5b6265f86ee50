"""GPU parity of the head's norm, its gradients, its weight in 8 bits and its logits with the fp64 oracle.

Tolerances (u = 2^-24, half a step of fp32; `half` = half a step of the storage type, relative):
  h: one fp32 sum, u |h|, and half |h|.
  rstd: h is off by u, its square by 3 u; a thread adds at most 16 of them, the wave's lanes 6 levels, the waves at
    most 15 more: 37 u; the mean, eps and the sum round 3 times: 43 u, halved by the root, whose rounding and the
    reciprocal's add 2: below 24 u.
  y: h u, rstd 24 u, two products: 27 u < 30 u of |y|, and half |y|.
  scales: the amax (30 u) and a quotient: 32 u.  Codes: the quotient is off by y's and amax's 30 u each and by
    448 / amax's and the product's rounding: 64 u |q| before it is rounded to half a step of e4m3.
    Weights: the quotient of bf16 values is corrected to the nearest fp32, 1 u; fp32 ones 4 u.
  grad_x: xh and g off by u each; dot: (3 + 37) u of mean |g xh|, and one division; then three operations on each
    side: u (rstd (5 |g| + |xh| (46 mean|g xh|)) + 3 |grad_x| + |grad_h|) and half |grad_x|.
  grad_w: 2 u of each term, at most ceil(N / 1024) rows added in fp32 by a thread and 3 more to join the teams of a
    workgroup, the rest fp64, rounded to fp32 (u of the sum) and to the type: u (6 + N / 1024) sum |gy xh|, and half.
  logits: the products of two e4m3 numbers are exact; whatever order the matrix unit adds 128 of them in, each
    addition off by at most 2 u (truncation): 256 u; the scales' product, the multiply-add and at most 128 additions of
    blocks: 131 u: below 400 u of the sum of the terms' magnitudes; and half.
    bf16 logits: the 8-bit form of the matrix unit first cuts each of 8 products off at 2^-13 of the power of two that
    the largest of them holds: 7 of them lose less than 2^-13 of the largest each (it loses nothing: its own product
    has 6 bits behind that power), so 7 2^-13 of the 8 products' magnitudes, in every group of 8.
  (second-order terms: 2^-10 of the above at most.)
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import oracle
from logits_plans import PLANS

DEV = "cuda:0"
U = 2.0 ** -24 * (1 + 2.0 ** -10)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import draft_verification_04_amd as m
    m.load_library()
    return m


def _np(t):
    return t.detach().cpu().float().double().numpy()


def _half(t):
    return torch.finfo(t.dtype).eps / 2 * (1 + 2.0 ** -10)


def _near(got, ref, tol):
    g, r = _np(got), np.asarray(ref)
    fin = np.isfinite(r)
    assert np.array_equal(g[~fin], r[~fin], equal_nan=True)
    err = np.abs(g[fin] - r[fin])
    bound = np.broadcast_to(tol, r.shape)[fin] + 1e-40
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(np.abs(g - r) > tol)[:4])


def _norm_inputs(seed, N, d, dtype, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, d), generator=g)
    r = 4 * torch.randn((N, d), generator=g) if residual else None
    w = 1 + 0.3 * torch.randn(d, generator=g)
    c = lambda t: None if t is None else t.to(DT[dtype]).to(DEV)
    return c(x), c(r), c(w)


def _check_codes(codes, scales, ref, qu, su):
    s = _np(scales)
    assert (np.abs(s - ref["scales"]) <= su * U * ref["scales"]).all()
    q, c = ref["q"], _np(codes)
    # half a step of the code's binade or of the quotient's, whichever is larger (at a power of two they differ)
    half = np.maximum(oracle.e4m3_step(q), oracle.e4m3_step(c)) / 2
    assert (np.abs(c - q) <= half + qu * U * np.abs(q)).all()


def _check_norm(sv, x, r, w, eps=1e-6, quantize=False, out=None):
    ref = oracle.head_norm(x, w, r, eps)
    keep = [None if t is None else t.clone() for t in (x, r, w)]
    o = sv.head_norm(x, w, r, eps=eps, quantize=quantize, out=out)
    torch.cuda.synchronize()
    if out is None:
        for t, k in zip((x, r, w), keep):
            assert t is None or torch.equal(t, k)
    if "rstd" in o:
        _near(o["rstd"], ref["rstd"], 24 * U * ref["rstd"])
    else:
        assert quantize
    if r is not None:
        _near(o["h"], ref["h"], (U + _half(x)) * np.abs(ref["h"]))
    if quantize:
        _check_codes(o["codes"], o["scales"], oracle.quantize(ref["y"], 1), 64, 32)
    else:
        _near(o["y"], ref["y"], (30 * U + _half(x)) * np.abs(ref["y"]))
    return o, ref


NORMS = [(1, 1), (3, 7), (2, 16), (5, 64), (2, 100), (4, 128), (3, 144), (4, 512), (3, 513), (2, 1001), (7, 1024), (2, 1040),
         (2, 2048), (3, 2064), (3, 4096), (2, 4999), (1, 8192), (2, 8208), (1, 16383), (2, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", NORMS)
def test_norm(sv, shape, dtype):
    for residual in (True, False):
        print(f"norm {shape} {dtype} residual={residual}", flush=True)
        x, r, w = _norm_inputs(sum(shape), *shape, dtype, residual)
        _check_norm(sv, x, r, w, eps=1e-5)
        if shape[1] % 16 == 0:
            _check_norm(sv, x, r, w, quantize=True)
            N, d = shape
            new = lambda s, t: torch.empty(s, dtype=t, device=DEV)
            out = dict(codes=new((N, d), torch.float8_e4m3fn), scales=new((N, -(-d // 128)), torch.float32),
                       rstd=new((N,), torch.float32), **(dict(h=new((N, d), x.dtype)) if residual else {}))
            _check_norm(sv, x, r, w, quantize=True, out=out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(sv, dtype):
    for d in (48, 1001, 4096):
        print(f"norm in place {d} {dtype}", flush=True)
        x, r, w = _norm_inputs(d, 5, d, dtype)
        o, _ = _check_norm(sv, x, r, w)
        for a, b in (("x", "r"), ("r", "x")):
            t = dict(x=x.clone(), r=r.clone())
            got = sv.head_norm(t["x"], w, t["r"], out=dict(h=t[a], y=t[b], rstd=torch.empty_like(o["rstd"])))
            torch.cuda.synchronize()
            assert torch.equal(got["h"], o["h"]) and torch.equal(got["y"], o["y"]) and got["h"] is t[a]
            assert torch.equal(got["rstd"], o["rstd"])


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_extreme_rows(sv, dtype, quantize):
    """Rows whose squares overflow or vanish, one loud value, zeros."""
    d = 1024
    x, _, w = _norm_inputs(5, 9, d, dtype, False)
    scale = torch.tensor([1e30, 3e37, 1e-30, 1e-38, 1e-12, 1.0, 1.0, 0.0, 1e18], device=DEV)
    x = (x.float() * scale[:, None]).to(x.dtype)
    x[5, 700] = 2e37
    x[6, 3] = -1e15
    for eps in (1e-6, 1e-30):
        print(f"extreme {dtype} eps={eps}", flush=True)
        _check_norm(sv, x, None, w, eps=eps, quantize=quantize)


def test_norm_of_bad_rows(sv):
    """A NaN or infinity spoils its own row: the norm's values there, and every logit formed from its codes."""
    x, r, w = _norm_inputs(6, 4, 256, "bf16")
    x[1, 17] = float("nan")
    r[2, 200] = float("inf")
    o = sv.head_norm(x, w, r)
    q = sv.head_norm(x, w, r, quantize=True)
    k = sv.head_quantize(_norm_inputs(7, 130, 256, "bf16", False)[0])
    z = sv.head_logits(q["codes"], q["scales"], k["codes"], k["scales"])
    torch.cuda.synchronize()
    assert torch.isnan(o["y"][1]).all() and torch.isnan(o["y"][2, 200]) and not torch.isnan(o["y"][[0, 3]]).any()
    assert torch.isnan(z[1:3]).all() and torch.isfinite(z[[0, 3]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", NORMS + [(1030, 72), (2500, 40), (3001, 9)])
def test_norm_backward(sv, shape, dtype):
    N, d = shape
    x, r, w = _norm_inputs(N + d, N, d, dtype)
    gy, gh, _ = _norm_inputs(N + d + 1, N, d, dtype)
    o = sv.head_norm(x, w, r)
    for g2 in (gh, None):
        print(f"norm backward {shape} {dtype} stream={g2 is not None}", flush=True)
        b = sv.head_norm_backward(gy, o["h"], w, o["rstd"], g2)
        torch.cuda.synchronize()
        ref = oracle.head_norm_grad(gy, o["h"], w, o["rstd"], g2)
        rs, g = _np(o["rstd"])[:, None], np.abs(_np(gy) * _np(w))
        xh = np.abs(_np(o["h"]) * rs)
        tol = U * (rs * (5 * g + 46 * xh * (g * xh).mean(axis=1, keepdims=True)) + 3 * np.abs(ref["grad_x"])
                   + (0 if g2 is None else np.abs(_np(g2)))) + _half(gy) * np.abs(ref["grad_x"])
        _near(b["grad_x"], ref["grad_x"], tol)
        tol = U * (6 + -(-N // 1024)) * (np.abs(_np(gy)) * xh).sum(axis=0) + _half(gy) * np.abs(ref["grad_weight"])
        _near(b["grad_weight"], ref["grad_weight"], tol)
    only = sv.head_norm_backward(gy, o["h"], w, o["rstd"], gh, need_weight=False)
    place = sv.head_norm_backward(gy, o["h"], w, o["rstd"], gh, out=dict(grad_x=gh))     # over the stream's own
    again = sv.head_norm_backward(gy, o["h"], w, o["rstd"], None, out=dict(grad_x=gy))
    torch.cuda.synchronize()
    assert "grad_weight" not in only and torch.equal(only["grad_x"], place["grad_x"])
    assert torch.equal(again["grad_x"], b["grad_x"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2100, 1032), (1100, 8192), (600, 16384), (515, 9001)])
def test_norm_backward_of_several_rows_each(sv, shape, dtype):
    """More rows than workgroups: a workgroup adds ceil(N / 1024) rows of its share in fp32 (2048 values or fewer: of
    each of its two teams), ceil(N / 512) where d > 4096 and ceil(N / 256) where d > 8192."""
    N, d = shape
    x, r, w = _norm_inputs(N + d, N, d, dtype)
    gy = _norm_inputs(N + d + 1, N, d, dtype)[0]
    o = sv.head_norm(x, w, r)
    print(f"norm backward {shape} {dtype}", flush=True)
    b = sv.head_norm_backward(gy, o["h"], w, o["rstd"])
    torch.cuda.synchronize()
    ref = oracle.head_norm_grad(gy, o["h"], w, o["rstd"], None)
    rs, g = _np(o["rstd"])[:, None], np.abs(_np(gy) * _np(w))
    xh = np.abs(_np(o["h"]) * rs)
    tol = U * (rs * (5 * g + 46 * xh * (g * xh).mean(axis=1, keepdims=True)) + 3 * np.abs(ref["grad_x"]))
    _near(b["grad_x"], ref["grad_x"], tol + _half(gy) * np.abs(ref["grad_x"]))
    rows = -(-N // (256 if d > 8192 else 512 if d > 4096 else 1024))
    tol = U * (6 + rows) * (np.abs(_np(gy)) * xh).sum(axis=0) + _half(gy) * np.abs(ref["grad_weight"])
    _near(b["grad_weight"], ref["grad_weight"], tol)


def test_float32_arrays_on_any_boundary(sv):
    """Scales and rstd need no more than their own 4 bytes' alignment."""
    off = lambda *s: torch.empty(int(np.prod(s)) + 1, device=DEV)[1:].view(*s)
    N, V, d = 37, 700, 1040
    x, r, w = _norm_inputs(31, N, d, "bf16")
    head = _norm_inputs(32, V, d, "bf16", False)[0]
    k, q = sv.head_quantize(head), sv.head_norm(x, w, r, quantize=True)
    k2 = sv.head_quantize(head, out=dict(codes=torch.empty_like(k["codes"]), scales=off(*k["scales"].shape)))
    q2 = sv.head_norm(x, w, r, quantize=True, out=dict(codes=torch.empty_like(q["codes"]), scales=off(N, 9),
                                                       h=torch.empty_like(x), rstd=off(N)))
    z, z2 = sv.head_logits(q["codes"], q["scales"], k["codes"], k["scales"]), \
        sv.head_logits(q2["codes"], q2["scales"], k2["codes"], k2["scales"])
    o = sv.head_norm(x, w, r)
    b, b2 = sv.head_norm_backward(x, o["h"], w, o["rstd"]), sv.head_norm_backward(x, q2["h"], w, q2["rstd"])
    torch.cuda.synchronize()
    assert torch.equal(q["scales"], q2["scales"]) and torch.equal(k["scales"], k2["scales"]) and torch.equal(z, z2)
    assert torch.equal(o["rstd"], q2["rstd"]) and torch.equal(b["grad_x"], b2["grad_x"])
    assert torch.equal(b["grad_weight"], b2["grad_weight"])


def test_norm_backward_against_differences(sv):
    """The formula's gradient against central differences of the forward call, in fp32.

    f(t) = sum(gy y(x + t v)) along a direction v: the difference over 2 t is off by t^2 / 6 of the third derivative
    and by the rounding of y, 30 u sum |gy y| / t.  At t = 2^-6, with |v| about 1 a value and rows of norm sqrt(d), the
    first is a t^2-th part (of order (v.x / d)^3 terms): 2^-12 of sum |gy| |v| covers it."""
    x, _, w = _norm_inputs(11, 6, 200, "f32", False)
    gy, v, _ = _norm_inputs(12, 6, 200, "f32")
    o = sv.head_norm(x, w)
    b = sv.head_norm_backward(gy, x, w, o["rstd"])
    t = 2.0 ** -6
    f = [(_np(sv.head_norm(x + s * t * v, w)["y"]) * _np(gy)).sum() for s in (1, -1)]
    scale = np.abs(_np(gy) * _np(w)).sum()
    want = (_np(b["grad_x"]) * _np(v)).sum()
    assert abs((f[0] - f[1]) / (2 * t) - want) <= 2.0 ** -12 * np.abs(_np(gy) * _np(v) * _np(w)).sum() + 60 * U * scale / t
    f = [(_np(sv.head_norm(x, w + s * t * v[0])["y"]) * _np(gy)).sum() for s in (1, -1)]      # linear in the weight
    want = (_np(b["grad_weight"]) * _np(v[0])).sum()
    assert abs((f[0] - f[1]) / (2 * t) - want) <= 60 * U * (np.abs(_np(gy) * _np(x)).sum() * 4 + scale) / t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 16), (5, 48), (127, 128), (128, 144), (129, 1040), (300, 272), (257, 4096)])
def test_quantize(sv, shape, dtype):
    print(f"quantize {shape} {dtype}", flush=True)
    w = _norm_inputs(shape[0], *shape, dtype, False)[0] * 0.05
    o = sv.head_quantize(w)
    torch.cuda.synchronize()
    ref = oracle.quantize(w, 128)
    _check_codes(o["codes"], o["scales"], ref, 4, 2)
    if dtype == "bf16":
        assert np.array_equal(_np(o["codes"]), ref["codes"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_extreme_blocks(sv, dtype):
    """Blocks of zeros, of tiny and of huge values; ties; one bad value spoils its block alone."""
    w = _norm_inputs(9, 300, 512, dtype, False)[0].float()
    w[:128, :128] = 0
    w[:128, 128:256] *= 1e-36
    w[:128, 256:384] *= 2e37
    w[:128, 384:] *= 1e-26
    w[128:256, :128] = torch.randint(-32, 33, (128, 128), device=DEV) * 0.5    # amax 16: quotients end in ties
    w = w.to(DT[dtype])
    o = sv.head_quantize(w)
    torch.cuda.synchronize()
    ref = oracle.quantize(w, 128)
    _check_codes(o["codes"], o["scales"], ref, 4, 2)
    assert np.array_equal(_np(o["codes"])[128:256, :128], ref["codes"][128:256, :128])
    w[200, 300] = float("nan")
    w[299, 500] = float("inf")
    b = sv.head_quantize(w)
    torch.cuda.synchronize()
    z = _np(b["codes"]) * np.repeat(np.repeat(_np(b["scales"]), 128, 0)[:300], 128, 1)
    bad = np.zeros((300, 512), dtype=bool)
    bad[128:256, 256:384] = bad[256:, 384:] = True
    assert np.isnan(z[bad]).all() and np.array_equal(_np(b["codes"])[~bad], _np(o["codes"])[~bad])


def _logit_inputs(seed, N, V, d):
    g = torch.Generator(device=DEV).manual_seed(seed)
    y = torch.randn((N, d), generator=g, device=DEV)
    w = torch.randn((V, d), generator=g, device=DEV) * (3 / d ** 0.5)
    # scales that differ from block to block by more than the codes' range
    y *= torch.exp2(torch.randint(-12, 13, (N, -(-d // 128)), generator=g, device=DEV).float()).repeat_interleave(128, 1)[:, :d]
    return y, w


def _as_codes(y, rows):
    n, d = y.shape
    a = torch.nn.functional.pad(y.abs(), (0, -d % 128, 0, -n % rows))
    s = a.view(a.shape[0] // rows, rows, -1, 128).amax((1, 3)) / 448
    full = s.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :d]
    return (y / full).to(torch.float8_e4m3fn), s


def _logit_tol(z, ref):
    cut = 7 * 2.0 ** -13 if z.dtype == torch.bfloat16 else 0.0
    return (400 * U + cut) * ref["mass"] + _half(z) * np.abs(ref["logits"])


def _check_logits(sv, codes, scales, wc, ws, dtype):
    z = sv.head_logits(codes, scales, wc, ws, dtype=dtype)
    torch.cuda.synchronize()
    ref = oracle.head_logits(codes, scales, wc, ws)
    _near(z, ref["logits"], _logit_tol(z, ref))
    return z


LOGITS = [(1, 1, 16), (1, 1000, 128), (2, 15, 112), (3, 1003, 272), (15, 64, 48), (16, 63, 256), (17, 129, 144), (31, 127, 1040),
          (32, 500, 384), (33, 65, 2064), (64, 1000, 4096), (65, 300, 640), (100, 257, 1024), (128, 128, 128), (129, 1003, 528),
          (200, 20011, 256), (256, 256, 2048), (257, 513, 1040), (300, 1001, 16), (511, 129, 272), (1000, 3001, 400), (2, 300, 16384),
          (70, 300, 16368), (513, 2050, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", LOGITS)
def test_logits(sv, shape, dtype):
    print(f"logits {shape} {dtype}", flush=True)
    y, w = _logit_inputs(sum(shape), *shape)
    _check_logits(sv, *_as_codes(y, 1), *_as_codes(w, 128), DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", list(PLANS))
def test_logits_of_every_tile(sv, shape, dtype):
    print(f"tile {PLANS[shape]} {shape} {dtype}", flush=True)
    y, w = _logit_inputs(sum(shape) + 1, *shape)
    _check_logits(sv, *_as_codes(y, 1), *_as_codes(w, 128), DT[dtype])


def test_logits_write_their_rows_alone(sv):
    """Odd rows of an odd vocabulary in the middle of a buffer: nothing around them is written."""
    for N, V, d in ((5, 1003, 144), (70, 333, 272), (300, 20011, 128), (520, 40003, 400), (200, 9001, 272), (50, 40001, 144)):
        for dt in (torch.bfloat16, torch.float32):
            print(f"rows {N} {V} {d} {dt}", flush=True)
            y, w = _logit_inputs(3, N, V, d)
            (c, s), (wc, ws) = _as_codes(y, 1), _as_codes(w, 128)
            buf = torch.full((N * V + 512,), 7.0, dtype=dt, device=DEV)
            sv.head_logits(c, s, wc, ws, out=buf[256:256 + N * V].view(N, V))
            z = sv.head_logits(c, s, wc, ws, dtype=dt)
            torch.cuda.synchronize()
            assert torch.equal(buf[256:256 + N * V].view(N, V), z)
            assert (buf[:256] == 7).all() and (buf[256 + N * V:] == 7).all()


def test_logits_of_bad_codes(sv):
    """A NaN code spoils its row or its column, also next to the end of a short last block."""
    for N in (3, 40, 300):
        y, w = _logit_inputs(4, N, 200, 272)
        (c, s), (wc, ws) = _as_codes(y, 1), _as_codes(w, 128)
        c.view(torch.uint8)[2, 271] = 0x7f
        wc.view(torch.uint8)[100, 0] = 0xff
        wc.view(torch.uint8)[199, 256] = 0x7f
        z = sv.head_logits(c, s, wc, ws)
        torch.cuda.synchronize()
        bad = torch.zeros((N, 200), dtype=torch.bool, device=DEV)
        bad[2] = bad[:, 100] = bad[:, 199] = True
        assert torch.equal(torch.isnan(z), bad), N


def test_offsets_past_32_bits(sv):
    """Rows past 2^32 bytes and 2^31 values of the activations, the logits and the weight."""
    d, N = 8192, 300000
    x = torch.zeros((N, d), dtype=torch.bfloat16, device=DEV)
    few, _, w = _norm_inputs(13, 4, d, "bf16", False)
    at = torch.tensor([0, 140000, 263000, N - 1], device=DEV)
    x[at] = few
    o, q = sv.head_norm(x, w), sv.head_norm(x, w, quantize=True)
    o4, q4 = sv.head_norm(few, w), sv.head_norm(few, w, quantize=True)
    b = sv.head_norm_backward(x, x, w, o["rstd"], out=dict(grad_x=x), need_weight=False)
    b4 = sv.head_norm_backward(few, few, w, o4["rstd"])
    torch.cuda.synchronize()
    assert torch.equal(o["y"][at], o4["y"]) and torch.equal(o["rstd"][at], o4["rstd"])
    assert torch.equal(q["codes"][at].view(torch.uint8), q4["codes"].view(torch.uint8))
    assert torch.equal(q["scales"][at], q4["scales"]) and torch.equal(b["grad_x"][at], b4["grad_x"])
    del o, x, b
    # logits [N, V] of 2.4 G values, and a weight of 4.3 GB
    few, wt = _logit_inputs(14, 40, 8000, 128)
    wc, ws = _as_codes(wt, 128)
    c4, s4 = _as_codes(few, 1)
    rep = 300000 // 40
    z = sv.head_logits(c4.view(torch.uint8).repeat(rep, 1).view(c4.dtype), s4.repeat(rep, 1), wc, ws)
    ref = oracle.head_logits(c4, s4, wc, ws)
    for k in (0, rep // 2, rep - 1):
        _near(z[40 * k:40 * k + 40], ref["logits"], _logit_tol(z, ref))
    del z
    V = 524288
    big = torch.zeros((V, d), dtype=torch.float8_e4m3fn, device=DEV)
    wt = _logit_inputs(15, 1, 128, d)[1]
    wc, ws = _as_codes(wt, 128)
    big.view(torch.uint8)[V - 128:] = wc.view(torch.uint8)
    scales = torch.ones((V // 128, d // 128), device=DEV)
    scales[-1] = ws[0]
    for n in (3, 300):
        few = _logit_inputs(16, n, 1, d)[0]
        c, s = _as_codes(few, 1)
        z = sv.head_logits(c, s, big, scales)
        torch.cuda.synchronize()
        assert (z[:, :V - 128] == 0).all()
        ref = oracle.head_logits(c, s, wc, ws)
        _near(z[:, V - 128:], ref["logits"], _logit_tol(z, ref))


def test_quantize_past_32_bits(sv):
    w = torch.zeros((524288, 8192), dtype=torch.bfloat16, device=DEV)
    few = _norm_inputs(17, 128, 8192, "bf16", False)[0]
    w[-128:] = few
    o, o4 = sv.head_quantize(w), sv.head_quantize(few)
    torch.cuda.synchronize()
    assert torch.equal(o["codes"][-128:].view(torch.uint8), o4["codes"].view(torch.uint8))
    assert torch.equal(o["scales"][-1], o4["scales"][0]) and (o["codes"][:1000].float() == 0).all()


def test_streams_and_a_captured_graph(sv):
    """The calls on side streams, and recorded into one graph that is replayed with eager work between."""
    x, r, w = _norm_inputs(18, 70, 1024, "bf16")
    gy, gh, _ = _norm_inputs(19, 70, 1024, "bf16")
    head = _norm_inputs(20, 700, 1024, "bf16", False)[0]

    def calls(stream=None):
        k = sv.head_quantize(head, stream=stream)
        q = sv.head_norm(x, w, r, quantize=True, stream=stream)
        z = sv.head_logits(q["codes"], q["scales"], k["codes"], k["scales"], stream=stream)
        o = sv.head_norm(x, w, r, stream=stream)
        b = sv.head_norm_backward(gy, o["h"], w, o["rstd"], gh, stream=stream)
        return [k["codes"].view(torch.uint8), k["scales"], q["codes"].view(torch.uint8), q["scales"], z, o["y"], o["h"],
                b["grad_x"], b["grad_weight"]]
    ref = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [calls(s) for s in side]
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = calls()
    for rep in range(3):
        for t in out:
            t.zero_()
        calls()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        print(f"graph replay {rep}", flush=True)
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_a_training_step_through_norm_and_head(sv):
    """norm -> cross entropy -> the head's gradients -> the norm's, as an autograd.Function, against torch in fp64."""
    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, r, w, head, labels):
            o = sv.head_norm(x, w, r)
            l = sv.head_xent(o["y"], head, labels)
            ctx.save_for_backward(o["y"], o["h"], o["rstd"], w, head, labels, l["lse"])
            return l["loss"]

        @staticmethod
        def backward(ctx, g):
            y, h, rstd, w, head, labels, lse = ctx.saved_tensors
            b = sv.head_xent_backward(y, head, labels, lse, g.contiguous())
            n = sv.head_norm_backward(b["grad_hidden"], h, w, rstd)
            return n["grad_x"], n["grad_x"], n["grad_weight"], b["grad_weight"], None
    N, V, d = 50, 300, 128
    x, r, w = _norm_inputs(21, N, d, "f32")
    head = _norm_inputs(22, V, d, "f32", False)[0] * 0.2
    labels = torch.randint(V, (N,), device=DEV).to(torch.int32)
    leaves = [t.clone().requires_grad_() for t in (x, r, w, head)]
    weight = torch.rand(N, device=DEV)
    loss = Loss.apply(*leaves, labels)
    (loss * weight).sum().backward()
    torch.cuda.synchronize()
    l64 = [t.cpu().double().requires_grad_() for t in (x, r, w, head)]
    h = l64[0] + l64[1]
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * l64[2]
    ref = torch.nn.functional.cross_entropy(y @ l64[3].t(), labels.cpu().long(), reduction="none")
    (ref * weight.cpu().double()).sum().backward()
    # logits: 128 products of y (30 u) and head, (d + 32) u of sum |y head| < 160 u * 40; the loss moves by twice
    # that, and the gradients' relative error is that of p, times the sums' own (some hundred u): 2^-10 covers both
    assert np.allclose(_np(loss), ref.detach().numpy(), rtol=0, atol=2 * 160 * 40 * U)
    for a, b in zip(leaves, l64):
        scale = b.grad.abs().max().item()
        assert (a.grad.cpu().double() - b.grad).abs().max().item() <= 2.0 ** -10 * scale


def test_from_hidden_states_to_verified_tokens(sv):
    """norm -> logits -> adjustment -> verification, each step against the oracle on what the step before gave it."""
    from parity import HostInputs, compare_verify, run_oracle_pooled
    B, G, V, d = 6, 4, 1511, 256
    R = G + 1
    x, r, w = _norm_inputs(23, B * R, d, "bf16")
    head = _norm_inputs(24, V, d, "bf16", False)[0] * 0.15
    k = sv.head_quantize(head)
    q = sv.head_norm(x, w, r, quantize=True)
    target = torch.empty((B, R, V), dtype=torch.bfloat16, device=DEV)
    sv.head_logits(q["codes"], q["scales"], k["codes"], k["scales"], out=target.view(B * R, V))
    g = torch.Generator(device=DEV).manual_seed(25)
    draft = (target[:, :G].float() + 0.3 * torch.randn((B, G, V), generator=g, device=DEV)).to(torch.bfloat16)
    rep = torch.linspace(1.0, 1.5, B, device=DEV)
    hist = torch.randint(V, (B, 60), generator=g, device=DEV).to(torch.int32)
    L = torch.tensor([4, 3, 0, 4, 2, 4], dtype=torch.int32, device=DEV)
    toks = draft.float().argmax(2).to(torch.int32)
    kw = dict(history=hist, repetition=rep, frequency=rep - 1, presence=rep * 0.1)
    before = target.clone()
    at = sv.adjust_logits(target, toks, L, in_place=True, **kw)
    ad = sv.adjust_logits(draft, toks, L, in_place=True, **kw)
    seed = torch.arange(B, device=DEV)
    out = sv.verify(target, draft, toks, L, None, None, seed)
    torch.cuda.synchronize()
    ref = oracle.head_norm(x, w, r)
    _check_codes(q["codes"], q["scales"], oracle.quantize(ref["y"], 1), 64, 32)
    z = oracle.head_logits(q["codes"], q["scales"], k["codes"], k["scales"])
    _near(before.view(B * R, V), z["logits"], _logit_tol(before, z))
    a = oracle.adjust_logits(before, toks, L, hist, repetition=rep, frequency=rep - 1, presence=rep * 0.1)
    _near(target, a["logits"], 5 * U * a["mass"] + _half(target) * np.abs(a["logits"]))
    assert at["status"].tolist() == [0] * B and ad["status"].tolist() == [0] * B
    h = HostInputs.of(target, draft, toks, L, None, None, seed)
    compare_verify(out, run_oracle_pooled(h), inputs=h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", list(PLANS))
def test_every_logit_in_its_place(sv, shape, dtype):
    """Rows that pick one column of the weight each: every logit is one code of the weight, exactly, so that values that
    change places between a wave's lanes on their way out cannot pass for rounding."""
    N, V, d = shape
    g = torch.Generator(device=DEV).manual_seed(N + V + d)
    w = torch.randint(0, 256, (V, d), generator=g, device=DEV, dtype=torch.uint8)
    w[(w & 0x7f) == 0x7f] = 0                                                      # not NaN
    w = w.view(torch.float8_e4m3fn)
    pick = torch.randint(0, d, (N,), generator=g, device=DEV)
    x = torch.zeros((N, d), device=DEV)
    x[torch.arange(N, device=DEV), pick] = 1.0
    ones = lambda *s: torch.ones(s, device=DEV)
    G = -(-d // 128)
    z = sv.head_logits(x.to(torch.float8_e4m3fn), ones(N, G), w, ones(-(-V // 128), G), dtype=DT[dtype])
    torch.cuda.synchronize()
    assert torch.equal(z.float(), w.float().t()[pick])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(4099, 72), (8195, 9), (4101, 1000), (2100, 2001), (1030, 4096), (2051, 2999), (1100, 8001),
                                   (300, 16384)])
def test_norm_backward_over_several_turns(sv, shape, dtype):
    """Teams of every size take more than one row each: both gradients, with the stream's own gradient and without it,
    and written over each input that may be."""
    N, d = shape
    x, r, w = _norm_inputs(N + d, N, d, dtype)
    gy, gh, _ = _norm_inputs(N + d + 1, N, d, dtype)
    o = sv.head_norm(x, w, r)
    rs, g = _np(o["rstd"])[:, None], np.abs(_np(gy) * _np(w))
    xh = np.abs(_np(o["h"]) * rs)
    rows = -(-N // (256 if d > 8192 else 512 if d > 4096 else 1024))
    for g2 in (gh, None):
        print(f"norm backward over turns {shape} {dtype} stream={g2 is not None}", flush=True)
        b = sv.head_norm_backward(gy, o["h"], w, o["rstd"], g2)
        torch.cuda.synchronize()
        ref = oracle.head_norm_grad(gy, o["h"], w, o["rstd"], g2)
        tol = U * (rs * (5 * g + 46 * xh * (g * xh).mean(axis=1, keepdims=True)) + 3 * np.abs(ref["grad_x"])
                   + (0 if g2 is None else np.abs(_np(g2)))) + _half(gy) * np.abs(ref["grad_x"])
        _near(b["grad_x"], ref["grad_x"], tol)
        tol = U * (6 + rows) * (np.abs(_np(gy)) * xh).sum(axis=0) + _half(gy) * np.abs(ref["grad_weight"])
        _near(b["grad_weight"], ref["grad_weight"], tol)
        for name, t in (("grad_y", gy), ("h", o["h"]), ("grad_h", g2)):
            if t is None:
                continue
            ins = dict(grad_y=gy, h=o["h"], grad_h=g2)
            ins[name] = t.clone()
            c = sv.head_norm_backward(ins["grad_y"], ins["h"], w, o["rstd"], ins["grad_h"],
                                      out=dict(grad_x=ins[name], grad_weight=torch.empty_like(w)))
            torch.cuda.synchronize()
            assert torch.equal(c["grad_x"], b["grad_x"]) and torch.equal(c["grad_weight"], b["grad_weight"]), name


def _e4m3_values():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return np.unique(v[np.isfinite(v)])


@pytest.mark.parametrize("kind", ["normal", "bf16 values", "next to halfway", "small and large"])
@pytest.mark.parametrize("shape", [(257, 4096), (1000, 1040)])
def test_codes_of_fp32_weights_are_the_nearest(sv, shape, kind):
    """Every code is the one nearest to w 448 / amax, the even one halfway between two.  Exact: 448 w and code * amax have at
    most 33 and 28 bits, and their difference is exact in fp64 for the code and its neighbours."""
    print(f"nearest codes {shape} {kind}", flush=True)
    V, d = shape
    rng = np.random.default_rng(V + d)
    w = (0.05 * rng.standard_normal((V, d))).astype(np.float32)
    if kind == "bf16 values":
        w = torch.from_numpy(w).to(torch.bfloat16).float().numpy()
    if kind == "small and large":
        w *= np.exp2(rng.integers(-120, 120, (-(-V // 128), -(-d // 128))).repeat(128, 0)[:V].repeat(128, 1)[:, :d]).astype(np.float32)
    spread = lambda m: m.repeat(128, 0)[:V].repeat(128, 1)[:, :d]
    pad = lambda a: np.pad(np.abs(a), ((0, -V % 128), (0, -d % 128))).reshape(-(-V // 128), 128, -(-d // 128), 128)
    values = _e4m3_values()
    if kind == "next to halfway":
        top = pad(w).max((1, 3))
        m = spread(top.astype(np.float64))
        k = rng.integers(0, len(values) - 1, (V, d))
        near = ((values[k] + values[k + 1]) / 2 * m / 448).astype(np.float32)
        step = rng.integers(-1, 2, (V, d))
        near = np.where(step == 0, near, np.nextafter(near, np.where(step > 0, np.inf, -np.inf).astype(np.float32)))
        w = np.where(np.abs(w) == m, w, near.astype(np.float32))
    m = spread(np.maximum(pad(w).max((1, 3)).astype(np.float64), 2.0 ** -100))
    o = sv.head_quantize(torch.from_numpy(w).to(DEV))
    torch.cuda.synchronize()
    c = _np(o["codes"])
    at = np.searchsorted(values, c)
    assert (values[at] == c).all()
    a = 448.0 * w.astype(np.float64)
    here = np.abs(a - c * m)
    even = (o["codes"].view(torch.uint8).cpu().numpy() & 1) == 0
    for by in (-1, 1):
        other = np.abs(a - values[np.clip(at + by, 0, len(values) - 1)] * m)
        ok = (at + by < 0) | (at + by >= len(values)) | (here < other) | ((here == other) & even)
        assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[:3].tolist())
