"""Every tile shape and way of sharing out rows of the vocabulary head against the definition in 64 bits.

Tolerances as in test_gpu_training.py: logits dz = (d + 2) u sum |h w| (u = 2^-24), lse max dz + 310 u + u |lse|,
G p (2 dz + dlse + 310 u) and half a step of the type, products (terms + 16) u, half a step of the result.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

from head_plans import PLANS

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


@pytest.mark.parametrize("shape", list(PLANS), ids=lambda s: "-".join(map(str, s)))
def test_head_of_every_plan(sv, shape):
    N, V, d, dtype = shape
    g = torch.Generator(device=DEV)
    g.manual_seed(N + V + d)
    h = torch.randn((N, d), generator=g, device=DEV).to(DT[dtype])
    w = (torch.randn((V, d), generator=g, device=DEV) * (3.0 / d ** 0.5)).to(DT[dtype])
    y = torch.randint(V, (N,), generator=g, device=DEV)
    y[torch.rand((N,), generator=g, device=DEV) < 0.1] = -1
    y[:2] = V - 1
    gl = torch.randn((N,), generator=g, device=DEV)
    y = y.to(torch.int32)
    print(f"head plan {shape}", flush=True)
    got = sv.head_xent(h, w, y)
    b = sv.head_xent_backward(h, w, y, got["lse"], gl)
    torch.cuda.synchronize()

    H, W, Y, gw = h.double(), w.double(), y.long(), gl.double().abs()[:, None]
    eps = torch.finfo(h.dtype).eps
    z = H @ W.t()
    dz = (d + 2) * U * (H.abs() @ W.abs().t())
    lse = torch.logsumexp(z, 1)
    mz = dz.amax(1)
    dlse = mz + 310 * U + U * lse.abs()
    used = Y >= 0
    rows = torch.nonzero(used)[:, 0]
    assert not got["status"].any()
    assert ((got["lse"].double() - lse).abs() <= dlse).all()
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, Y[rows]]
    assert ((got["loss"].double() - loss).abs() <= dlse + mz + U * loss.abs()).all()
    p = torch.exp_(z.sub_(lse[:, None]))
    e = dz.mul_(2.0).add_(dlse[:, None] + 310 * U).mul_(p).mul_(1.01 * gw)
    p[rows, Y[rows]] -= 1.0
    G = p.mul_(torch.where(used, gl.double(), 0.0)[:, None])
    e[~used] = 0.0
    e += (eps / 2 * 1.01 + 4 * U) * G.abs() + 1e-38 * used[:, None]
    for name, ref, tol in (
            ("grad_hidden", G @ W, e @ W.abs() + (V + 16) * U * (G.abs() @ W.abs())),
            ("grad_weight", G.t() @ H, e.t() @ H.abs() + (N + 16) * U * (G.abs().t() @ H.abs()))):
        err = (b[name].double() - ref).abs()
        tol = tol + eps / 2 * 1.01 * ref.abs() + 1e-37
        assert (err <= tol).all(), (name, torch.nonzero(~(err <= tol))[:5].tolist(), float(err.max()))
