"""Cases that measure the operators between the last hidden state and the logits that verification reads: the
head's norm (with the residual's addition, an output in 8 bits and its gradients), the head's weight in 8 bits,
the logits as a product of 8-bit numbers with a scale for each block of 128, and the adjustment of logits by
penalties, biases and masks.

`listed()` names the cases, `draw(rng)` makes one more of the same ranges, `prepare` builds a case's inputs from a
seed, `run` makes one pass (the plain form in elementary torch operations, or, with `own`, the library's calls),
`work` counts what a pass cannot do without and `exact` evaluates the definition in 64 bits.

  norm     h = x + residual;  y = h / sqrt(mean(h^2) + eps) * w, stored in the inputs' type or as e4m3 codes with
           a scale for each 128 of a row (scale = max(amax, 2^-100) / 448, code = y / scale); a "step" also forms
           the gradients of h (with the residual stream's own gradient added) and of w, at the stored h;
  weight   codes and scales of a weight, a scale for each block of 128 x 128;
  logits   z[n, v] = sum over blocks g of sx[n, g] sw[v / 128, g] sum over k in g of x[n, k] w[v, k];
  adjust   per request, row k of its block, token v, with the counts taken over the history and the draft tokens
           before row k: a token of the prompt or the output has z divided by the repetition penalty where z > 0
           and multiplied by it elsewhere; then z -= frequency * count, z -= presence where the count (of output
           tokens) is not 0, z += bias, and -inf where the mask's bit is 0.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_EPS = 1e-6
_FLOOR = 2.0 ** -100


def listed():
    return [
        # the norm of one token: the latency of a call
        dict(name="norm_one", op="norm", N=1, d=1024, dtype="bf16", residual=True, q8=True, step=False),
        # the rows of the verification batch of 256 blocks of 16 drafts and a bonus row, for an 8-bit head
        dict(name="norm_batch_8bit", op="norm", N=4352, d=4096, dtype="bf16", residual=True, q8=True, step=False),
        # a training step's norm in front of the head, on 512 anchors with blocks of 16
        dict(name="norm_step", op="norm", N=8192, d=4096, dtype="bf16", residual=True, q8=False, step=True),
        # the same in fp32, rows that do not start on a 16-byte boundary, no residual
        dict(name="norm_step_odd", op="norm", N=1791, d=1001, dtype="f32", residual=False, q8=False, step=True),
        # a trained head made ready for serving
        dict(name="weight_full", op="weight", V=151936, d=4096, dtype="bf16"),
        # a small drafter's, fp32, blocks that end inside 128 both ways
        dict(name="weight_odd", op="weight", V=20011, d=1040, dtype="f32"),
        # a few rows against a small vocabulary: latency
        dict(name="logits_small", op="logits", N=3, V=1003, d=272, out="f32"),
        # one request's block of 16 drafts and the bonus row: bound by reading the weight
        dict(name="logits_block", op="logits", N=17, V=151936, d=4096, out="bf16"),
        # the rows of a verify budget of 2048 tokens
        dict(name="logits_budget", op="logits", N=2048, V=151936, d=4096, out="bf16"),
        # one token of one request, no drafts: latency
        dict(name="adjust_one", op="adjust", B=1, gamma=0, V=1000, H=100, dtype="f32", bias=True, masks=False,
             ragged=False),
        # 64 blocks of 16 drafts, penalties on ordinary histories and a short list of biases
        dict(name="adjust_batch", op="adjust", B=64, gamma=16, V=151936, H=2048, dtype="bf16", bias=True,
             masks=False, ragged=True),
        # the second vocabulary, blocks of 7 after long histories, every second request under a grammar
        dict(name="adjust_grammar", op="adjust", B=96, gamma=7, V=129280, H=30011, dtype="bf16", bias=False,
             masks=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "weight", "logits", "logits", "adjust", "adjust"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        while True:
            q8, N, d = rng.random() < 0.5, _log(rng, 1, 16384), _log(rng, 64, 8192)
            if N * d <= 8192 * 4096 // (2 if dtype == "f32" else 1):
                return dict(op=op, N=N, d=16 * (d // 16) if q8 else d, dtype=dtype, residual=rng.random() < 0.7,
                            q8=q8, step=not q8 and rng.random() < 0.7)
    if op == "weight":
        while True:
            V, d = _log(rng, 500, 151936), 16 * _log(rng, 8, 512)
            if V * d <= 151936 * 4096 // (2 if dtype == "f32" else 1):
                return dict(op=op, V=V, d=d, dtype=dtype)
    if op == "logits":
        while True:
            N, V, d = _log(rng, 1, 2048), _log(rng, 500, 151936), 16 * _log(rng, 8, 512)
            if N * V * d <= 2048 * 151936 * 4096 and V * d <= 151936 * 4096:
                return dict(op=op, N=N, V=V, d=d, out=dtype)
    while True:
        B, gamma, V, H = _log(rng, 1, 256), rng.randint(0, 16), _log(rng, 300, 262144), _log(rng, 1, 32768)
        if B * (gamma + 1) * V <= 64 * 17 * 151936 // (2 if dtype == "f32" else 1) and B * V <= 128 * 151936:
            return dict(op=op, B=B, gamma=gamma, V=V, H=H, dtype=dtype, bias=rng.random() < 0.5,
                        masks=rng.random() < 0.4, ragged=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------

def _chunks(n, per_row, limit=1 << 28):
    step = max(128, limit // max(1, per_row) // 128 * 128)
    return [(i, min(n, i + step)) for i in range(0, n, step)]


def _scaled(x, scale):
    """x in blocks of `scale`'s, divided by it: [rows, d] by [rows or blocks of 128 rows, blocks of 128 columns]"""
    rows, d = x.shape
    if scale.shape[0] != rows:
        scale = scale.repeat_interleave(128, 0)[:rows]
    return x / scale.repeat_interleave(128, 1)[:, :d]


def _block_amax(x, rows):
    """The largest magnitude of every block of `rows` rows and 128 columns."""
    n, d = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -d % 128, 0, -n % rows))
    return a.view(a.shape[0] // rows, rows, a.shape[1] // 128, 128).amax((1, 3))


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 29)
    st = dict(case=case)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)
    rand = lambda *s: torch.rand(s, generator=g, device=dev)
    if case["op"] == "norm":
        N, d, dt = case["N"], case["d"], _DT[case["dtype"]]
        # a residual stream has a few columns much larger than the others
        loud = torch.where(rand(d) < 0.01, 20.0, 1.0)
        st["x"] = randn(N, d).to(dt)
        st["residual"] = (randn(N, d) * 4.0 * loud).to(dt) if case["residual"] else None
        st["w"] = (1.0 + 0.2 * randn(d)).to(dt)
        if case["step"]:
            st["grad_y"] = (randn(N, d) / N).to(dt)
            st["grad_h"] = (randn(N, d) / N).to(dt) if case["residual"] else None
        return st
    if case["op"] == "weight":
        V, d = case["V"], case["d"]
        st["weight"] = torch.empty((V, d), dtype=_DT[case["dtype"]], device=dev)
        for i, j in _chunks(V, d):
            st["weight"][i:j] = (randn(j - i, d) * (3.0 / math.sqrt(d))).to(_DT[case["dtype"]])
        return st
    if case["op"] == "logits":
        N, V, d = case["N"], case["V"], case["d"]
        y = randn(N, d) * torch.where(rand(d) < 0.01, 10.0, 1.0)
        st["scales"] = _block_amax(y, 1) / 448.0
        st["codes"] = _scaled(y, st["scales"]).to(_F8)
        st["weight_codes"] = torch.empty((V, d), dtype=_F8, device=dev)
        st["weight_scales"] = torch.empty((-(-V // 128), -(-d // 128)), device=dev)
        for i, j in _chunks(V, d):
            w = randn(j - i, d) * (3.0 / math.sqrt(d))
            s = _block_amax(w, 128) / 448.0
            st["weight_scales"][i // 128:-(-j // 128)] = s
            st["weight_codes"][i:j] = _scaled(w, s).to(_F8)
        return st
    B, G, V, H, dt = case["B"], case["gamma"], case["V"], case["H"], _DT[case["dtype"]]
    R = G + 1
    # tokens of text: a few are frequent, most are rare
    text = lambda *s: (V * rand(*s) ** 4).to(torch.int32).clamp(max=V - 1)
    st["history"] = text(B, H)
    st["history_len"] = torch.randint(H // 2, H + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    st["prompt_len"] = (st["history_len"] * rand(B)).to(torch.int32)
    st["draft_tokens"] = text(B, G) if G else None
    st["lengths"] = torch.randint(0, G + 1, (B,), generator=g, device=dev, dtype=torch.int32) if case["ragged"] and G else None
    plain = rand(B) < 0.2   # requests without penalties
    st["repetition"] = torch.where(plain, 1.0, 1.0 + 0.3 * rand(B))
    st["frequency"] = torch.where(plain, 0.0, 0.6 * rand(B))
    st["presence"] = torch.where(plain, 0.0, 0.4 * rand(B))
    st["bias"] = None
    if case["bias"]:
        # up to 64 tokens for each request, of which a tenth are banned
        n = torch.randint(0, min(64, V) + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        at = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        at[1:] = n.cumsum(0)
        toks = rand(B, V).topk(min(64, V), 1).indices.to(torch.int32)
        keep = torch.arange(min(64, V), device=dev)[None, :] < n[:, None]
        toks = toks[keep].contiguous()
        vals = torch.where(rand(len(toks)) < 0.1, -math.inf, 4.0 * randn(len(toks)))
        st["bias"] = (at, toks, vals)
    st["mask"] = st["mask_index"] = None
    if case["masks"]:
        M = (B + 1) // 2
        st["mask_index"] = torch.full((B,), -1, dtype=torch.int32, device=dev)
        st["mask_index"][::2] = torch.arange(M, device=dev, dtype=torch.int32)
        # states that allow a few tokens, and states that forbid a few
        words = -(-V // 32)
        allow = torch.where(rand(M, R) < 0.5, 0.002, 0.95)
        st["mask"] = torch.empty((M, R, words), dtype=torch.int32, device=dev)
        bit = 2 ** torch.arange(32, device=dev)
        for i in range(M):
            on = rand(R, words, 32) < allow[i, :, None, None]
            st["mask"][i] = (on * bit).sum(2).to(torch.int32)
    st["logits"] = torch.empty((B, R, V), dtype=dt, device=dev)
    flat = st["logits"].view(B * R, V)
    for i, j in _chunks(B * R, V):
        flat[i:j] = (randn(j - i, V) * 3.0).to(dt)
    st["out"] = torch.zeros_like(st["logits"])   # the rows past a request's length stay as they are
    return st


# ---- the library's calls --------------------------------------------------------------------

def _run_own(st):
    import draft_verification_04_amd as sv
    case = st["case"]
    if case["op"] == "norm":
        o = sv.head_norm(st["x"], st["w"], st["residual"], eps=_EPS, quantize=case["q8"])
        if case["q8"]:
            r = dict(codes=o["codes"], scales=o["scales"])
        else:
            r = dict(y=o["y"], rstd=o["rstd"])
        if case["residual"]:
            r["h"] = o["h"]
        if case["step"]:
            b = sv.head_norm_backward(st["grad_y"], o["h"], st["w"], o["rstd"], st["grad_h"])
            r["grad_x"], r["grad_w"] = b["grad_x"], b["grad_weight"]
        return r
    if case["op"] == "weight":
        o = sv.head_quantize(st["weight"])
        return dict(codes=o["codes"], scales=o["scales"])
    if case["op"] == "logits":
        return dict(logits=sv.head_logits(st["codes"], st["scales"], st["weight_codes"], st["weight_scales"],
                                          dtype=_DT[case["out"]]))
    o = sv.adjust_logits(st["logits"], st["draft_tokens"], st["lengths"], history=st["history"],
                         history_len=st["history_len"], prompt_len=st["prompt_len"], repetition=st["repetition"],
                         frequency=st["frequency"], presence=st["presence"], bias=st["bias"], mask=st["mask"],
                         mask_index=st["mask_index"], out=st["out"])
    return dict(logits=o["logits"], status=o["status"])


# ---- the plain form -------------------------------------------------------------------------

def _plain_norm(st):
    case, dt = st["case"], _DT[st["case"]["dtype"]]
    h, w = st["x"].float(), st["w"].float()
    if case["residual"]:
        h = h + st["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS)
    y = h * rstd * w
    if case["q8"]:
        s = _block_amax(y, 1).clamp(min=_FLOOR) / 448.0
        r = dict(codes=_scaled(y, s).to(_F8), scales=s)
    else:
        r = dict(y=y.to(dt), rstd=rstd[:, 0])
    if case["residual"]:
        r["h"] = h.to(dt)
    if case["step"]:
        xh = h.to(dt).float() * rstd
        gy = st["grad_y"].float()
        g = gy * w
        gx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
        if case["residual"]:
            gx = gx + st["grad_h"].float()
        r["grad_x"] = gx.to(dt)
        r["grad_w"] = (gy * xh).sum(0, dtype=torch.float64).to(dt)
    return r


def _plain_weight(st):
    w = st["weight"].float()
    s = _block_amax(w, 128).clamp(min=_FLOOR) / 448.0
    return dict(codes=_scaled(w, s).to(_F8), scales=s)


def _unscaled(codes, scale):
    rows, d = codes.shape
    if scale.shape[0] != rows:
        scale = scale.repeat_interleave(128, 0)[:rows]
    return codes.float() * scale.repeat_interleave(128, 1)[:, :d]


def _plain_logits(st):
    x = _unscaled(st["codes"], st["scales"])
    w = _unscaled(st["weight_codes"], st["weight_scales"])
    return dict(logits=(x @ w.t()).to(_DT[st["case"]["out"]]))


def _bits(words, V):
    """The mask's truth values, a byte each."""
    b = words.view(torch.uint8)   # little-endian: bit v is bit v % 8 of byte v / 8
    on = (b[..., None] >> torch.arange(8, device=words.device, dtype=torch.uint8)) & 1
    return on.flatten(-2)[..., :V].bool()


def _plain_adjust(st):
    x = st["logits"]
    B, R, V = x.shape
    dev = x.device
    at = torch.arange(st["history"].shape[1], device=dev)[None, :]
    out_tok = (at < st["history_len"][:, None]) & (at >= st["prompt_len"][:, None])
    toks = st["history"].long()
    count = torch.zeros((B, V), device=dev).scatter_add_(1, toks, out_tok.float())
    prompt = torch.zeros((B, V), device=dev).scatter_add_(1, toks, (at < st["prompt_len"][:, None]).float())
    c = torch.zeros((B, R, V), device=dev)
    if R > 1:
        c[:, 1:].scatter_(2, st["draft_tokens"].long()[..., None], 1.0)
    c[:, 0] += count
    c = c.cumsum(1)
    z = x.float()
    p = st["repetition"][:, None, None]
    z = torch.where((c > 0) | (prompt > 0)[:, None], torch.where(z > 0, z / p, z * p), z)
    z = z - st["frequency"][:, None, None] * c
    z = z - torch.where(c > 0, st["presence"][:, None, None], 0.0)
    del c
    if st["bias"] is not None:
        offsets, ids, vals = st["bias"]
        row = torch.repeat_interleave(torch.arange(B, device=dev), (offsets[1:] - offsets[:-1]).long(), output_size=len(ids))
        b = torch.zeros((B, V), device=dev)
        b[row, ids.long()] = vals
        z = z + b[:, None]
    if st["mask"] is not None:
        idx = st["mask_index"].long()
        allowed = _bits(st["mask"], V)[idx.clamp(min=0)]
        z = torch.where(allowed | (idx < 0)[:, None, None], z, -math.inf)
        del allowed
    z = z.to(x.dtype)
    if st["lengths"] is not None:
        live = torch.arange(R, device=dev)[None, :] <= st["lengths"][:, None]
        z = torch.where(live[..., None], z, st["out"])
    return dict(logits=z, status=torch.zeros(B, dtype=torch.int32, device=dev))


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "weight": _plain_weight, "logits": _plain_logits,
            "adjust": _plain_adjust}[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        es, n = (2 if case["dtype"] == "bf16" else 4), case["N"] * case["d"]
        b = n * es * (3 if case["residual"] else 1)                          # x, residual and the sum
        b += n + 4 * n // 128 if case["q8"] else n * es + 4 * case["N"]
        if case["step"]:                                                     # grad_y, h, grad_x and the stream's own
            b += n * es * (4 if case["residual"] else 3)
        return dict(bytes=b, flops=n * (20 if case["step"] else 8))
    if case["op"] == "weight":
        n = case["V"] * case["d"]
        return dict(bytes=n * (3 if case["dtype"] == "bf16" else 5), flops=3 * n)
    if case["op"] == "logits":
        N, V, d = case["N"], case["V"], case["d"]
        return dict(bytes=V * d + N * d + (V // 128 + 4 * N) * (d // 128) + N * V * (2 if case["out"] == "bf16" else 4),
                    flops=2 * N * V * d)
    rows = case["B"] * (1 + case["gamma"] * (0.5 if case["ragged"] else 1.0))   # ragged lengths average gamma / 2
    b = rows * case["V"] * (4 if case["dtype"] == "bf16" else 8) + case["B"] * case["H"] * 3
    if case["masks"]:
        b += rows / 2 * case["V"] / 8
    return dict(bytes=int(b), flops=int(rows * case["V"] * 4))


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_codes(y, rows):
    """The values that the codes stand for, and the scales, block by block of the padded array."""
    n, d = y.shape
    n1, d1 = -(-n // rows) * rows, -(-d // 128) * 128
    full = torch.zeros((n1, d1), dtype=torch.float64, device=y.device)
    full[:n, :d] = y
    blocks = full.view(n1 // rows, rows, d1 // 128, 128)
    s = torch.clamp(blocks.abs().amax(dim=(1, 3)), min=_FLOOR) / 448.0
    q = (blocks / s[:, None, :, None]).view(n1, d1)[:n, :d]
    # e4m3: 3 bits behind the leading one, exponents down to 2^-6; halves to even
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(q / step) * step, s


def _exact_norm(st):
    case = st["case"]
    h, w = st["x"].double(), st["w"].double()
    if case["residual"]:
        h = h + st["residual"].double()
    norm = torch.sqrt(h.square().sum(dim=1) / h.shape[1] + _EPS)
    y = w[None, :] * (h / norm[:, None])
    r = {}
    if case["q8"]:
        r["codes"], r["scales"] = _exact_codes(y, 1)
    else:
        r["y"], r["rstd"] = y, 1.0 / norm
    if case["residual"]:
        r["h"] = h
    if case["step"]:
        gy = st["grad_y"].double()
        unit = h / norm[:, None]
        along = ((gy * w) * unit).sum(dim=1, keepdim=True) / h.shape[1]
        gx = (gy * w - unit * along) / norm[:, None]
        r["grad_x"] = gx + st["grad_h"].double() if case["residual"] else gx
        r["grad_w"] = torch.sum(gy * unit, dim=0)
    return r


def _exact_weight(st):
    w = st["weight"]
    parts = [_exact_codes(w[i:j].double(), 128) for i, j in _chunks(w.shape[0], w.shape[1])]
    return dict(codes=torch.cat([p[0].float() for p in parts]), scales=torch.cat([p[1] for p in parts]))


def _exact_logits(st):
    x, w = st["codes"].double(), st["weight_codes"].double()
    for k in range(st["scales"].shape[1]):
        x[:, 128 * k:128 * k + 128] *= st["scales"][:, k:k + 1].double()
    for v in range(st["weight_scales"].shape[0]):
        w[128 * v:128 * v + 128] *= st["weight_scales"][v].double().repeat_interleave(128)[:w.shape[1]]
    return dict(logits=torch.mm(x, w.t()))


def _exact_adjust(st):
    x = st["logits"]
    B, R, V = x.shape
    res = st["out"].double()
    for b in range(B):
        n, p = int(st["history_len"][b]), int(st["prompt_len"][b])
        line = st["history"][b, :n].long()
        seen = torch.zeros(V, dtype=torch.bool, device=x.device)
        seen[line] = True
        times = torch.bincount(line[p:], minlength=V).double()
        rep, freq, pres = (float(st[k][b]) for k in ("repetition", "frequency", "presence"))
        add = torch.zeros(V, dtype=torch.float64, device=x.device)
        if st["bias"] is not None:
            lo, hi = int(st["bias"][0][b]), int(st["bias"][0][b + 1])
            add[st["bias"][1][lo:hi].long()] = st["bias"][2][lo:hi].double()
        m = -1 if st["mask"] is None else int(st["mask_index"][b])
        last = R - 1 if st["lengths"] is None else int(st["lengths"][b])
        for k in range(last + 1):
            if k:
                tok = int(st["draft_tokens"][b, k - 1])
                seen[tok] = True
                times[tok] += 1
            z = x[b, k].double()
            z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
            z = z - freq * times - pres * (times > 0).double() + add
            if m >= 0:
                word = st["mask"][m, k].long()
                v = torch.arange(V, device=x.device)
                z[(word[v // 32] >> (v % 32)) % 2 == 0] = -math.inf
            res[b, k] = z
    return dict(logits=res, status=torch.zeros(B, dtype=torch.int32, device=x.device))


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "weight": _exact_weight, "logits": _exact_logits,
            "adjust": _exact_adjust}[case["op"]](st)
