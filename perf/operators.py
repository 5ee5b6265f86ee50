"""Cases that measure the drafter's training operators: the teacher's top logits, the distillation
loss on them and the cross entropy of a vocabulary head, each with its gradient.

`listed()` names the cases, `draw(rng)` makes one more of the same ranges, `prepare` builds a
case's inputs from a seed, `run` makes one pass (the plain form in elementary torch operations, or,
with `own`, the library's calls), `work` counts what a pass cannot do without and `exact` evaluates
the definition in 64 bits.

The operators, for rows of V logits:

  teacher  the K largest logits of every target row (value descending, id ascending) and
           ln sum exp(z / T) over the row;
  distill  KL(p || q) or the total variation of a teacher's top-K list p against the draft
           distribution q = softmax(z / T), with the teacher's mass outside the list renormalised
           away or kept as one bucket ("tail"); a "step" also forms the gradient;
  xent     cross entropy of softmax(H W^T) against labels (-1: ignored), without the logits being
           kept; a "step" also forms the gradients of H and W.

The draft blocks have the shapes [B, gamma, V] of verification, with a length per block.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one short block: the latency of a call
        dict(name="teacher_small", op="teacher", B=1, gamma=4, V=1000, dtype="f32", K=8, ragged=False),
        # the verification batch of 256 blocks of 16 whose lists are kept for training
        dict(name="teacher_batch", op="teacher", B=256, gamma=16, V=151936, dtype="bf16", K=64, ragged=True),
        # long lists from the second vocabulary, blocks of 7
        dict(name="teacher_long_list", op="teacher", B=96, gamma=7, V=129280, dtype="bf16", K=256, ragged=False),
        # evaluation of the loss on one short block: latency
        dict(name="distill_small", op="distill", B=1, gamma=4, V=1000, dtype="f32", K=8, mode="kl", tail=False,
             step=False, ragged=False),
        # a training step on 512 anchors, blocks of 7, the total-variation loss
        dict(name="distill_step_tv", op="distill", B=512, gamma=7, V=151936, dtype="bf16", K=64, mode="tv",
             tail=False, step=True, ragged=True),
        # the loss alone (validation) with the teacher's tail kept
        dict(name="distill_loss_tail", op="distill", B=128, gamma=16, V=129280, dtype="bf16", K=200, mode="kl",
             tail=True, step=False, ragged=False),
        # a step in fp32 on rows that do not start on a 16-byte boundary
        dict(name="distill_step_f32", op="distill", B=33, gamma=5, V=20011, dtype="f32", K=50, mode="kl",
             tail=True, step=True, ragged=True),
        # the head's loss for a few rows of a small vocabulary: latency
        dict(name="xent_small", op="xent", N=16, V=1000, d=256, dtype="bf16", step=False),
        # few rows against the whole vocabulary: bound by reading the weight once
        dict(name="xent_few_rows", op="xent", N=64, V=129280, d=4096, dtype="bf16", step=False),
        # a training step of a small drafter, odd row and vocabulary counts
        dict(name="xent_step_odd", op="xent", N=1791, V=20011, d=1024, dtype="bf16", step=True),
        # a step in fp32 on a small head
        dict(name="xent_step_f32", op="xent", N=500, V=8000, d=512, dtype="f32", step=True),
        # a training step on 256 blocks of 16: hidden width 4096 and a 256-wide Markov embedding beside it
        dict(name="xent_step_full", op="xent", N=4096, V=151936, d=4352, dtype="bf16", step=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["teacher", "distill", "xent"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "xent":
        while True:
            N, V = _log(rng, 1, 4096), _log(rng, 500, 151936)
            d = 8 * _log(rng, 8, 544)
            if N * V * d <= (4096 * 151936 * 4352 if dtype == "bf16" else 1024 * 32000 * 2048):
                return dict(op=op, N=N, V=V, d=d, dtype=dtype, step=rng.random() < 0.6)
    while True:
        B, gamma, V = _log(rng, 1, 512), rng.randint(1, 16), _log(rng, 300, 262144)
        if B * gamma * V <= 512 * 7 * 151936:
            break
    case = dict(op=op, B=B, gamma=gamma, V=V, dtype=dtype, K=_log(rng, 1, 256), ragged=rng.random() < 0.5)
    if op == "distill":
        case.update(mode=rng.choice(["kl", "tv"]), tail=rng.random() < 0.5, step=rng.random() < 0.6)
    return case


# ---- inputs ---------------------------------------------------------------------------------

def _chunks(n, per_row, limit=1 << 28):
    step = max(1, limit // max(1, per_row))
    return [(i, min(n, i + step)) for i in range(0, n, step)]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 17)
    dt = _DT[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "xent":
        N, V, d = case["N"], case["V"], case["d"]
        # unit hidden states and a weight that gives logits of standard deviation about 3
        st["hidden"] = torch.randn((N, d), generator=g, device=dev).to(dt)
        st["weight"] = torch.empty((V, d), dtype=dt, device=dev)
        for i, j in _chunks(V, d):
            st["weight"][i:j] = (torch.randn((j - i, d), generator=g, device=dev) * (3.0 / math.sqrt(d))).to(dt)
        labels = torch.randint(V, (N,), generator=g, device=dev)
        labels[torch.rand((N,), generator=g, device=dev) < 0.1] = -1
        st["labels"] = labels.to(torch.int32)
        pos = torch.arange(N, device=dev) % 7
        st["grad_loss"] = (torch.exp(-pos.float() / 7.0) / N)
        return st
    B, G, V, K = case["B"], case["gamma"], case["V"], case["K"]
    lengths = None
    if case["ragged"]:
        lengths = torch.randint(0, G + 1, (B,), generator=g, device=dev).to(torch.int32)
    st["lengths"] = lengths
    st["temperature"] = 0.6 + 0.6 * torch.rand((B,), generator=g, device=dev)
    if case["op"] == "teacher":
        st["target"] = torch.empty((B, G + 1, V), dtype=dt, device=dev)
        flat = st["target"].view(B * (G + 1), V)
        for i, j in _chunks(B * (G + 1), V):
            z = torch.randn((j - i, V), generator=g, device=dev) * 3.0
            z.scatter_add_(1, torch.randint(V, (j - i, 1), generator=g, device=dev),
                           torch.full((j - i, 1), 8.0, device=dev))
            flat[i:j] = z.to(dt)
        return st
    # distill: the teacher's rows are made, listed by torch.topk and dropped; the draft follows them
    st["draft"] = torch.empty((B, G, V), dtype=dt, device=dev)
    ids = torch.full((B * G, K), -1, dtype=torch.int32, device=dev)
    vals = torch.full((B * G, K), -math.inf, device=dev)
    tlse = torch.empty((B * G,), dtype=torch.float64, device=dev)
    flat = st["draft"].view(B * G, V)
    Trow = st["temperature"].repeat_interleave(G)
    for i, j in _chunks(B * G, V):
        z = torch.randn((j - i, V), generator=g, device=dev) * 2.0
        z.scatter_add_(1, torch.randint(V, (j - i, 1), generator=g, device=dev),
                       torch.full((j - i, 1), 8.0, device=dev))
        z = z.to(dt).float()
        top = torch.topk(z, min(K, V), dim=1)
        ids[i:j, :min(K, V)] = top.indices.to(torch.int32)
        vals[i:j, :min(K, V)] = top.values
        m = top.values[:, :1].double()
        e = torch.exp((z - top.values[:, :1]) / Trow[i:j, None])
        tlse[i:j] = torch.log(e.sum(1, dtype=torch.float64)) + m[:, 0] / Trow[i:j].double()
        flat[i:j] = (z + torch.randn((j - i, V), generator=g, device=dev) * 0.5).to(dt)
    st["ids"], st["values"] = ids.view(B, G, K), vals.view(B, G, K)
    st["teacher_lse"] = tlse.view(B, G).float() if case["tail"] else None
    w = torch.exp(-torch.arange(G, device=dev).float() / G)
    st["grad_loss"] = (w / (B * float(w.sum()))).expand(B, G).contiguous()
    return st


# ---- the library's calls --------------------------------------------------------------------

def _run_own(st):
    import draft_verification_04_amd as sv
    case = st["case"]
    if case["op"] == "teacher":
        o = sv.teacher_topk(st["target"], case["K"], st["lengths"], st["temperature"])
        return dict(ids=o["ids"], values=o["values"], lse=o["lse"], status=o["status"])
    if case["op"] == "distill":
        mode = sv.SPEC_DISTILL_KL if case["mode"] == "kl" else sv.SPEC_DISTILL_TV
        o = sv.distill_loss(st["draft"], st["ids"], st["values"], st["teacher_lse"], mode, st["lengths"],
                            st["temperature"])
        r = dict(loss=o["loss"], status=o["status"])
        if case["step"]:
            r["grad"] = sv.distill_loss_backward(st["draft"], st["ids"], st["values"], o["saved"], st["grad_loss"],
                                                 mode, st["temperature"])
        return r
    o = sv.head_xent(st["hidden"], st["weight"], st["labels"])
    r = dict(loss=o["loss"], lse=o["lse"], status=o["status"])
    if case["step"]:
        b = sv.head_xent_backward(st["hidden"], st["weight"], st["labels"], o["lse"], st["grad_loss"])
        r["grad_hidden"], r["grad_weight"] = b["grad_hidden"], b["grad_weight"]
    return r


# ---- the plain form -------------------------------------------------------------------------

def _live(lengths, B, G, dev):
    k = torch.arange(G, device=dev)
    return torch.ones((B, G), dtype=torch.bool, device=dev) if lengths is None else k[None, :] < lengths[:, None]


def _plain_teacher(st):
    x, K = st["target"], st["case"]["K"]
    B, G1, V = x.shape
    G, dev = G1 - 1, x.device
    live = _live(st["lengths"], B, G, dev)
    ids = torch.full((B, G, K), -1, dtype=torch.int32, device=dev)
    vals = torch.full((B, G, K), -math.inf, device=dev)
    lse = torch.full((B, G), -math.inf, device=dev)
    n = min(K, V)
    low = (V - 1 - torch.arange(V, device=dev, dtype=torch.int64))
    for i, j in _chunks(B, G * V):
        z = x[i:j, :G].float() + 0.0   # -0 becomes 0: the two are equal
        # a key of 64 bits that orders by value, then by the lower id
        u = z.view(torch.int32).to(torch.int64)
        u = torch.where(u < 0, -(u + 2 ** 31) - 1, u)
        top = torch.topk((u << 20) | low, n, dim=2).values
        t = V - 1 - (top & (2 ** 20 - 1))
        v = torch.gather(z, 2, t)
        T = st["temperature"][i:j, None, None]
        m = v[..., :1]
        e = torch.exp((z - m) / T)
        s = torch.log(e.sum(2, dtype=torch.float64)) + (m[..., 0].double() / T[..., 0].double())
        on = live[i:j]
        ids[i:j, :, :n] = torch.where(on[..., None], t, -1).to(torch.int32)
        vals[i:j, :, :n] = torch.where(on[..., None], v, -math.inf)
        lse[i:j] = torch.where(on, s, -math.inf).float()
    return dict(ids=ids, values=vals, lse=lse, status=torch.zeros(B, dtype=torch.int32, device=dev))


def _plain_distill(st):
    case, x, ids, vals = st["case"], st["draft"], st["ids"], st["values"]
    B, G, V = x.shape
    dev = x.device
    live = _live(st["lengths"], B, G, dev)
    loss = torch.zeros((B, G), device=dev)
    grad = torch.zeros((B, G, V), dtype=x.dtype, device=dev) if case["step"] else None
    for i, j in _chunks(B, G * V):
        z = x[i:j].float()
        T = st["temperature"][i:j, None, None]
        T64 = T.double()
        use = (ids[i:j] >= 0) & (vals[i:j] > -math.inf)
        at = ids[i:j].clamp(min=0).long()
        v = torch.where(use, vals[i:j], -math.inf).double() / T64
        tn = torch.logsumexp(v, 2) if st["teacher_lse"] is None else st["teacher_lse"][i:j].double()
        p = torch.exp(v - tn[..., None])
        m = z.amax(2, keepdim=True)
        e = torch.exp((z - m) / T)
        # the list in 64 bits, the rest of the row summed in 64 bits without it
        el = torch.where(use, torch.exp((torch.gather(z, 2, at).double() - m.double()) / T64), 0.0)
        inlist = torch.zeros(z.shape, device=dev)
        inlist.scatter_add_(2, at, use.float())
        out = torch.where(inlist > 0, 0.0, e).sum(2, dtype=torch.float64)
        tot = out + el.sum(2)
        q, rs = el / tot[..., None], out / tot
        rt = (1.0 - p.sum(2)).clamp(min=0.0) if case["tail"] else torch.zeros_like(rs)
        if case["mode"] == "kl":
            lo = torch.where(p > 0, p * (torch.log(p) - torch.log(q)), 0.0).sum(2)
            lo = lo + torch.where(rt > 0, rt * (torch.log(rt) - torch.log(rs)), 0.0)
            a, b, c = 1.0 - torch.where(rt > 0, rt / rs, 0.0), torch.ones_like(rs), p
        else:
            up, tup = p > q, (rt > rs).double()
            lo = torch.where(up, p - q, 0.0).sum(2) + (rt - rs).clamp(min=0.0)
            b = torch.where(up, q, 0.0).sum(2) + tup * rs
            a, c = b - tup, torch.where(up, q, 0.0)
        loss[i:j] = torch.where(live[i:j], lo, 0.0).float()
        if case["step"]:
            s = torch.where(live[i:j], st["grad_loss"][i:j].double() / T64[..., 0], 0.0)
            d = e * (s * a / tot).float()[..., None]
            dl = (s[..., None] * (q * b[..., None] - c)).float()
            # unused entries point at token 0 with weight 0
            d = torch.where(inlist > 0, 0.0, d).scatter_add_(2, at, torch.where(use, dl, 0.0))
            grad[i:j] = d.to(x.dtype)
    r = dict(loss=loss, status=torch.zeros(B, dtype=torch.int32, device=dev))
    if case["step"]:
        r["grad"] = grad
    return r


def _plain_xent(st):
    h, w, y = st["hidden"].float(), st["weight"].float(), st["labels"]
    z = h @ w.t()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, dtype=torch.float64)
    lse = torch.log(s) + m[:, 0].double()
    used = y >= 0
    at = y.clamp(min=0).long()[:, None]
    loss = torch.where(used, lse - torch.gather(z, 1, at)[:, 0].double(), 0.0).float()
    r = dict(loss=loss, lse=lse.float(), status=torch.zeros(len(y), dtype=torch.int32, device=y.device))
    if st["case"]["step"]:
        del z
        g = torch.where(used, st["grad_loss"], 0.0)[:, None]
        p = e / s.float()[:, None]
        p.scatter_add_(1, at, -torch.ones_like(g))
        p = p * g
        r["grad_hidden"] = (p @ w).to(st["hidden"].dtype)
        r["grad_weight"] = (p.t() @ h).to(st["weight"].dtype)
    return r


def run(state):
    if own:
        return _run_own(state)
    return {"teacher": _plain_teacher, "distill": _plain_distill, "xent": _plain_xent}[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "xent":
        N, V, d = case["N"], case["V"], case["d"]
        b = N * d * es + V * d * es + N * 16
        # a step forms the logits' product once for the loss and once more for the gradient (they are not kept)
        return dict(bytes=b * (2 if case["step"] else 1), flops=N * V * d * (8 if case["step"] else 2))
    rows = case["B"] * case["gamma"] * (0.5 if case["ragged"] else 1.0)   # ragged lengths average gamma / 2
    V, K = case["V"], case["K"]
    b = rows * V * es + rows * (8 * K + 8)
    if case["op"] == "distill" and case["step"]:
        b += rows * V * es + case["B"] * case["gamma"] * V * es   # read again; every row of the gradient is written
    return dict(bytes=int(b), flops=int(rows * V * (8 if case.get("step") else 4)))


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_teacher(st):
    x, K = st["target"], st["case"]["K"]
    B, G1, V = x.shape
    out_ids, out_vals, out_lse = [], [], []
    for b in range(B):
        L = G1 - 1 if st["lengths"] is None else int(st["lengths"][b])
        ids = torch.full((G1 - 1, K), -1, dtype=torch.int32, device=x.device)
        vals = torch.full((G1 - 1, K), -math.inf, device=x.device)
        lse = torch.full((G1 - 1,), -math.inf, dtype=torch.float64, device=x.device)
        if L:
            z = x[b, :L].double()
            order = torch.sort(z, dim=1, descending=True, stable=True)
            n = min(K, V)
            ids[:L, :n] = order.indices[:, :n].to(torch.int32)
            vals[:L, :n] = order.values[:, :n].float()
            lse[:L] = torch.logsumexp(z / float(st["temperature"][b]), 1)
        out_ids.append(ids)
        out_vals.append(vals)
        out_lse.append(lse)
    return dict(ids=torch.stack(out_ids), values=torch.stack(out_vals), lse=torch.stack(out_lse),
                status=torch.zeros(B, dtype=torch.int32, device=x.device))


def _exact_distill(st):
    case, x = st["case"], st["draft"]
    B, G, V = x.shape
    loss = torch.zeros((B, G), dtype=torch.float64, device=x.device)
    grad = torch.zeros((B, G, V), dtype=torch.float64, device=x.device) if case["step"] else None
    for b in range(B):
        L = G if st["lengths"] is None else int(st["lengths"][b])
        if L == 0:
            continue
        T = float(st["temperature"][b])
        logq = torch.log_softmax(x[b, :L].double() / T, 1)
        k = min(case["K"], V)
        at = st["ids"][b, :L, :k].long()
        tv = st["values"][b, :L, :k].double() / T
        if case["tail"]:
            logp = tv - st["teacher_lse"][b, :L, None].double()
            rt = torch.clamp(1.0 - torch.exp(logp).sum(1), min=0.0)
        else:
            logp = torch.log_softmax(tv, 1)
            rt = torch.zeros(L, dtype=torch.float64, device=x.device)
        outside = torch.ones_like(logq).scatter_(1, at, 0.0)
        q = torch.exp(logq)
        rs = (q * outside).sum(1)
        p, lq = torch.exp(logp), torch.gather(logq, 1, at)
        ql = torch.exp(lq)
        if case["mode"] == "kl":
            t = torch.where(rt > 0, rt * (torch.log(rt) - torch.log(rs)), 0.0)
            loss[b, :L] = (p * (logp - lq)).sum(1) + t
            # dL/dq of each token: -p/q in the list, -rt/rs outside it
            dq = outside * (-torch.where(rt > 0, rt / rs, 0.0))[:, None]
            dq.scatter_(1, at, -p / ql)
        else:
            loss[b, :L] = torch.relu(p - ql).sum(1) + torch.relu(rt - rs)
            dq = outside * (-(rt > rs).double())[:, None]
            dq.scatter_(1, at, -(p > ql).double())
        if case["step"]:
            # through the softmax: q (dq - sum q dq), then the temperature and the incoming gradient
            dz = q * (dq - (q * dq).sum(1, keepdim=True))
            grad[b, :L] = dz * (st["grad_loss"][b, :L, None].double() / T)
    r = dict(loss=loss, status=torch.zeros(B, dtype=torch.int32, device=x.device))
    if case["step"]:
        r["grad"] = grad
    return r


def _exact_xent(st):
    h, w, y = st["hidden"].double(), st["weight"].double(), st["labels"].long()
    logp = torch.mm(h, w.t())
    lse = torch.logsumexp(logp, 1)
    logp -= lse[:, None]
    rows = torch.nonzero(y >= 0)[:, 0]
    loss = torch.zeros(len(y), dtype=torch.float64, device=y.device)
    loss[rows] = -logp[rows, y[rows]]
    r = dict(loss=loss, lse=lse, status=torch.zeros(len(y), dtype=torch.int32, device=y.device))
    if st["case"]["step"]:
        gz = logp.exp_()
        gz[rows, y[rows]] -= 1.0
        weight = torch.zeros(len(y), dtype=torch.float64, device=y.device)
        weight[rows] = st["grad_loss"].double()[rows]
        gz *= weight[:, None]
        r["grad_hidden"] = torch.mm(gz, w)
        r["grad_weight"] = torch.mm(gz.t(), h)
    return r


def exact(case, seed):
    st = prepare(case, seed)
    return {"teacher": _exact_teacher, "distill": _exact_distill, "xent": _exact_xent}[case["op"]](st)
