"""Timed cases of the drafter's training operators: the row normalisation in front of the LM
head, the cross entropy over the full vocabulary and the distillation from a teacher's top
logits, each forward and backward, with the Markov bias in the logits.

Where ``own`` is false ``run`` computes them in their plain form with elementary torch
operations in 32 bits; where it is true it makes the calls a user makes of
``block_draft_readout_amd``.

Formulas (rows n, vocabulary v, features h, rank j; all sums over the whole axis):

    norm      y = (x - mean) * rstd * w + b, rstd = (var + eps)^-1/2; the root-mean-square
              form takes mean = 0
    logits    z[n, v] = sum_h hidden[n, h] W[v, h] + sum_j w1[prev[n], j] w2[v, j]
              (a previous token outside [0, V) adds nothing)
    cross entropy of row n with label y (a label outside [0, V): loss and lse 0, no gradient)
              loss = lse - z[y], lse = log sum_v exp z[v];  dz = g (softmax(z) - onehot(y))
    distillation at temperature T from entries (id_j, u_j) (an id outside [0, V) is left out)
              t = softmax_j(u / T), lse = log sum_v exp(z[v] / T)
              loss = T^2 sum_j t_j (log t_j - (z[id_j] / T - lse))
              dz = g T (softmax(z / T) - sum_j t_j onehot(id_j))
    gradients d hidden = dz W, d W = dz^T hidden, d w2 = dz^T w1[prev],
              d w1[p] = sum_{n : prev[n] = p} dz[n] w2
"""
import math

import torch

own = False

EPS = 1e-6


def _bdr():
    import block_draft_readout_amd
    return block_draft_readout_amd


def _norm(name, rows, hidden, dtype, rms, step):
    return dict(name=name, op="norm", rows=rows, hidden=hidden, dtype=dtype, rms=rms, step=step)


def _ce(name, rows, hidden, vocab, rank, dtype, step, head, ignored):
    return dict(name=name, op="ce", rows=rows, hidden=hidden, vocab=vocab, rank=rank, dtype=dtype,
                step=step, head=head, ignored=ignored)


def _distill(name, rows, hidden, vocab, rank, dtype, step, head, ignored, top, temperature):
    return dict(name=name, op="distill", rows=rows, hidden=hidden, vocab=vocab, rank=rank,
                dtype=dtype, step=step, head=head, ignored=ignored, top=top,
                temperature=temperature)


def listed():
    return [
        # one token in front of the LM head while serving: latency
        _norm("norm_1x5120_bf16", 1, 5120, "bf16", False, False),
        # an odd number of rows of an fp32 model, forward and backward
        _norm("norm_step_1023x1000_f32", 1023, 1000, "f32", False, True),
        # a training batch of 4096 positions, forward and backward
        _norm("norm_step_4096x5120_bf16", 4096, 5120, "bf16", False, True),
        # a large batch of the narrower drafter, root-mean-square form
        _norm("rms_step_16381x2560_bf16", 16381, 2560, "bf16", True, True),
        # the fp32 drafter of the tests: launches, not bytes
        _ce("ce_step_60x64_v1000_f32", 60, 64, 1000, 8, "f32", True, True, 0.1),
        # scoring one drafted block of seven positions against given tokens
        _ce("ce_score_7x5120_bf16", 7, 5120, 151936, 32, "bf16", False, False, 0.0),
        # training on the 16 x 8 positions of one batched block-step, head included
        _ce("ce_step_128x5120_bf16", 128, 5120, 151936, 64, "bf16", True, True, 0.0),
        # a training batch of 4096 positions, a quarter of them prompt (no loss), head trained
        _ce("ce_step_4096x5120_bf16", 4096, 5120, 151936, 64, "bf16", True, True, 0.25),
        # the narrower drafter on a larger odd batch, the target's head shared and frozen
        _ce("ce_frozen_8191x2560_bf16", 8191, 2560, 151936, 32, "bf16", True, False, 0.25),
        # distillation loss of a single position (monitoring while serving)
        _distill("distill_score_1x5120_bf16", 1, 5120, 151936, 32, "bf16", False, False, 0.0, 20,
                 1.0),
        # a ragged batch and vocabulary, head trained, softened teacher
        _distill("distill_step_1000x2560_bf16", 1000, 2560, 131071, 32, "bf16", True, True, 0.1,
                 20, 2.0),
        # 4096 positions against 64 stored teacher logits each, head frozen
        _distill("distill_frozen_4096x5120_bf16", 4096, 5120, 151936, 64, "bf16", True, False,
                 0.25, 64, 1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("norm", "ce", "distill", "ce", "distill"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    step = rng.random() < 0.75
    if op == "norm":
        return dict(op=op, rows=_log_int(rng, 1, 16381), hidden=8 * _log_int(rng, 8, 640),
                    dtype=dtype, rms=rng.random() < 0.5, step=step)
    rows = _log_int(rng, 1, 4096)
    hidden = 8 * _log_int(rng, 8, 640)
    vocab = _log_int(rng, 1000, 151936)
    if dtype == "f32":   # fp32 models are small ones
        rows, hidden, vocab = min(rows, 1024), min(hidden, 1024), min(vocab, 32768)
    case = dict(op=op, rows=rows, hidden=hidden, vocab=vocab,
                rank=rng.choice((0, 8, 32, 64, 8 * rng.randint(1, 16))), dtype=dtype, step=step,
                head=rng.random() < 0.5, ignored=round(rng.uniform(0.0, 0.5), 3))
    if op == "distill":
        case.update(top=_log_int(rng, 1, 128), temperature=round(rng.uniform(0.5, 4.0), 3))
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n, h = case["rows"], case["hidden"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        # residual-stream rows: a common offset, a row scale and a few large features
        x = normal(n, h) * (0.5 + uniform(n, 1) * 2) + 0.3 * normal(1, h)
        x[:, :: max(1, h // 8)] *= 8
        s = dict(case=case, x=x.to(dt), w=(1 + normal(h, std=0.1)).to(dt),
                 b=None if case["rms"] else normal(h, std=0.1).to(dt))
        if case["step"]:
            s["dy"] = normal(n, h, std=1 / math.sqrt(n)).to(dt)
        return s
    v, r = case["vocab"], case["rank"]
    w = normal(v, h, std=1 / math.sqrt(h)).to(dt)
    s = dict(case=case, w=w, w1=None, w2=None, prev=None)
    if r:
        s["w1"] = normal(v, r).to(dt)
        s["w2"] = normal(v, r, std=math.sqrt(0.1 / r * 8)).to(dt)
        # previous tokens: common ones repeat; a few positions have none
        prev = (uniform(n) ** 4 * v).long().clamp_(max=v - 1)
        s["prev"] = torch.where(uniform(n) < 0.03, -1, prev).int()
    # hidden states that raise the wanted token's logit by 0 to 12
    want = (uniform(n) ** 2 * v).long().clamp_(max=v - 1)
    x = normal(n, h) + 12 * uniform(n, 1) * w[want].float()
    s["x"] = x.to(dt)
    left_out = uniform(n) < case["ignored"]
    if case["op"] == "ce":
        s["labels"] = torch.where(left_out, -100, want).int()
    else:
        # the teacher's K best entries: distinct ids, common ones more often, the wanted
        # token first; some lists are shorter (id -1), rows left out have an empty one
        k = min(case["top"], v)
        at = (uniform(n, k) ** 3 * (v - k + 1)).long().clamp_(max=v - k).sort(dim=1).values
        ids = at + torch.arange(k, device="cuda")
        ids = ids.gather(1, uniform(n, k).argsort(dim=1))
        first = torch.where((ids == want[:, None]).any(dim=1), ids[:, 0], want)
        ids[:, 0] = first
        u = (normal(n, k) * 3 + 12).sort(dim=1, descending=True).values
        u[:, 0] += 4 * uniform(n)
        kept = (1 + uniform(n) * 2 * k).long().clamp_(max=k)
        gone = (torch.arange(k, device="cuda") >= kept[:, None]) | left_out[:, None]
        s["ids"] = torch.where(gone, -1, ids).int()
        s["u"] = torch.where(gone, torch.finfo(torch.float32).min, u)
    if case["step"]:
        # the gradient of a weighted mean over the rows
        s["g"] = (0.5 + uniform(n)) / n
    return s


def _grad_names(case):
    names = ["hidden"]
    if case["head"]:
        names.append("lm_head_w")
    if case["rank"]:
        names += ["markov_w1", "markov_w2"]
    return tuple(names)


def _run_own(s):
    bdr, c = _bdr(), s["case"]
    if c["op"] == "norm":
        if not c["step"]:
            return bdr.dspark_norm(s["x"], s["w"], s["b"], eps=EPS, rms=c["rms"])
        y, mean, rstd = bdr.dspark_norm(s["x"], s["w"], s["b"], eps=EPS, rms=c["rms"], stats=True)
        dx, dw, db = bdr.dspark_norm_backward(s["dy"], s["x"], s["w"], mean, rstd,
                                              bias=not c["rms"])
        return dict(y=y, dx=dx, dw=dw, db=db)
    markov = dict(markov_w1=s["w1"], markov_w2=s["w2"], prev_token=s["prev"])
    if c["op"] == "ce":
        loss, lse = bdr.dspark_ce_loss(s["x"], s["w"], s["labels"], **markov)
        if not c["step"]:
            return dict(loss=loss, lse=lse)
        grads = bdr.dspark_ce_backward(s["x"], s["w"], s["labels"], lse, s["g"],
                                       grads=_grad_names(c), **markov)
    else:
        loss, lse, picked = bdr.dspark_distill_loss(s["x"], s["w"], s["ids"], s["u"],
                                                    temperature=c["temperature"], **markov)
        if not c["step"]:
            return dict(loss=loss)
        grads = bdr.dspark_distill_backward(s["x"], s["w"], s["ids"], s["u"], lse, picked, s["g"],
                                            temperature=c["temperature"], grads=_grad_names(c),
                                            **markov)
    return dict(loss=loss, **grads)


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    mean = x.new_zeros(x.shape[0], 1) if c["rms"] else x.mean(dim=1, keepdim=True)
    xc = x - mean
    rstd = ((xc * xc).mean(dim=1, keepdim=True) + EPS).rsqrt()
    xh = xc * rstd
    y = xh * w
    if s["b"] is not None:
        y = y + s["b"].float()
    if not c["step"]:
        return y.to(dt)
    dy = s["dy"].float()
    gy = dy * w
    inner = gy - xh * (gy * xh).mean(dim=1, keepdim=True)
    if not c["rms"]:
        inner = inner - gy.mean(dim=1, keepdim=True)
    return dict(y=y.to(dt), dx=(inner * rstd).to(dt), dw=(dy * xh).sum(dim=0).to(dt),
                db=None if c["rms"] else dy.sum(dim=0).to(dt))


def _plain_loss(s):
    c = s["case"]
    dt = s["x"].dtype
    v = s["w"].shape[0]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if c["rank"]:
        prev = s["prev"].long()
        has = ((prev >= 0) & (prev < v))[:, None]
        prev = prev.clamp(0, v - 1)
        w2 = s["w2"].float()
        e = torch.where(has, s["w1"].float()[prev], 0.0)
        z = z + e @ w2.t()
    temp = c.get("temperature", 1.0)
    if temp != 1.0:
        z = z / temp
    top = z.max(dim=1).values
    lse = top + (z - top[:, None]).exp().sum(dim=1).log()
    if c["op"] == "ce":
        ids = s["labels"].long()[:, None]
        valid = (ids >= 0) & (ids < v)
        t = valid.float()
    else:
        ids = s["ids"].long()
        valid = (ids >= 0) & (ids < v)
        u = torch.where(valid, s["u"] / temp, -math.inf)
        best = u.max(dim=1, keepdim=True).values
        best = torch.where(best == -math.inf, 0.0, best)
        t = (u - best).exp()
        total = t.sum(dim=1, keepdim=True)
        t = t / torch.where(total > 0, total, 1.0)
    ids = ids.clamp(0, v - 1)
    logp = z.gather(1, ids) - lse[:, None]
    entropy = torch.where(t > 0, t * t.clamp(min=1e-38).log(), 0.0)
    loss = temp * temp * torch.where(valid, entropy - t * logp, 0.0).sum(dim=1)
    counts = valid.any(dim=1) if c["op"] == "ce" else total[:, 0] > 0
    if not c["step"]:
        return dict(loss=loss, lse=torch.where(counts, lse, 0.0)) if c["op"] == "ce" else dict(loss=loss)
    g = torch.where(counts, s["g"], 0.0) * temp
    z = (z - lse[:, None]).exp_()
    z.scatter_add_(1, ids, -t)
    z *= g[:, None]
    out = dict(loss=loss, hidden=(z @ w).to(dt))
    if c["head"]:
        out["lm_head_w"] = (z.t() @ x).to(dt)
    if c["rank"]:
        de = torch.where(has, z @ w2, 0.0)
        d1 = torch.zeros(v, c["rank"], device=z.device).index_put_((prev,), de, accumulate=True)
        out["markov_w1"] = d1.to(dt)
        out["markov_w2"] = (z.t() @ e).to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    return _plain_norm(state) if state["case"]["op"] == "norm" else _plain_loss(state)


def work(case):
    n, h, c = case["rows"], case["hidden"], case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        vec = (1 if c["rms"] else 2) * h * e
        if not c["step"]:
            return dict(bytes=2 * n * h * e + vec, flops=6.0 * n * h)
        # x, dy in; y, dx out; the vectors in and their gradients out
        return dict(bytes=4 * n * h * e + vec + vec, flops=16.0 * n * h)
    v, r = c["vocab"], c["rank"]
    live = n * (1 - c["ignored"])
    given = 8 * n * c["top"] if c["op"] == "distill" else 4 * n
    read = (n * h + v * h + (v + min(n, v)) * r) * e + given + (4 * n if r else 0)
    if not c["step"]:
        return dict(bytes=read + 8 * n, flops=2.0 * live * v * (h + r))
    wrote = (n * h + (v * h if c["head"] else 0) + 2 * v * r) * e + 4 * n
    # logits, d hidden and, where the head is trained, d W; the Markov head's three likewise
    products = 2.0 * live * v * (h * (3 if c["head"] else 2) + 3 * r)
    return dict(bytes=read + wrote + 4 * n, flops=products)


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions, in blocks of rows."""
    s = prepare(case, seed)
    d = torch.float64
    x = s["x"].to(d)
    n, h = x.shape
    if case["op"] == "norm":
        w = s["w"].to(d)
        mean = torch.zeros(n, dtype=d, device=x.device) if case["rms"] else x.sum(1) / h
        xc = x - mean[:, None]
        sigma = torch.sqrt((xc ** 2).sum(1) / h + EPS)
        y = xc / sigma[:, None] * w
        if s["b"] is not None:
            y += s["b"].to(d)
        if not case["step"]:
            return y
        dy = s["dy"].to(d)
        # y = xc w / sigma:  dx = dy w / sigma - xc (xc . dy w) / (h sigma^3), less the mean
        dxc = dy * w / sigma[:, None] - xc * ((xc * dy * w).sum(1) / (h * sigma ** 3))[:, None]
        dx = dxc if case["rms"] else dxc - dxc.sum(1, keepdim=True) / h
        dw = (xc / sigma[:, None] * dy).sum(0)
        return dict(y=y, dx=dx, dw=dw, db=None if case["rms"] else dy.sum(0))
    v, r = case["vocab"], case["rank"]
    T = case.get("temperature", 1.0)
    full = s["w"].to(d)
    feats = x
    if r:
        prev = s["prev"].long()
        emb = torch.zeros(n, r, dtype=d, device=x.device)
        has = (prev >= 0) & (prev < v)
        emb[has] = s["w1"].to(d)[prev[has]]
        feats = torch.cat([x, emb], dim=1)
        full = torch.cat([full, s["w2"].to(d)], dim=1)
    loss = torch.zeros(n, dtype=d, device=x.device)
    lses = torch.zeros(n, dtype=d, device=x.device)
    dfeats = torch.zeros_like(feats)
    dfull = torch.zeros_like(full) if case["step"] and (case["head"] or r) else None
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        z = feats[a:b] @ full.t() / T
        lse = torch.logsumexp(z, dim=1)
        target = torch.zeros_like(z)
        if case["op"] == "ce":
            y = s["labels"][a:b].long()
            rows = torch.nonzero((y >= 0) & (y < v))[:, 0]
            target[rows, y[rows]] = 1.0
        else:
            ids, u = s["ids"][a:b].long(), s["u"][a:b].to(d)
            ok = (ids >= 0) & (ids < v)
            u = torch.where(ok, u / T, torch.full_like(u, -math.inf))
            rows = torch.nonzero(ok.any(dim=1))[:, 0]
            t = torch.zeros_like(u)
            t[rows] = torch.softmax(u[rows], dim=1)
            target.scatter_add_(1, ids.clamp(0, v - 1), t)
        logp = z - lse[:, None]
        # sum t log t - sum t log p over the entries that have mass
        cross = torch.special.xlogy(target, target).sum(1) - (target * logp).sum(1)
        loss[a + rows] = T * T * cross[rows]
        lses[a + rows] = lse[rows]
        if case["step"]:
            scale = torch.zeros(b - a, dtype=d, device=x.device)
            scale[rows] = s["g"][a:b].to(d)[rows] * T
            dz = (logp.exp_() - target) * scale[:, None]
            dfeats[a:b] = dz @ full
            if dfull is not None:
                dfull += dz.t() @ feats[a:b]
        del z, target, logp
    if not case["step"]:
        return dict(loss=loss, lse=lses) if case["op"] == "ce" else dict(loss=loss)
    out = dict(loss=loss, hidden=dfeats[:, :h])
    if case["head"]:
        out["lm_head_w"] = dfull[:, :h]
    if r:
        d1 = torch.zeros(v, r, dtype=d, device=x.device)
        d1.index_add_(0, prev[has], dfeats[has, h:])
        out["markov_w1"] = d1
        out["markov_w2"] = dfull[:, h:]
    return out
