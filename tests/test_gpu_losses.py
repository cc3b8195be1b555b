"""GPU parity of the vocabulary losses (dspark_ce_*, dspark_distill_*) against
oracle.training.

Exact cases.  With hidden = 0 (or every weight 0) the logits are 0, the softmax is 1 / V
for every entry, and d logits are two known numbers per row; against small whole numbers
every product is a multiple of one power of two, so where the sum of magnitudes is below
2^24 of it the fp32 partial sums are exact and d hidden (or a weight gradient) is one
rounding of a number the test computes; a longer sum is off by its fp32 additions, (K / 4 +
40) u times the sum of magnitudes, before that rounding.  These pin the tiles, operand
layouts, edges and pieces.

Tolerances elsewhere.  u = 2^-24.  A logit is off by at most zerr = (K / 4 + 40) u zabs (an
MFMA adds to its accumulator at least four products of fp32, thirty-two of bf16, at a
time; zabs is the sum of the products' magnitudes) and the loss by 2 zerr T plus 64 u
(1 + |lse| + ...) of the exponentials, logarithms and row sums.  A softmax entry has
then relative error ep = 2 zerr / T + 64 u (1 + |lse| + max |z| / T).  d logits are off by
gp ep + rnd |dz|, rnd being the storage rounding (bf16 2^-8, in two terms 2^-16; fp32 u), which
the product carries to sum |.| |operand|; its own sums add (K / 4 + 40) u times the sum of magnitudes
and the output one more rounding.  Below the normal range, where an exponential or a
product of fp32 or bf16 may come out as 0, each number is off by at most TINY = 2^-126: d logits
by that (each term), and a product of K of them by TINY (K + sum |operand|) at most.
"""
import numpy as np
import pytest

import oracle
from oracle import training as T
from workloads import synth
from gpu_util import dev, host_bits, log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TINY = 2.0 ** -126
RND = {"bf16": 2.0 ** -8, "f32": U}
LABEL_ROWS = 512     # of up to this many, weight gradients get the rounding of the label's entry back
TWO_TERM_ROWS = 64   # bf16 d logits of up to this many rows are a sum of two bf16 terms
ALL = ("hidden", "lm_head_w", "markov_w1", "markov_w2")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


def dz_rnd(dtype, rows):
    """Relative rounding of d logits: half a step, of the first term's half step for the second."""
    return RND[dtype] ** 2 if dtype == "bf16" and rows <= TWO_TERM_ROWS else RND[dtype]


def bdr():
    import block_draft_readout_amd as m
    return m


def _st(a, dtype):
    return synth.store(np.ascontiguousarray(a, dtype=np.float32), dtype)


def _opt(a):
    return None if a is None else dev(a)


def _case(seed, N, H, V, r, dtype, top=0, empty=0.2):
    g = np.random.default_rng(seed)
    c = dict(dtype=dtype, N=N, V=V, hidden=_st(g.standard_normal((N, H)), dtype),
             w=_st(g.standard_normal((V, H)) * 2 / np.sqrt(H), dtype), w1=None, w2=None, prev=None,
             g=(g.random(N) + 0.2).astype(np.float32))
    if r:
        c["w1"] = _st(g.standard_normal((V, r)), dtype)
        c["w2"] = _st(g.standard_normal((V, r)) * 0.3, dtype)
        c["prev"] = np.where(g.random(N) < 0.4, g.integers(0, max(1, V // 50), N),
                             g.integers(-1, V + 1, N)).astype(np.int32)
    out = g.random(N) < empty
    if top:
        ids = g.integers(0, V, (N, top))
        if top > 1:
            ids[:, 1] = np.where(g.random(N) < 0.3, ids[:, 0], ids[:, 1])   # an id twice
        bad = (g.random((N, top)) < 0.2) | out[:, None]
        c["ids"] = np.where(bad, g.choice([-1, V, -(2 ** 31), 2 ** 31 - 1], (N, top)), ids).astype(np.int32)
        u = g.standard_normal((N, top)) * 2
        u = np.where(g.random((N, top)) < 0.05, -np.inf, u)
        c["u"] = np.where(bad, np.nan, u).astype(np.float32)
    else:
        c["labels"] = np.where(out, g.choice([-100, -1, V, 2 ** 31 - 1], N), g.integers(0, V, N)).astype(np.int32)
        if N > 1:
            c["labels"][1] = V - 1
    return c


def _markov(c):
    return dict(markov_w1=_opt(c["w1"]), markov_w2=_opt(c["w2"]), prev_token=_opt(c["prev"]))


def _run(c, temp=1.0, grads=None, udt=torch.float32):
    """(loss, lse, picked or None, gradients) of the library's calls."""
    m = bdr()
    x, w, g, mk = dev(c["hidden"]), dev(c["w"]), dev(c["g"]), _markov(c)
    if "labels" in c:
        lab = dev(c["labels"])
        loss, lse = m.dspark_ce_loss(x, w, lab, **mk)
        return loss, lse, None, m.dspark_ce_backward(x, w, lab, lse, g, grads=grads, **mk)
    ids, u = dev(c["ids"]), dev(c["u"]).to(udt)
    loss, lse, picked = m.dspark_distill_loss(x, w, ids, u, temperature=temp, **mk)
    return loss, lse, picked, m.dspark_distill_backward(x, w, ids, u, lse, picked, g,
                                                        temperature=temp, grads=grads, **mk)


def _oracle(c, temp=1.0, **kw):
    t = dict(labels=c["labels"]) if "labels" in c else dict(ids=c["ids"], u=c["u"], T=temp)
    return T.loss(c["hidden"], c["w"], c["dtype"], w1=c["w1"], w2=c["w2"], prev=c["prev"],
                  loss_grad=c["g"], **t, **kw)


def _np(t, dtype=None):
    return oracle.widen(host_bits(t), dtype) if dtype else t.cpu().numpy().astype(np.float64)


def _within(name, got, ref, tol):
    err = np.abs(got - ref)
    ok = err <= tol
    assert ok.all(), (name, np.argwhere(~ok)[:3].tolist(), float(np.nanmax(err / np.maximum(tol, 1e-300))))
    return float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0


def _check(c, temp=1.0, udt=torch.float32):
    dtype, rnd = c["dtype"], RND[c["dtype"]]
    loss, lse, picked, grads = _run(c, temp, udt=udt)
    o = _oracle(c, temp)
    live = o["live"]
    H = c["hidden"].shape[1] + (c["w1"].shape[1] if c["w1"] is not None else 0)
    zerr = (H / 4 + 40) * U * o["zabs"]
    mag = 1 + np.abs(o["lse"]) + o["zabs"] / temp
    ep = 2 * zerr / temp + 64 * U * mag
    got = _np(loss)
    assert not got[~live].any() and not _np(lse)[~live].any()
    logt = 0.0
    if picked is not None:
        t = T.teacher_targets(c["ids"], c["u"], c["V"], temp)
        logt = np.abs(np.log(np.where(t > 0, t, 1.0))).max(axis=1)
        pk = _np(picked)
        assert not pk[o["picked"] == 0].any()
        _within("picked", pk, o["picked"], zerr[:, None] + U)
    worst = [_within("lse", _np(lse), o["lse"], (zerr / temp + 64 * U * mag) * live),
             _within("loss", got, o["loss"], temp * temp * (ep + 64 * U * (mag + logt)) * live)]
    E = o["gp"] * ep[:, None] + (dz_rnd(dtype, c["N"]) + 4 * U) * np.abs(o["dz"]) + 2 * TINY * live[:, None]
    W = np.abs(oracle.widen(c["w"], dtype))
    X = np.where(live[:, None], np.abs(oracle.widen(c["hidden"], dtype)), 0.0)
    N, V = c["N"], c["V"]
    moved = dict(hidden=E @ W, lm_head_w=E.T @ X)
    if c["w1"] is not None:
        W2 = np.abs(oracle.widen(c["w2"], dtype))
        has = (c["prev"] >= 0) & (c["prev"] < V) & live
        e = np.zeros((N, W2.shape[1]))
        e[has] = np.abs(oracle.widen(c["w1"], dtype))[c["prev"][has]]
        d1 = np.zeros_like(W2)
        np.add.at(d1, c["prev"][has], (E @ W2)[has])
        moved.update(markov_w1=d1, markov_w2=E.T @ e)
    chain = dict(hidden=V, lm_head_w=N, markov_w1=V + 4 * N, markov_w2=N)
    assert set(grads) == set(moved)
    for k, v in grads.items():
        tol = moved[k] + (chain[k] / 4 + 40) * U * o["abs_" + k] + rnd * np.abs(o[k])
        tol = tol + TINY * chain[k]
        worst.append(_within(k, _np(v, dtype), o[k], tol))
        if k == "hidden":
            assert not _np(v, dtype)[~live].any()
    return max(worst)


CE = [("f32", 1, 4, 1, 0), ("f32", 5, 64, 1000, 8), ("f32", 60, 64, 1000, 0), ("f32", 33, 132, 257, 128),
      ("f32", 200, 36, 2600, 4), ("f32", 130, 260, 129, 12),
      ("bf16", 1, 8, 2, 0), ("bf16", 1, 72, 1000, 8), ("bf16", 7, 320, 4001, 32), ("bf16", 64, 64, 127, 64),
      ("bf16", 129, 136, 2561, 24), ("bf16", 300, 520, 1031, 128), ("bf16", 513, 200, 517, 0),
      ("bf16", 31, 1000, 5003, 40), ("bf16", 50, 72, 61501, 8), ("bf16", 100, 136, 61501, 0),
      ("bf16", 290, 72, 31003, 16)]


@pytest.mark.parametrize("dtype,N,H,V,r", CE)
def test_cross_entropy(dtype, N, H, V, r):
    w = _check(_case(N * 31 + V, N, H, V, r, dtype, empty=0.0 if N == 1 else 0.2))
    log(f"ce {dtype} {N}x{H} V={V} r={r}: worst error / tolerance {w:.3f}")


DISTILL = [("f32", 5, 64, 1000, 8, 4, 1.0), ("f32", 70, 36, 300, 0, 256, 2.0), ("f32", 40, 68, 65, 4, 65, 0.5),
           ("bf16", 1, 72, 1000, 8, 1, 1.0), ("bf16", 19, 320, 4001, 32, 20, 2.0),
           ("bf16", 140, 136, 2561, 24, 64, 1.0), ("bf16", 300, 264, 1031, 128, 7, 3.5),
           ("bf16", 65, 64, 2, 0, 3, 1.0)]


@pytest.mark.parametrize("dtype,N,H,V,r,top,temp", DISTILL)
def test_distillation(dtype, N, H, V, r, top, temp):
    w = _check(_case(N * 17 + V, N, H, V, r, dtype, top=top, empty=0.0 if N == 1 else 0.2), temp)
    log(f"distill {dtype} {N}x{H} V={V} r={r} top={top} T={temp}: worst error / tolerance {w:.3f}")


def test_distillation_with_bf16_teacher_logits():
    c = _case(5, 33, 64, 500, 8, "bf16", top=9)
    keep = np.isfinite(c["u"])
    c["u"][keep] = oracle.widen(synth.to_bf16_bits(c["u"][keep]), "bf16")
    _check(c, 1.5, udt=torch.bfloat16)


FLAT = [(1, 64, 256, 8), (3, 200, 1000, 0), (130, 328, 2560, 64), (257, 72, 130, 16), (40, 2568, 5000, 128),
        (700, 136, 3001, 8), (16, 640, 20011, 32), (61, 328, 61501, 8), (125, 136, 61501, 8),
        (1601, 136, 16501, 8)]


@pytest.mark.parametrize("N,H,V,r", FLAT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_flat_softmax_is_exact(N, H, V, r, dtype):
    """hidden = 0: d hidden = (mean of W - W[label]) g; then W = 0: d W from whole hidden."""
    g = np.random.default_rng(N + V)
    small = lambda *s: _st(g.integers(-3, 4, s), dtype)
    prev = g.integers(0, min(V, 5), N).astype(np.int32)
    labels = np.where(g.random(N) < 0.2, -1, g.integers(0, V, N)).astype(np.int32)
    gr = 2.0 ** g.integers(-2, 3, N).astype(np.float32)
    live = labels >= 0
    p = 1.0 / V
    rd = T.round_bf16 if dtype == "bf16" else lambda a: np.asarray(a, np.float32).astype(np.float64)
    # the two values of d logits / g, which powers of two scale exactly.  (p - 1 in fp32 depends on
    # the last bit of p; only bf16's values are pinned exactly, far from a rounding border.)
    one_term = dtype == "bf16" and N > TWO_TERM_ROWS
    lo, hi = (float(rd(p)), float(rd(p - 1.0))) if one_term else (p, p - 1.0)
    for v in (p, p - 1.0):
        if one_term:
            assert rd(v * (1 + 1e-5)) == rd(v * (1 - 1e-5))
    base = dict(dtype=dtype, N=N, V=V, prev=prev if r else None, labels=labels, g=gr)
    zero = lambda *s: _st(np.zeros(s), dtype)
    def dlogits(hi):
        one = np.zeros((N, V))
        one[live] = lo
        one[live, labels[live]] = hi
        return one * gr[:, None]

    # the label's entry: in one term its rounding comes back in fp32 to d hidden and d w1, and to
    # the weights' gradients up to LABEL_ROWS rows
    dz = dlogits(p - 1.0)
    dzw = dlogits(hi if one_term and N > LABEL_ROWS else p - 1.0)
    # fp32 and two terms: p is off by at most 64 u (lse, two exponentials) and the storage's
    # rounding; everything else is exact
    off = 0.0 if one_term else 128 * U + dz_rnd(dtype, N)

    # every product is a multiple of this: 8 bits of lo (hi has a larger last bit), the smallest g
    last = 2.0 ** (np.floor(np.log2(p)) - 7) * float(gr.min())

    def same(name, got, ref, mags, K, whole):
        # whole: rows of the gradient that no label's entry in fp32 reaches
        err = np.abs(_np(got, dtype) - ref)
        sums = (K / 4 + 40) * U * mags
        tol = np.where(whole[:, None], off, 128 * U + (0.0 if one_term else off)) * mags
        assert (err <= RND[dtype] * np.abs(ref) + sums + tol).all(), name
        if one_term:
            exact = (mags < 2.0 ** 24 * last) & whole[:, None]
            assert np.array_equal(_np(got, dtype)[exact], T.round_bf16(ref)[exact]), name

    w, w1z, w2 = small(V, H), zero(V, r) if r else None, small(V, r) if r else None
    gr1 = _run(dict(base, hidden=zero(N, H), w=w, w1=w1z, w2=w2))[3]
    Wd, adz = oracle.widen(w, dtype), np.abs(dz)
    same("hidden", gr1["hidden"], dz @ Wd, adz @ np.abs(Wd), V, ~live)
    if r:
        d1, a1 = np.zeros((V, r)), np.zeros((V, r))
        np.add.at(d1, prev, dz @ oracle.widen(w2, dtype))
        np.add.at(a1, prev, adz @ np.abs(oracle.widen(w2, dtype)))
        same("markov_w1", gr1["markov_w1"], d1, a1, V + 4 * N, ~a1.any(axis=1))
        assert not gr1["markov_w2"].any()
    x, w1 = small(N, H), small(V, r) if r else None
    gr2 = _run(dict(base, hidden=x, w=zero(V, H), w1=w1, w2=zero(V, r) if r else None))[3]
    Xd, adz = oracle.widen(x, dtype), np.abs(dzw)
    whole = np.ones(V, dtype=bool)
    if N <= LABEL_ROWS:
        whole[labels[live]] = False
    same("lm_head_w", gr2["lm_head_w"], dzw.T @ Xd, adz.T @ np.abs(Xd), N, whole)
    if r:
        Ed = oracle.widen(w1, dtype)[prev]
        same("markov_w2", gr2["markov_w2"], dzw.T @ Ed, adz.T @ np.abs(Ed), N, whole)
    assert not gr2["hidden"].any()


@pytest.mark.parametrize("dtype,N,H,V,r", [("bf16", 26000, 64, 12000, 8), ("bf16", 53000, 136, 5121, 8),
                                            ("f32", 27000, 16, 5121, 8)])
def test_several_pieces_match_one(dtype, N, H, V, r):
    """Enough rows that the backward pass walks the vocabulary in pieces (the last one a single
    entry in the second and third case): the same gradients as the rows in two halves give, up to
    the order of sums and the roundings of the halves."""
    g = torch.Generator(device="cuda").manual_seed(1)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = rn(N, H).to(t)
    w = (rn(V, H) / 8).to(t)
    w1, w2 = rn(V, r).to(t), (rn(V, r) * 0.3).to(t)
    lab = torch.randint(-1, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    prev = torch.randint(-1, 40, (N,), generator=g, device="cuda", dtype=torch.int32)
    lg = torch.rand(N, generator=g, device="cuda") / N
    m = bdr()
    dt = m.BDR_BF16 if dtype == "bf16" else m.BDR_F32
    assert m.lib().dspark_ce_workspace_bytes(N, H, V, r, dt, 1) < N * V * (2 if dtype == "bf16" else 4)
    mk = dict(markov_w1=w1, markov_w2=w2)
    loss, lse = m.dspark_ce_loss(x, w, lab, prev_token=prev, **mk)
    whole = m.dspark_ce_backward(x, w, lab, lse, lg, prev_token=prev, **mk)
    k = N // 2
    parts = []
    for s in (slice(0, k), slice(k, N)):
        l2, e2 = m.dspark_ce_loss(x[s], w, lab[s], prev_token=prev[s], **mk)
        assert torch.equal(l2, loss[s]) and torch.equal(e2, lse[s])
        parts.append(m.dspark_ce_backward(x[s], w, lab[s], e2, lg[s], prev_token=prev[s], **mk))
    # the same d logits; fp32 sums in another order (1e-5 of the largest is far above K u of any
    # element's magnitudes), then one rounding each: half a step of the values on either side
    rnd, far = RND[dtype], 1e-5

    def near(a, b, mags):
        assert ((a - b).abs() <= rnd * mags + far * b.abs().max()).all()

    hid = torch.cat([p["hidden"] for p in parts]).float()
    near(hid, whole["hidden"].float(), 2 * hid.abs())
    for name in ("lm_head_w", "markov_w1", "markov_w2"):
        a, b = (p[name].float() for p in parts)
        near(a + b, whole[name].float(), a.abs() + b.abs() + whole[name].float().abs())


@pytest.mark.parametrize("top", [0, 6])
def test_rows_left_out_may_hold_anything(top):
    c = _case(11, 50, 136, 700, 16, "bf16", top=top, empty=0.4)
    live = _oracle(c)["live"]
    ref = _run(c)
    d = dict(c, hidden=c["hidden"].copy(), g=c["g"].copy(), prev=c["prev"].copy())
    d["hidden"][~live] = 0x7FFF          # NaN
    d["g"][~live] = np.nan
    d["prev"][~live] = 2 ** 31 - 1
    got = _run(d)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    for k in ref[3]:
        assert torch.equal(ref[3][k], got[3][k]), k
    # and wherever they stand: the rows with a target first, the others after them, is the same
    # product.  (As many rows in all: the tiles, and so the order of sums, go by that number.)
    order = np.concatenate([np.flatnonzero(live), np.flatnonzero(~live)])
    e = {k: (v[order] if k in ("hidden", "g", "prev", "labels", "ids", "u") else v) for k, v in c.items()}
    got = _run(e)
    back = torch.from_numpy(order).cuda()
    assert torch.equal(ref[0][back], got[0]) and torch.equal(ref[3]["hidden"][back], got[3]["hidden"])
    for k in ("lm_head_w", "markov_w1", "markov_w2"):
        assert torch.equal(ref[3][k], got[3][k]), k


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_row_with_a_target_and_no_rows(top, dtype):
    c = _case(13, 21, 64, 300, 8, dtype, top=top, empty=1.1)
    if not top:
        c["labels"][:] = -1
    loss, lse, picked, grads = _run(c)
    assert not loss.any() and not lse.any() and (picked is None or not picked.any())
    for k, v in grads.items():
        assert not v.any(), k
    z = {k: (v[:0] if k in ("hidden", "g", "prev", "labels", "ids", "u") else v) for k, v in c.items()}
    z["N"] = 0
    loss, lse, picked, grads = _run(z)
    assert loss.shape == (0,) and grads["hidden"].shape == (0, 64)
    for k in ("lm_head_w", "markov_w1", "markov_w2"):
        assert not grads[k].any()


def test_nothing_to_learn_in_the_large_tiles():
    """No row with a target where the weight gradient's workgroups walk their tiles."""
    c = _case(14, 21, 640, 20011, 32, "bf16", empty=1.1)
    c["labels"][:] = -1
    _, _, _, grads = _run(c)
    for k, v in grads.items():
        assert not v.any(), k


def test_single_gradients_equal_the_joint_call():
    c = _case(15, 90, 200, 900, 24, "bf16")
    full = _run(c)[3]
    for k in ALL:
        assert torch.equal(_run(c, grads=(k,))[3][k], full[k]), k
    again = _run(c)[3]
    for k in ALL:
        assert torch.equal(again[k], full[k]), k


def test_every_row_the_same_previous_token():
    c = _case(16, 600, 64, 150, 40, "f32", empty=0.1)
    c["prev"][:] = 149
    _check(c)


def test_large_logits_stay_finite():
    """Logits of +-200: the running maximum keeps every exponential in range."""
    c = _case(18, 20, 64, 400, 0, "f32", empty=0.0)
    c["w"] *= np.float32(40)
    loss, lse, _, grads = _run(c)
    o = _oracle(c)
    assert o["zabs"].max() > 300 and torch.isfinite(loss).all()
    _check(c)


def test_captured_and_replayed_on_another_stream():
    m = bdr()
    a, b = (_case(s, 70, 136, 1500, 16, "bf16", empty=0.3) for s in (20, 21))
    d = _case(22, 70, 136, 1500, 16, "bf16", top=5, empty=0.3)
    x, w, lab, prev, g = (dev(a[k]) for k in ("hidden", "w", "labels", "prev", "g"))
    ids, u = dev(d["ids"]), dev(d["u"])
    w1, w2 = dev(a["w1"]), dev(a["w2"])
    mk = dict(markov_w1=w1, markov_w2=w2, prev_token=prev)
    L = m.lib()
    n = max(L.dspark_ce_workspace_bytes(70, 136, 1500, 16, m.BDR_BF16, 1),
            L.dspark_distill_workspace_bytes(70, 136, 1500, 16, 5, m.BDR_BF16, 1))
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")

    def step():
        loss, lse = m.dspark_ce_loss(x, w, lab, workspace=ws, **mk)
        gr = m.dspark_ce_backward(x, w, lab, lse, g, workspace=ws, **mk)
        l2, e2, pk = m.dspark_distill_loss(x, w, ids, u, temperature=2.0, workspace=ws, **mk)
        g2 = m.dspark_distill_backward(x, w, ids, u, e2, pk, g, temperature=2.0, workspace=ws, **mk)
        return [loss, lse, l2, e2, pk, *(gr[k] for k in ALL), *(g2[k] for k in ALL)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k, c in enumerate((b, a, b)):
        x.copy_(dev(c["hidden"]))
        lab.copy_(dev(c["labels"]))
        prev.copy_(dev(c["prev"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for i, (p, q) in enumerate(zip(got, step())):
            assert torch.equal(p, q), (k, i)


def test_two_streams_at_once():
    """Calls that share inputs but no workspace, in flight together."""
    m = bdr()
    c = _case(24, 400, 264, 30011, 16, "bf16", empty=0.2)
    d = _case(25, 50, 264, 30011, 16, "bf16", top=8, empty=0.2)
    serial = [_run(c), _run(d, 2.0)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        both = []
        for st, (k, t) in zip(s, ((c, 1.0), (d, 2.0))):
            with torch.cuda.stream(st):
                both.append(_run(k, t))
        torch.cuda.synchronize()
        for a, b in zip(serial, both):
            assert torch.equal(a[0], b[0])
            for n in a[3]:
                assert torch.equal(a[3][n], b[3][n]), n
    assert m is not None


@pytest.mark.parametrize("N,H,V,r", [(5, 2560, 60001, 16), (60, 2560, 60001, 32), (100, 2560, 60001, 0),
                                     (60, 2568, 60001, 0), (100, 2568, 60001, 8), (128, 2624, 60033, 8)])
def test_one_row_of_tiles_over_a_large_weight(N, H, V, r):
    """Few rows and a weight larger than the caches, with rows of whole cache lines and rows that
    end inside one: the float64 reference and the tolerances of _check, on the device."""
    m = bdr()
    g = torch.Generator(device="cuda").manual_seed(N + H)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w = rn(N, H).bfloat16(), (rn(V, H) * 2 / H ** 0.5).bfloat16()
    lab = torch.randint(-V // 5, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    lab[0] = V - 1
    gr = torch.rand(N, generator=g, device="cuda") + 0.2
    mk = {}
    if r:
        mk = dict(markov_w1=rn(V, r).bfloat16(), markov_w2=(rn(V, r) * 0.3).bfloat16(),
                  prev_token=torch.randint(-1, 40, (N,), generator=g, device="cuda", dtype=torch.int32))
    loss, lse = m.dspark_ce_loss(x, w, lab, **mk)
    got = m.dspark_ce_backward(x, w, lab, lse, gr, **mk)
    live = lab >= 0
    X, W = x.double() * live[:, None], w.double()
    z, zabs = X @ W.t(), X.abs() @ W.abs().t()
    if r:
        prev = mk["prev_token"].long()
        has = (prev >= 0) & live
        e = mk["markov_w1"].double()[prev.clamp(min=0)] * has[:, None]
        W2 = mk["markov_w2"].double()
        z, zabs = z + e @ W2.t(), zabs + e.abs() @ W2.abs().t()
    zabs = zabs.max(dim=1).values
    ref = torch.logsumexp(z, dim=1)
    at = lab.long().clamp(min=0)[:, None]
    zerr = ((H + r) / 4 + 40) * U * zabs
    mag = 1 + ref.abs() + zabs
    ep = 2 * zerr + 64 * U * mag
    assert ((lse.double() - ref * live).abs() <= (zerr + 64 * U * mag) * live).all()
    assert ((loss.double() - (ref - z.gather(1, at)[:, 0]) * live).abs() <= (ep + 64 * U * mag) * live).all()
    gp = (z - ref[:, None]).exp() * (gr.double() * live)[:, None]
    dz = gp.clone()
    dz.scatter_add_(1, at, -(gr.double() * live)[:, None])
    E = gp * ep[:, None] + (dz_rnd("bf16", N) + 4 * U) * dz.abs() + 2 * TINY * live[:, None]

    def near(name, want, moved, mags, K):
        tol = moved + (K / 4 + 40) * U * mags + RND["bf16"] * want.abs() + TINY * K
        assert ((got[name].double() - want).abs() <= tol).all(), name

    near("hidden", dz @ W, E @ W.abs(), dz.abs() @ W.abs(), V)
    assert not got["hidden"][~live].any()
    near("lm_head_w", dz.t() @ X, E.t() @ X.abs(), dz.abs().t() @ X.abs(), N)
    if r:
        near("markov_w2", dz.t() @ e, E.t() @ e.abs(), dz.abs().t() @ e.abs(), N)
        rows = prev.clamp(min=0)

        def d1(a):
            return torch.zeros(V, r, dtype=torch.float64, device="cuda").index_add_(0, rows, a * has[:, None])

        near("markov_w1", d1(dz @ W2), d1(E @ W2.abs()), d1(dz.abs() @ W2.abs()), V + 4 * N)


def test_weights_beyond_32_bit_offsets():
    """2^21 entries of 1032 features: 4.3 GB of weight and as much gradient.  The loss and the rows
    of d W that the last entries get, against float64 on the device."""
    m = bdr()
    N, H, V = 3, 1032, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 1 << 18):
        w[a:a + (1 << 18)] = torch.randn(1 << 18, H, generator=g, device="cuda") / 32
    x = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    lab = torch.tensor([V - 1, 0, V - 2], dtype=torch.int32, device="cuda")
    one = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    loss, lse = m.dspark_ce_loss(x, w, lab)
    gr = m.dspark_ce_backward(x, w, lab, lse, one)
    z = torch.cat([x.double() @ w[a:a + (1 << 18)].double().t() for a in range(0, V, 1 << 18)], dim=1)
    ref = torch.logsumexp(z, dim=1)
    zabs = max(float((x.double().abs() @ w[a:a + (1 << 18)].double().abs().t()).max())
               for a in range(0, V, 1 << 18))
    zerr = (H / 4 + 40) * U * zabs
    assert (lse.double() - ref).abs().max() <= zerr + 64 * U * (1 + float(ref.abs().max()))
    pick = z.gather(1, lab.long()[:, None])[:, 0]
    assert (loss.double() - (ref - pick)).abs().max() <= 2 * zerr + 64 * U * (1 + float(ref.abs().max()))
    dz = (z - ref[:, None]).exp_()
    dz[torch.arange(N), lab.long()] -= 1
    dz *= one.double()[:, None]
    for lo, hi in ((0, 4), (V - 1000, V)):
        want = dz[:, lo:hi].t() @ x.double()
        mags = dz[:, lo:hi].abs().t() @ x.double().abs()
        p = dz[:, lo:hi].abs() + torch.where(dz[:, lo:hi] < 0, one.double()[:, None], 0.0)
        ep = 2 * zerr + 64 * U * (1 + float(ref.abs().max()) + zabs)
        tol = (ep * p.t() @ x.double().abs()) + 2.0 ** -8 * (mags + want.abs()) + TINY * N
        assert ((gr["lm_head_w"][lo:hi].double() - want).abs() <= tol).all()
    dh = sum(dz[:, a:a + (1 << 18)] @ w[a:a + (1 << 18)].double() for a in range(0, V, 1 << 18))
    ah = sum(dz[:, a:a + (1 << 18)].abs() @ w[a:a + (1 << 18)].double().abs() for a in range(0, V, 1 << 18))
    # d logits' rounding and the softmax's error against the sum of magnitudes, V / 4 fp32 additions
    tol = (2.0 ** -8 + 2 * zerr + (V / 4 + 40) * U) * ah + 2.0 ** -8 * dh.abs()
    assert ((gr["hidden"].double() - dh).abs() <= tol).all()


def test_refusals():
    m = bdr()
    c = _case(30, 6, 64, 100, 8, "bf16")
    x, w, lab, mk = dev(c["hidden"]), dev(c["w"]), dev(c["labels"]), _markov(c)
    with pytest.raises(ValueError):
        m.dspark_ce_loss(x.t(), w, lab, **mk)
    with pytest.raises(ValueError):
        m.dspark_ce_loss(x[:, :32], w, lab, **mk)
    with pytest.raises(TypeError):
        m.dspark_ce_loss(x, w, lab.long(), **mk)
    with pytest.raises(TypeError):
        m.dspark_ce_loss(x.half(), w.half(), lab)
    with pytest.raises(ValueError):
        m.dspark_ce_loss(x, w, lab[:5], **mk)
    with pytest.raises(ValueError):
        m.dspark_ce_loss(x, w, lab, markov_w1=mk["markov_w1"])
    with pytest.raises(ValueError):
        m.dspark_ce_loss(x, w, lab, markov_w1=mk["markov_w1"], markov_w2=mk["markov_w2"])
    with pytest.raises(m.BdrError):
        m.dspark_ce_loss(x, w, lab, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    loss, lse = m.dspark_ce_loss(x, w, lab, **mk)
    with pytest.raises(ValueError):
        m.dspark_ce_backward(x, w, lab, lse, lse, grads=("head",), **mk)
    with pytest.raises(ValueError):
        m.dspark_ce_backward(x, w, lab, lse, lse, grads=("markov_w1",))
    with pytest.raises(m.BdrError):
        m.dspark_ce_backward(x, w, lab, lse, lse, grads=(), **mk)
    with pytest.raises(m.BdrError):
        m.dspark_distill_loss(x, w, lab[:, None].contiguous(), lse[:, None].contiguous(), temperature=0.0)


@pytest.mark.parametrize("dtype,top", [("f32", 0), ("bf16", 0), ("f32", 3), ("bf16", 3)])
def test_many_rows(dtype, top):
    """Rows counted block by block before the compaction (the last block ends inside), and a
    previous token that first appears thousands of rows in."""
    c = _case(60 + top, 9001, 8, 130, 8, dtype, top=top)
    c["prev"][c["prev"] == 77] = 0
    for n, tok in ((7000, 77), (8990, 77)):
        c["prev"][n] = tok
        if top:
            c["ids"][n, 0], c["u"][n, 0] = 5, 0.5
        else:
            c["labels"][n] = 5
    _check(c, 1.5 if top else 1.0)


def test_small_temperature_keeps_close_teacher_logits_apart():
    """hidden = 0 and W = 1 on the diagonal: d hidden is d logits itself, g T (1 / V - t).  The
    teacher's logits differ by a few steps of fp32, which T = 1e-4 makes differences of up to
    19 in the exponent.

    t: the division's rounding and that of the sum add at most u (2 d / T + top) and the
    exponential a few u; the other factors a few u each: 64 u (1 + max d / T) covers them
    (u top = 40 u).  The product only adds zeros."""
    m = bdr()
    V = H = 128
    N, top, temp = 33, 40, float(np.float32(1e-4))
    gn = np.random.default_rng(8)
    step = gn.integers(0, 2001, (N, top))
    u = (8.0 + step * 2.0 ** -20).astype(np.float32)
    ids = np.stack([gn.permutation(V)[:top] for _ in range(N)]).astype(np.int32)
    gr = (gn.random(N) + 0.5).astype(np.float32)
    x = torch.zeros((N, H), dtype=torch.float32, device="cuda")
    w = torch.eye(V, dtype=torch.float32, device="cuda")
    _, lse, picked = m.dspark_distill_loss(x, w, dev(ids), dev(u), temperature=temp)
    got = _np(m.dspark_distill_backward(x, w, dev(ids), dev(u), lse, picked, dev(gr), temperature=temp,
                                        grads=("hidden",))["hidden"])
    t = T.teacher_targets(ids, u, V, temp)
    target = np.zeros((N, V))
    np.put_along_axis(target, ids.astype(np.int64), t, axis=1)
    scale = gr.astype(np.float64)[:, None] * temp
    big = 64 * U * (1 + 2000 * 2.0 ** -20 / temp)
    _within("d hidden", got, scale * (1 / V - target), scale * big * (1 / V + target) + TINY)


def test_training_step_of_the_readout():
    """norm -> cross entropy -> backward through both, as a drafter trains them, against
    differences of the summed loss along random directions (fp32).

    The five-point difference with step h is off by the loss's own error (each value within
    loss_err of the exact loss) over h and by h^4 |fifth derivative| / 30, which the change
    from 2 h to h bounds: the sum of both is the tolerance."""
    m = bdr()
    N, H, V, r = 24, 64, 500, 8
    c = _case(40, N, H, V, r, "f32")
    x, w, lab, g, mk = dev(c["hidden"]), dev(c["w"]), dev(c["labels"]), dev(c["g"]), _markov(c)
    gn = np.random.default_rng(41)
    nw, nb = dev((1 + 0.1 * gn.standard_normal(H)).astype(np.float32)), dev((0.1 * gn.standard_normal(H)).astype(np.float32))

    def loss(x, w, nw, nb, w1, w2):
        y = m.dspark_norm(x, nw, nb, eps=1e-5)
        l, _ = m.dspark_ce_loss(y, w, lab, markov_w1=w1, markov_w2=w2, prev_token=mk["prev_token"])
        return float((l.double() * g.double()).sum())

    y, mean, rstd = m.dspark_norm(x, nw, nb, eps=1e-5, stats=True)
    l, lse = m.dspark_ce_loss(y, w, lab, **mk)
    gr = m.dspark_ce_backward(y, w, lab, lse, g, **mk)
    dx, dnw, dnb = m.dspark_norm_backward(gr["hidden"], x, nw, mean, rstd)
    args = [x, w, nw, nb, mk["markov_w1"], mk["markov_w2"]]
    zabs = float((y.abs() @ w.abs().t()).max()) + r
    loss_err = float(g.sum()) * (2 * (H / 4 + 60) * U * zabs + 128 * U * (1 + zabs))
    for i, d in enumerate((dx, gr["lm_head_w"], dnw, dnb, gr["markov_w1"], gr["markov_w2"])):
        v = dev(gn.standard_normal(tuple(d.shape)).astype(np.float32))
        v *= float(d.abs().sum() and 1.0) / float(v.norm())

        def diff(h):
            f = [loss(*(a + k * h * v if j == i else a for j, a in enumerate(args))) for k in (-2, -1, 1, 2)]
            return (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h)

        h = 0.25
        d1, d2 = diff(h), diff(2 * h)
        want = float((d.double() * v.double()).sum())
        tol = 1.5 * loss_err / h + abs(d1 - d2)
        log(f"direction {i}: gradient {want:.6f}, difference {d1:.6f}, tolerance {tol:.2e}")
        assert abs(want - d1) <= tol
