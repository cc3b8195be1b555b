"""Float64 oracle of the drafter's training operators: the row normalisation, the cross
entropy over the full vocabulary and the distillation from a teacher's top logits, with
their gradients.

Arrays are in the storage convention (bf16 as uint16 bit patterns); everything is
widened exactly to float64 and nothing is rounded, except where ``round_dlogits`` asks
for the one rounding the operators document: d logits rounded to bf16 before they enter
the gradients' products.
"""
from __future__ import annotations

import numpy as np

from .reference import widen


def norm(x, w, b, dtype, eps, rms=False):
    """(y, mean, rstd) with mean None for the root-mean-square form."""
    x, w = widen(x, dtype), widen(w, dtype)
    mean = np.zeros(x.shape[0]) if rms else x.mean(axis=1)
    xc = x - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).mean(axis=1) + eps)
    y = xc * rstd[:, None] * w
    if b is not None:
        y = y + widen(b, dtype)
    return y, (None if rms else mean), rstd


def norm_backward(dy, x, w, dtype, eps, rms=False):
    """(dx, dw, db) of sum(dy * y)."""
    _, mean, rstd = norm(x, w, None, dtype, eps, rms)
    x, w, dy = widen(x, dtype), widen(w, dtype), widen(dy, dtype)
    xh = (x if rms else x - mean[:, None]) * rstd[:, None]
    gy = dy * w
    dx = gy - xh * (gy * xh).mean(axis=1, keepdims=True)
    if not rms:
        dx = dx - gy.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)


def round_bf16(x):
    """float64 -> nearest bf16 value (ties to even), as float64; normal range."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def teacher_targets(ids, u, V, T):
    """t [rows, top]: softmax over the listed entries of u / T; zeros for a row without mass."""
    ids = np.asarray(ids, dtype=np.int64)
    ok = (ids >= 0) & (ids < V)
    s = np.where(ok, np.asarray(u, dtype=np.float64) / T, -np.inf)
    t = np.zeros(s.shape)
    for n in range(s.shape[0]):
        mx = s[n].max() if s.shape[1] else -np.inf
        if mx > -np.inf:
            e = np.exp(s[n] - mx)
            t[n] = e / e.sum()
    return t


def _features(hidden, w, w1, w2, prev, dtype):
    x, W = widen(hidden, dtype), widen(w, dtype)
    V = W.shape[0]
    if w1 is None:
        return x, W, np.zeros((x.shape[0], 0)), np.zeros((V, 0)), None
    prev = np.asarray(prev, dtype=np.int64)
    has = (prev >= 0) & (prev < V)
    e = np.zeros((x.shape[0], np.asarray(w1).shape[1]))
    e[has] = widen(w1, dtype)[prev[has]]
    return x, W, e, widen(w2, dtype), np.where(has, prev, -1)


def loss(hidden, w, dtype, labels=None, ids=None, u=None, T=1.0, w1=None, w2=None, prev=None,
         loss_grad=None, round_dlogits=False):
    """The loss values and, with loss_grad [rows], the gradients.

    labels [rows]: cross entropy (T = 1); ids / u [rows, top]: distillation.  Returns a
    dict: live (rows that have a target), loss, lse (0 for the others), picked
    (distillation), zabs (per row, the largest sum of |products| of a logit: what its
    fp32 error scales with), gp (loss_grad T softmax), dz and the gradients hidden, lm_head_w, markov_w1,
    markov_w2, and for each product its sum of magnitudes under "abs_" + name.
    """
    x, W, e, W2, prevc = _features(hidden, w, w1, w2, prev, dtype)
    N, V = x.shape[0], W.shape[0]
    if labels is not None:
        lab = np.asarray(labels, dtype=np.int64)
        live = (lab >= 0) & (lab < V)
        target = np.zeros((N, V))
        target[live, lab[live]] = 1.0
    else:
        t = teacher_targets(ids, u, V, T)
        live = t.sum(axis=1) > 0
        target = np.zeros((N, V))
        ii = np.asarray(ids, dtype=np.int64)
        for n in range(N):
            ok = (ii[n] >= 0) & (ii[n] < V)
            np.add.at(target[n], ii[n][ok], t[n][ok])
    x = np.where(live[:, None], x, 0.0)     # rows that are left out may hold anything
    e = np.where(live[:, None], e, 0.0)
    z = x @ W.T + e @ W2.T
    s = z / T
    mx = s.max(axis=1)
    lse = mx + np.log(np.exp(s - mx[:, None]).sum(axis=1))
    out = dict(live=live, lse=np.where(live, lse, 0.0),
               zabs=(np.abs(x) @ np.abs(W).T + np.abs(e) @ np.abs(W2).T).max(axis=1))
    if labels is not None:
        at = np.where(live, lab, 0)
        out["loss"] = np.where(live, lse - z[np.arange(N), at], 0.0)
    else:
        ok = (ii >= 0) & (ii < V) & live[:, None]
        picked = np.where(ok, np.take_along_axis(z, np.clip(ii, 0, V - 1), axis=1), 0.0)
        logt = np.log(np.where(t > 0, t, 1.0))
        terms = np.where(t > 0, t * (logt - picked / T + lse[:, None]), 0.0)
        out["loss"] = T * T * terms.sum(axis=1)
        out["picked"] = picked
    if loss_grad is None:
        return out
    g = np.where(live, np.asarray(loss_grad, dtype=np.float64), 0.0) * T
    gp = g[:, None] * np.exp(s - lse[:, None])
    dz = gp - g[:, None] * target
    if round_dlogits:
        dz = round_bf16(dz)
    a = np.abs(dz)
    out.update(dz=dz, gp=gp, hidden=dz @ W, lm_head_w=dz.T @ x, abs_hidden=a @ np.abs(W),
               abs_lm_head_w=a.T @ np.abs(x))
    if w1 is not None:
        de, ade = dz @ W2, a @ np.abs(W2)
        d1, a1 = np.zeros((V, e.shape[1])), np.zeros((V, e.shape[1]))
        has = (prevc >= 0) & live
        np.add.at(d1, prevc[has], de[has])
        np.add.at(a1, prevc[has], ade[has])
        out.update(markov_w1=d1, abs_markov_w1=a1, markov_w2=dz.T @ e,
                   abs_markov_w2=a.T @ np.abs(e))
    return out
