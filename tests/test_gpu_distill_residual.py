"""Distillation, bf16, more than 64 rows: what rounding d logits takes from the teacher's heaviest
entry comes back in fp32, to d hidden and d w1 for any number of rows, to d W and d w2 for up to 512.

The logits are 0, so the softmax is p = 1 / V and d logits are g (p - t) at the listed entries and
g p elsewhere, rounded to bf16 but for the heaviest entry.  The gradients' other contributions
cancel, so that their own rounding does not hide that entry's: the weights are 1 (sometimes 0 or 2),
which makes sum_v p W[v] - sum_j t_j W[id_j] small; and rows come in pairs of the same list, nearly
the same g and opposite features, so that d W of an entry is the small difference of the pair.

Tolerance, u = 2^-24: p, t and their product and difference are off by 64 u of their magnitudes; an
entry this may carry over a rounding border by a whole step, 2^-7 of it; a product of K entries is off
by (K / 4 + 40) u times the sum of magnitudes, and the result is rounded once (2^-8).

The host test takes the heaviest entry's rounding from the expected values the other way (kept where
it comes back, given back where it does not): most of the compared values leave the tolerance.
"""
import numpy as np
import pytest

from oracle import training as T

U = 2.0 ** -24
CASES = [(130, 136, 500, 8), (300, 520, 1000, 24), (512, 1032, 20012, 64), (600, 200, 1000, 8),
         (1602, 136, 5122, 16)]
BACK_ROWS = 512      # weight gradients of up to this many rows get the rounding back


def _case(N, H, V, r):
    g = np.random.default_rng(N + H)
    pair = np.repeat(np.arange((N + 1) // 2), 2)[:N]
    a, b, c = (g.permutation(V)[:(N + 1) // 2][pair] for _ in range(3))
    none = np.full(N, -1)
    # one entry, two, the heaviest one twice, three
    lists = np.stack([np.stack(l, axis=1) for l in ((a, none, none), (a, b, none), (a, b, a), (a, b, c))])
    u = np.array([[0, 0, 0], [2, 0.5, 0], [2, 0.5, 1.5], [2, 0.5, 1]], dtype=np.float32)
    ids, u = lists[pair % 4, np.arange(N)].astype(np.int32), u[pair % 4]
    gr = (0.5 + g.random((N + 1) // 2))[pair]
    gr[1::2] *= 1 + g.uniform(0.004, 0.02, N // 2)
    mk = lambda *s: g.choice([1, 1, 1, 0, 2], s)
    x = g.choice([-1, 0, 1], (N, H))
    x[1::2] = -x[0:N - 1:2]
    prev = (np.arange(N) % V).astype(np.int32)
    e = g.choice([-1, 0, 1], (V, r))
    e[1::2] = -e[0:V - 1:2]
    return ids, u, gr.astype(np.float32), prev, mk(V, H), mk(V, r), x, e


def _dlogits(ids, u, gr, V):
    """(exact d logits, heaviest entry of each row, sum of magnitudes of an entry's parts)."""
    N = len(gr)
    t = T.teacher_targets(ids, u, V, 1.0)
    target = np.zeros((N, V))
    for j in range(ids.shape[1]):
        ok = ids[:, j] >= 0
        target[np.flatnonzero(ok), ids[ok, j]] += t[ok, j]
    g = gr.astype(np.float64)[:, None]
    return g * (1.0 / V - target), ids[np.arange(N), t.argmax(axis=1)], g * (1.0 / V + target)


def _expected(c, V, back_features, back_weights):
    """name -> (gradient, tolerance) with the heaviest entries exact or rounded in the products
    that feed the features' and the weights' gradients."""
    ids, u, gr, prev, W, W2, x, e = c
    dz, at, parts = _dlogits(ids, u, gr, V)
    rd = T.round_bf16(dz)
    off = 64 * U * parts
    E = off + np.where(T.round_bf16(dz - off) != T.round_bf16(dz + off), 2.0 ** -7 * np.abs(dz), 0.0)
    n = np.arange(len(gr))
    exact_top = rd.copy()
    exact_top[n, at] = dz[n, at]
    f, w = (exact_top if b else rd for b in (back_features, back_weights))
    out = {}

    def put(name, d, m, K, rows=None):
        """d (E alike) times m, rows of the product summed by `rows`."""
        ref, mags, moved = d @ m, np.abs(d) @ np.abs(m), (E if rows is not None or d.shape == E.shape else E.T) @ np.abs(m)
        if rows is not None:
            by = [np.zeros((V, m.shape[1])) for _ in range(3)]
            for s, v in zip(by, (ref, mags, moved)):
                np.add.at(s, rows, v)
            ref, mags, moved = by
        out[name] = ref, moved + (K / 4 + 40) * U * mags + 2.0 ** -8 * np.abs(ref)

    put("hidden", f, W, V)
    put("markov_w1", f, W2, V + 4 * len(gr), rows=prev)
    put("lm_head_w", w.T, x, len(gr))
    put("markov_w2", w.T, e[prev], len(gr))
    return out, np.unique(at)


@pytest.mark.parametrize("N,H,V,r", CASES)
def test_the_other_rounding_leaves_the_tolerance(N, H, V, r):
    c = _case(N, H, V, r)
    right, top = _expected(c, V, True, N <= BACK_ROWS)
    wrong, _ = _expected(c, V, False, N > BACK_ROWS)
    rows = dict(hidden=np.arange(N), markov_w1=np.unique(c[3]), lm_head_w=top, markov_w2=top)
    for k, (ref, tol) in right.items():
        seen = np.abs(wrong[k][0] - ref)[rows[k]] > 2 * tol[rows[k]]
        assert seen.mean() > 0.15, (k, seen.mean())


@pytest.mark.gpu
@pytest.mark.parametrize("N,H,V,r", CASES)
def test_rounding_of_the_heaviest_entry(N, H, V, r):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as m
    c = _case(N, H, V, r)
    ids, u, gr, prev = (torch.from_numpy(a).cuda() for a in c[:4])
    W, W2, x, e = (torch.from_numpy(a).cuda().bfloat16() for a in c[4:])

    def step(x, w, w1, w2, grads):
        mk = dict(markov_w1=w1, markov_w2=w2, prev_token=prev)
        _, lse, picked = m.dspark_distill_loss(x, w, ids, u, **mk)
        return m.dspark_distill_backward(x, w, ids, u, lse, picked, gr, grads=grads, **mk)

    z = torch.zeros_like
    got = step(z(x), W, z(e), W2, ("hidden", "markov_w1"))
    got.update(step(x, z(W), e, z(W2), ("lm_head_w", "markov_w2")))
    for k, (ref, tol) in _expected(c, V, True, N <= BACK_ROWS)[0].items():
        err = np.abs(got[k].double().cpu().numpy() - ref)
        assert (err <= tol).all(), (k, float((err / np.maximum(tol, 1e-30)).max()))
