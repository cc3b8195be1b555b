"""Exact bits of the feature gradients (d hidden, d w1) of bf16 cross entropy.

hidden = 0: every softmax entry is p = 1 / V, and d logits are g lo with lo = p rounded to bf16 (of
up to 64 rows: to two bf16 terms), except at the row's label.  Against weights of -1, 0, 1 and g a
power of two, every product is a multiple of g times the last bit of lo, which has 8 bits (two terms:
at most 17).  Where a row's sum of weights' magnitudes stays below 2^16 (two terms: 2^7), its
products' sum stays below 2^24 last bits and is exact in fp32, in any order.  What the label's entry
adds is nothing where the label's weight is 0.  There d hidden is one rounding of g lo sum_v W[v],
and d w1 of lo sum_v w2[v] sum_n g over the rows n with that previous token, if the weight is 0 for
all of them.

The host test leaves out one entry of the vocabulary in the expected values: some of the compared
ones change, so a kernel that loses an entry (an edge of a tile or of a piece) fails.
"""
import numpy as np
import pytest

from oracle import training as T

# rows, features, entries, rank: two terms in narrow tiles and in tiles of 64 and 128 rows, weights
# within and beyond the caches; one term in narrow tiles, tiles of 128 and of 256 rows, a weight
# beyond the caches, several pieces (the last of a single entry)
CASES = [(7, 72, 1003, 8), (61, 328, 61501, 8), (20, 1000, 60004, 8), (20, 2568, 60004, 16),
         (60, 2568, 60004, 16), (130, 328, 2560, 64), (257, 72, 130, 16), (125, 264, 61501, 8), (100, 2568, 60001, 16),
         (300, 520, 20011, 32), (1601, 136, 16501, 8), (26000, 64, 12000, 8), (53000, 136, 5121, 8)]


def _lo(N, V):
    """p as the products take it, and the most that magnitudes of weights may add up to."""
    def terms(p):
        hi = float(T.round_bf16(p))
        return (hi, float(T.round_bf16(p - hi))) if N <= 64 else (hi, 0.0)
    p = 1.0 / V
    # fp32's error of p changes neither term: log2(V) < 16 is joined, scaled by ln 2, and back by
    # log2(e), each off by half a step of 16 (5e-7) or, the logarithm, a whole one, and the two
    # constants by 5e-7 of it in all: 2.6e-6, times ln 2 relative in p, and the exponential's step
    assert terms(p * (1 + 3e-6)) == terms(p) == terms(p * (1 - 3e-6))
    return sum(terms(p)), 2 ** 7 if N <= 64 else 2 ** 16


def _case(N, H, V, r):
    g = np.random.default_rng(N + V)
    most = _lo(N, V)[1]

    def signs(cols, few):
        w = g.integers(0, 2, (V, cols), dtype=np.int8) * 2 - 1
        return np.where(g.random((V, cols), dtype=np.float32) < few, w, 0).astype(np.int8)

    W = signs(H, min(0.67, most / (2.0 * V)))
    prev = (np.arange(N) // 2 % V).astype(np.int32)
    # the rows of a token add up, at up to 8 times the smallest g
    W2 = signs(r, min(0.5, most / (24.0 * V * np.bincount(prev).max())))
    W[-1] = W2[-1] = 1
    labels = np.where(g.random(N) < 0.2, -1, g.integers(0, V, N)).astype(np.int32)
    gr = (2.0 ** g.integers(-2, 2, N)).astype(np.float32)
    return W, W2, prev, labels, gr


def _expected(W, W2, prev, labels, gr, drop=None):
    """((values, where they are exact) of d hidden, of d w1)."""
    V = W.shape[0]
    lo, most = _lo(len(labels), V)
    keep = np.ones(V, dtype=bool)
    if drop is not None:
        keep[drop] = False
    live = labels >= 0
    S, S2 = (w[keep].sum(axis=0, dtype=np.int64) for w in (W, W2))
    at = np.where(live, labels, 0)
    g = np.where(live, gr, 0.0).astype(np.float64)
    hid = T.round_bf16(g[:, None] * lo * S[None, :])
    exact = (W[at] == 0) | ~live[:, None]
    assert int(np.abs(W).sum(axis=0, dtype=np.int64).max()) < most
    sums, spoiled = np.zeros(V), np.zeros((V, W2.shape[1]), dtype=np.int64)
    np.add.at(sums, prev, g)
    np.add.at(spoiled, prev, ((W2[at] != 0) & live[:, None]).astype(np.int64))
    d1 = T.round_bf16(sums[:, None] * lo * S2[None, :])
    # in units of the smallest g: the sum of magnitudes of d w1
    assert (sums / gr.min()).max() * int(np.abs(W2).sum(axis=0, dtype=np.int64).max()) < most
    return (hid, exact), (d1, spoiled == 0)


@pytest.mark.parametrize("N,H,V,r", CASES)
def test_a_lost_entry_changes_compared_values(N, H, V, r):
    c = _case(N, H, V, r)
    right = _expected(*c)
    live = c[3] >= 0
    for (a, ok), reached in zip(right, (live.sum() * H, np.unique(c[2][live]).size * r)):
        assert np.count_nonzero(a[ok]) > reached // 5
    # the last entry has a weight everywhere, another one (of d w1 few do) wherever it is not 0
    for drop, seen in ((V - 1, (0, 1)), (int(np.flatnonzero(c[0].any(axis=1))[0]), (0,))):
        wrong = _expected(*c, drop=drop)
        for k in seen:
            assert (right[k][0] != wrong[k][0])[right[k][1]].any()


@pytest.mark.gpu
@pytest.mark.parametrize("N,H,V,r", CASES)
def test_feature_gradients_are_exact(N, H, V, r):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as m
    c = _case(N, H, V, r)
    W, W2, prev, labels, gr = (torch.from_numpy(a).cuda() for a in c)
    W, W2 = W.bfloat16(), W2.bfloat16()
    x = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
    mk = dict(markov_w1=torch.zeros_like(W2), markov_w2=W2, prev_token=prev)
    _, lse = m.dspark_ce_loss(x, W, labels, **mk)
    got = m.dspark_ce_backward(x, W, labels, lse, gr, grads=("hidden", "markov_w1"), **mk)
    for name, (ref, ok) in zip(("hidden", "markov_w1"), _expected(*c)):
        a = got[name].double().cpu().numpy()
        bad = (a != ref) & ok
        assert not bad.any(), (name, np.argwhere(bad)[:3].tolist(), int(bad.sum()))
        assert np.isfinite(a).all()
