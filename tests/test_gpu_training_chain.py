"""norm -> loss -> both backward passes against differences of the summed loss along each
gradient's own direction (fp32), where the derivative is the gradient's norm and not zero.

The five-point difference with step h is off by the loss's own error over h, 1.5 loss_err / h, and by
h^4 |fifth derivative| / 30, which the change from 2 h to h bounds: the sum of both is the
tolerance, which the derivative has to exceed several times.  loss_err: a logit is off by at most
(H / 4 + 60) u zabs and a loss by twice that and 128 u (1 + zabs), zabs the largest sum of a
logit's magnitudes."""
import numpy as np
import pytest

from gpu_util import dev, log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("distill", [False, True])
def test_gradients_against_differences(distill, rms):
    import block_draft_readout_amd as m
    N, H, V, r, top, temp = 24, 64, 500, 8, 6, 1.5
    gn = np.random.default_rng(41)
    f = lambda *s, k=1.0: dev((gn.standard_normal(s) * k).astype(np.float32))
    x, w, w1, w2 = f(N, H), f(V, H, k=2 / 8), f(V, r), f(V, r, k=0.3)
    nw, nb = f(H, k=0.1) + 1, f(H, k=0.1)
    g = dev((gn.random(N) + 0.2).astype(np.float32))
    prev = dev(gn.integers(-1, 12, N).astype(np.int32))
    lab = gn.integers(0, V, N).astype(np.int32)
    lab[3] = -100
    lab = dev(lab)
    ids = np.stack([gn.permutation(V)[:top] for _ in range(N)]).astype(np.int32)
    ids[5] = -1
    ids, u = dev(ids), f(N, top, k=2.0)
    args = [x, nw, nb, w, w1, w2]

    def forward(x, nw, nb, w, w1, w2):
        y, mean, rstd = m.dspark_norm(x, nw, nb, eps=1e-5, rms=rms, stats=True)
        mk = dict(markov_w1=w1, markov_w2=w2, prev_token=prev)
        if distill:
            return (y, mean, rstd, mk, *m.dspark_distill_loss(y, w, ids, u, temperature=temp, **mk))
        return (y, mean, rstd, mk, *m.dspark_ce_loss(y, w, lab, **mk))

    y, mean, rstd, mk, _, *saved = forward(*args)
    if distill:
        gr = m.dspark_distill_backward(y, w, ids, u, *saved, g, temperature=temp, **mk)
    else:
        gr = m.dspark_ce_backward(y, w, lab, *saved, g, **mk)
    grads = [*m.dspark_norm_backward(gr["hidden"], x, nw, mean, rstd), gr["lm_head_w"], gr["markov_w1"],
             gr["markov_w2"]]
    zabs = float((y.abs() @ w.abs().t()).max()) + float((w1.abs().max(0).values @ w2.abs().t()).max())
    loss_err = float(g.sum()) * (2 * (H / 4 + 60) * U * zabs + 128 * U * (1 + zabs)) * (temp if distill else 1)
    for i, d in enumerate(grads):
        norm = float(d.double().norm())
        v = (d.double() / norm).float()

        def diff(h):
            s = [float((forward(*(a + k * h * v if j == i else a for j, a in enumerate(args)))[4].double()
                        * g.double()).sum()) for k in (-2, -1, 1, 2)]
            return (s[0] - 8 * s[1] + 8 * s[2] - s[3]) / (12 * h)

        h = 0.25
        d1, d2 = diff(h), diff(2 * h)
        want = float((d.double() * v.double()).sum())
        tol = 1.5 * loss_err / h + abs(d1 - d2)
        log(f"distill={distill} rms={rms} gradient {i}: norm {want:.5f}, difference {d1:.5f}, tolerance {tol:.2e}")
        assert norm > 0 and want > 4 * tol and abs(want - d1) <= tol
