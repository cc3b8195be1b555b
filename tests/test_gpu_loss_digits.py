"""The loss values keep their digits where the logits share a large offset.

The first feature adds 2^20 to every logit; the others are small whole numbers, so every
logit is a whole number below 2^24 and exact in fp32, whatever the order of its sum.  The
loss, lse - z[label], depends on the differences of the logits alone.  Where the sum's
reference is 2^20 log2(e), the logarithm joined to it in one fp32 number is off by up to
half a step of that (0.06); kept apart until the label's logit has been taken off, it is not.

Tolerance, u = 2^-24, D the largest minus the smallest logit of a row over T, V entries.  All
logits are scaled by one rounded log2(e) / T (2 u D, and u of the loss for ln 2).  An exponent is
one rounding (1.5 u (D + 1), times ln 2 relative in its exponential, itself 2 u); at most 24
additions of a tile's columns, 3 + 6 + V / (64 * 128) joins of 3 roundings each; the logarithm
2 u of itself, at most log2(V) + 1; label's difference, sum and product 3 u (1.5 D + 1.5 log V
+ 1).  In all below 64 u (1 + D + log V) for V up to 2^16.  Distillation: the same for each
listed entry, its t off by 64 u at most, which the factor log t - log p of at most
(D + 2 log V + max |log t|) carries, and logf(t) by 2 u: T^2 128 u (1 + D + 2 log V + max |log t|).
"""
import numpy as np
import pytest

from oracle import training as T
from workloads import synth
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


def _case(N, V, dtype):
    g = np.random.default_rng(N + V)
    x, w = g.integers(-2, 3, (N, 8)), g.integers(-1, 2, (V, 8))
    x[:, 0] = w[:, 0] = 1024
    st = lambda a: synth.store(a.astype(np.float32), dtype)
    z = x @ w.T
    return g, st(x), st(w), z, (z.max(axis=1) - z.min(axis=1)).astype(np.float64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 2), (7, 1000), (65, 40007), (300, 517)])
def test_cross_entropy(N, V, dtype):
    import block_draft_readout_amd as m
    g, x, w, z, D = _case(N, V, dtype)
    lab = g.integers(0, V, N).astype(np.int32)
    loss, _ = m.dspark_ce_loss(dev(x), dev(w), dev(lab))
    ref = T.loss(x, w, dtype, labels=lab)["loss"]
    err = np.abs(loss.cpu().numpy().astype(np.float64) - ref)
    tol = 64 * U * (1 + D + np.log(V))
    log(f"offset logits, cross entropy {dtype} {N} V={V}: worst error {err.max():.2e}, tolerance {tol.min():.2e}")
    assert (err <= tol).all()


@pytest.mark.parametrize("dtype,temp", [("f32", 1.0), ("bf16", 2.0)])
@pytest.mark.parametrize("N,V,top", [(1, 40, 1), (9, 1000, 20), (130, 40007, 100)])
def test_distillation(N, V, top, dtype, temp):
    import block_draft_readout_amd as m
    g, x, w, z, D = _case(N, V, dtype)
    ids = np.stack([g.permutation(V)[:top] for _ in range(N)]).astype(np.int32)
    u = (g.standard_normal((N, top)) * 3).astype(np.float32)
    loss, _, picked = m.dspark_distill_loss(dev(x), dev(w), dev(ids), dev(u), temperature=temp)
    assert np.array_equal(picked.cpu().numpy(), np.take_along_axis(z, ids.astype(np.int64), axis=1))
    ref = T.loss(x, w, dtype, ids=ids, u=u, T=temp)["loss"]
    logt = np.abs(np.log(T.teacher_targets(ids, u, V, temp))).max(axis=1)
    err = np.abs(loss.cpu().numpy().astype(np.float64) - ref)
    tol = temp * temp * 128 * U * (1 + D / temp + 2 * np.log(V) + logt)
    log(f"offset logits, distillation {dtype} {N} V={V}: worst error {err.max():.2e}, tolerance {tol.min():.2e}")
    assert (err <= tol).all()
