"""The training oracle against differences of its own losses and against torch's float64
autograd of the textbook formulas."""
import numpy as np
import pytest

from oracle import training as T
from workloads import synth

torch = pytest.importorskip("torch")


def _case(seed, N=7, V=23, H=12, r=4):
    g = np.random.default_rng(seed)
    return dict(hidden=g.standard_normal((N, H)).astype(np.float32),
                w=g.standard_normal((V, H)).astype(np.float32),
                w1=g.standard_normal((V, r)).astype(np.float32),
                w2=g.standard_normal((V, r)).astype(np.float32),
                prev=np.array([3, 3, -1, 5, V, 0, 3], np.int32)[:N],
                labels=np.array([0, V - 1, 4, -100, 4, V, 2], np.int32)[:N],
                g=g.random(N).astype(np.float32))


def _differences(f, x, h=1e-5):
    x = x.astype(np.float64)
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        a = f(x)
        x[i] = keep - h
        b = f(x)
        x[i] = keep
        d[i] = (a - b) / (2 * h)
    return d


@pytest.fixture()
def float64_storage(monkeypatch):
    """Lets the oracle take float64 arrays as they are, for differences of 1e-5."""
    monkeypatch.setattr(T, "widen", lambda x, dtype: np.asarray(x, dtype=np.float64))


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_loss_gradients_against_differences(float64_storage, kind):
    c = _case(1)
    g = np.random.default_rng(2)
    if kind == "ce":
        kw = dict(labels=c["labels"])
    else:   # short lists, an id twice, an entry without mass, an empty row
        ids = g.integers(0, 23, (7, 5))
        ids[0, 3:] = -1
        ids[1] = [4, 9, 4, 23, 2]
        ids[5] = -1
        u = g.standard_normal((7, 5)) * 2
        u[2, 1] = -np.inf
        kw = dict(ids=ids, u=u, T=1.7)
    arrays = {k: c[k].astype(np.float64) for k in ("hidden", "w", "w1", "w2")}

    def total(**over):
        a = {**arrays, **over}
        o = T.loss(a["hidden"], a["w"], "f32", w1=a["w1"], w2=a["w2"], prev=c["prev"], **kw)
        return float((o["loss"] * c["g"]).sum())

    o = T.loss(arrays["hidden"], arrays["w"], "f32", w1=arrays["w1"], w2=arrays["w2"],
               prev=c["prev"], loss_grad=c["g"], **kw)
    for name, key in (("hidden", "hidden"), ("w", "lm_head_w"), ("w1", "markov_w1"),
                      ("w2", "markov_w2")):
        d = _differences(lambda x: total(**{name: x}), arrays[name])
        # central differences at 1e-5: third derivatives of order 10 and 1e-11 / 1e-5 of rounding
        assert np.abs(d - o[key]).max() < 1e-7, name


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_losses_against_torch(kind):
    c = _case(3)
    t = lambda x: torch.from_numpy(np.asarray(x)).double().requires_grad_()
    x, w = t(c["hidden"]), t(c["w"])
    z = x @ w.t()
    gr = torch.from_numpy(c["g"]).double()
    if kind == "ce":
        lab = torch.from_numpy(c["labels"]).long()
        keep = (lab >= 0) & (lab < 23)
        ref = torch.nn.functional.cross_entropy(z, torch.where(keep, lab, -100), reduction="none")
        o = T.loss(c["hidden"], c["w"], "f32", labels=c["labels"], loss_grad=c["g"])
    else:
        ids = np.stack([np.random.default_rng(9).permutation(23)[:6] for _ in range(7)])
        u = np.random.default_rng(4).standard_normal((7, 6))
        full = torch.full((7, 23), -np.inf, dtype=torch.float64)
        full.scatter_(1, torch.from_numpy(ids), torch.from_numpy(u))
        p = torch.softmax(full / 2.5, dim=1)
        ref = 2.5 ** 2 * torch.nn.functional.kl_div(torch.log_softmax(z / 2.5, dim=1), p,
                                                    reduction="none").sum(dim=1)
        o = T.loss(c["hidden"], c["w"], "f32", ids=ids, u=u, T=2.5, loss_grad=c["g"])
    (ref * gr).sum().backward()
    assert np.abs(o["loss"] - ref.detach().numpy()).max() < 1e-12
    assert np.abs(o["hidden"] - x.grad.numpy()).max() < 1e-12
    assert np.abs(o["lm_head_w"] - w.grad.numpy()).max() < 1e-12


@pytest.mark.parametrize("rms", [False, True])
def test_norm_against_torch(rms):
    g = np.random.default_rng(5)
    x, dy = (g.standard_normal((5, 16)).astype(np.float32) for _ in range(2))
    w, b = (g.standard_normal(16).astype(np.float32) for _ in range(2))
    X, Wt, B = (torch.from_numpy(a).double().requires_grad_() for a in (x, w, b))
    if rms:
        ref = X * (X.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * Wt
    else:
        ref = torch.nn.functional.layer_norm(X, (16,), Wt, B, 1e-5)
    (ref * torch.from_numpy(dy)).sum().backward()
    y, mean, rstd = T.norm(x, w, None if rms else b, "f32", 1e-5, rms)
    dx, dw, db = T.norm_backward(dy, x, w, "f32", 1e-5, rms)
    assert (mean is None) == rms
    assert np.abs(y - ref.detach().numpy()).max() < 1e-12
    assert np.abs(dx - X.grad.numpy()).max() < 1e-12
    assert np.abs(dw - Wt.grad.numpy()).max() < 1e-12
    if not rms:
        assert np.abs(db - B.grad.numpy()).max() < 1e-12


def test_round_bf16_is_the_storage_rounding():
    x = np.random.default_rng(6).standard_normal(4096).astype(np.float32) * 3
    bits = synth.to_bf16_bits(x)
    assert np.array_equal(T.round_bf16(x.astype(np.float64)),
                          (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64))
