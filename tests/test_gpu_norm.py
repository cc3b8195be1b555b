"""GPU parity of the row normalisation (dspark_norm, dspark_norm_backward) against
oracle.training: layer and root-mean-square form, bf16 and fp32, one row to thousands,
every lane layout (8 to 16384 features), row strides, in-place outputs, single gradients,
replayed graphs.

Tolerances.  u = 2^-24 is half an fp32 step, rnd the storage rounding (bf16 2^-8, fp32
u).  A lane adds at most H / 64 elements in a row and the lanes join in at most 16 more
additions, so a sum over a row is off by at most C u times the sum of magnitudes with
C = H / 64 + 16; the elementwise steps add a few u.  With A = mean |x| of the row and
D = |xh| + rstd A (what an error of the mean moves xh by, in units of u):
  y        rnd |y| + (C + 8) u |w| D + u |b|
  dx       rnd |dx| + (3 C + 32) u rstd (|gy| + mean |gy| + D mean(|gy| D))
  dw, db   rnd |.| + (rows + C + 32) u sum |dy| D   (db: without D)
"""
import numpy as np
import pytest

from oracle import training as T
from workloads import synth
from gpu_util import dev, host_bits, log
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
RND = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


def bdr():
    import block_draft_readout_amd as m
    return m


def _case(seed, rows, H, dtype, rms):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, H)) * np.exp(g.uniform(-2, 2, (rows, 1))) + g.standard_normal((1, H))
    x[:, ::13] *= 9
    st = lambda a: synth.store(np.ascontiguousarray(a, dtype=np.float32), dtype)
    return (st(x), st(1 + 0.2 * g.standard_normal(H)), None if rms else st(g.standard_normal(H)),
            st(g.standard_normal((rows, H))))


def _tols(x, w, b, dy, dtype, eps, rms):
    y, mean, rstd = T.norm(x, w, b, dtype, eps, rms)
    dx, dw, db = T.norm_backward(dy, x, w, dtype, eps, rms)
    X, Wt, DY = (oracle.widen(a, dtype) for a in (x, w, dy))
    H, rows = X.shape[1], X.shape[0]
    C, rnd = H / 64 + 16, RND[dtype]
    xh = (X - (0 if rms else mean[:, None])) * rstd[:, None]
    D = np.abs(xh) + (rstd * np.abs(X).mean(axis=1))[:, None]
    gy = np.abs(DY * Wt)
    ref = dict(y=y, dx=dx, dw=dw, db=db, mean=mean, rstd=rstd)
    tol = dict(y=rnd * np.abs(y) + (C + 8) * U * np.abs(Wt) * D
               + (0 if b is None else U * np.abs(oracle.widen(b, dtype))),
               dx=rnd * np.abs(dx) + (3 * C + 32) * U * rstd[:, None] * (
                   gy + gy.mean(axis=1, keepdims=True) + D * (gy * D).mean(axis=1, keepdims=True)),
               dw=rnd * np.abs(dw) + (rows + C + 32) * U * (np.abs(DY) * D).sum(axis=0),
               db=rnd * np.abs(db) + (rows + C + 32) * U * np.abs(DY).sum(axis=0),
               rstd=(C + 8) * U * rstd * (1 + rstd * np.abs(X).mean(axis=1)),
               mean=None if rms else (C + 2) * U * np.abs(X).mean(axis=1))
    return ref, tol


def _check(name, got, ref, tol, dtype):
    g = oracle.widen(host_bits(got), dtype) if dtype else got.cpu().numpy().astype(np.float64)
    err = np.abs(g - ref)
    assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))
    return float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0


CASES = [("bf16", 1, 5120, False), ("bf16", 1, 8, True), ("bf16", 3, 2560, True),
         ("bf16", 67, 512, False), ("bf16", 5, 1032, False), ("bf16", 130, 1544, True),
         ("bf16", 9, 2048, False), ("bf16", 9, 2056, False), ("bf16", 1025, 4104, False),
         ("bf16", 33, 8192, True), ("bf16", 33, 8200, False), ("bf16", 7, 16384, False),
         ("f32", 1, 4, False), ("f32", 2, 1000, False), ("f32", 1023, 260, True),
         ("f32", 17, 1024, False), ("f32", 17, 1028, True), ("f32", 10, 3076, False),
         ("f32", 6, 4100, False), ("f32", 6, 8196, True), ("f32", 5, 16384, False)]


@pytest.mark.parametrize("dtype,rows,H,rms", CASES)
def test_norm_forward_and_backward(dtype, rows, H, rms):
    eps = 1e-5
    x, w, b, dy = _case(rows * 7 + H, rows, H, dtype, rms)
    m = bdr()
    X, Wt, B, DY = dev(x), dev(w), None if b is None else dev(b), dev(dy)
    y, mean, rstd = m.dspark_norm(X, Wt, B, eps=eps, rms=rms, stats=True)
    dx, dw, db = m.dspark_norm_backward(DY, X, Wt, mean, rstd, bias=not rms)
    ref, tol = _tols(x, w, b, dy, dtype, eps, rms)
    worst = [_check("y", y, ref["y"], tol["y"], dtype), _check("dx", dx, ref["dx"], tol["dx"], dtype),
             _check("dw", dw, ref["dw"], tol["dw"], dtype),
             _check("rstd", rstd, ref["rstd"], tol["rstd"], None)]
    if rms:
        assert mean is None and db is None
    else:
        worst += [_check("db", db, ref["db"], tol["db"], dtype),
                  _check("mean", mean, ref["mean"], tol["mean"], None)]
    log(f"norm {dtype} {rows}x{H} rms={rms}: worst error / tolerance {max(worst):.3f}")
    # the same bits again, and single gradients equal to the joint call's
    again = m.dspark_norm_backward(DY, X, Wt, mean, rstd, bias=not rms)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only = m.dspark_norm_backward(DY, X, Wt, mean, rstd, bias=False, want_weight=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = m.dspark_norm_backward(DY, X, Wt, mean, rstd, bias=False, want_x=False)
    assert only[0] is None and torch.equal(only[1], dw)


def test_strided_rows_and_in_place():
    m = bdr()
    x, w, b, dy = _case(3, 37, 512, "bf16", False)
    X, Wt, B, DY = dev(x), dev(w), dev(b), dev(dy)
    y, mean, rstd = m.dspark_norm(X, Wt, B, stats=True)
    dx, dw, db = m.dspark_norm_backward(DY, X, Wt, mean, rstd)
    wide = torch.full((37, 1040), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:520] = X
    gwide = torch.full((37, 768), float("nan"), dtype=torch.bfloat16, device="cuda")
    gwide[:, :512] = DY
    y2, mean2, rstd2 = m.dspark_norm(wide[:, 8:520], Wt, B, stats=True)
    assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    for a, b2 in zip(m.dspark_norm_backward(gwide[:, :512], wide[:, 8:520], Wt, mean, rstd),
                     (dx, dw, db)):
        assert torch.equal(a, b2)
    assert torch.isnan(wide[:, 520:]).all() and torch.isnan(gwide[:, 512:]).all()
    z = X.clone()
    assert m.dspark_norm(z, Wt, B, out=z) is z and torch.equal(z, y)
    with pytest.raises(m.BdrError):     # rows 2 bytes off a 16-byte boundary
        m.dspark_norm(wide[:, 7:519], Wt, B)


def test_rows_with_nan_stay_alone_and_no_rows():
    m = bdr()
    x, w, b, dy = _case(4, 9, 256, "f32", False)
    X, Wt, B, DY = dev(x), dev(w), dev(b), dev(dy)
    y = m.dspark_norm(X, Wt, B)
    X2 = X.clone()
    X2[4, 3] = float("nan")
    X2[6] = float("inf")
    y2 = m.dspark_norm(X2, Wt, B)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y2[keep], y[keep])
    assert torch.isnan(y2[4]).all() and torch.isnan(y2[6]).all()
    e = X[:0]
    y0, mean, rstd = m.dspark_norm(e, Wt, B, stats=True)
    dx, dw, db = m.dspark_norm_backward(e, e, Wt, mean, rstd)
    assert y0.shape == (0, 256) and dx.shape == (0, 256)
    assert not dw.any() and not db.any()


def test_constant_row_and_leading_axes():
    m = bdr()
    X = torch.full((2, 3, 64), 7.25, device="cuda")
    Wt, B = torch.ones(64, device="cuda"), torch.full((64,), 0.5, device="cuda")
    y, mean, rstd = m.dspark_norm(X, Wt, B, eps=0.25, stats=True)
    assert y.shape == X.shape and mean.shape == (6,)
    assert (mean == 7.25).all() and (rstd == 2.0).all() and (y == 0.5).all()


def test_norm_captured_and_replayed():
    m = bdr()
    rows, H = 300, 640
    x, w, b, dy = _case(6, rows, H, "bf16", False)
    X, Wt, B, DY = dev(x), dev(w), dev(b), dev(dy)
    ws = torch.full((m.lib().dspark_norm_backward_workspace_bytes(rows, H) + 256,), 255,
                    dtype=torch.uint8, device="cuda")

    def step():
        y, mean, rstd = m.dspark_norm(X, Wt, B, stats=True)
        return (y, *m.dspark_norm_backward(DY, X, Wt, mean, rstd, workspace=ws))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        X.copy_(dev(_case(60 + k, rows, H, "bf16", False)[0]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, e in zip(got, step()):
            assert torch.equal(a, e)
