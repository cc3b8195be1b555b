"""Host-side checks of the training calls: sizes, strides, pointers and workspaces are
rejected with the documented codes before the device is touched, and the binding
rejects tensors of other shapes, types and places."""
import ctypes as C
import os

import pytest

P = 1 << 20     # an aligned address; never dereferenced: every call below fails before that


@pytest.fixture(scope="module")
def A():
    from block_draft_readout_amd import _abi
    if not os.path.exists(_abi.LIB_PATH):
        from block_draft_readout_amd import build
        build.build()
    _abi.load()
    return _abi


def _norm(A, **k):
    a = dict(x=P, rows=4, hidden=64, stride=64, dt=A.BDR_BF16, w=P, b=P, eps=1e-6, y=P << 1, mean=P,
             rstd=P)
    a.update(k)
    return A.load().dspark_norm(a["x"], a["rows"], a["hidden"], a["stride"], a["dt"], a["w"], a["b"],
                                a["eps"], a["y"], a["mean"], a["rstd"], None)


def test_norm_refusals(A):
    E, U = A.BDR_EINVAL, A.BDR_EUNSUPPORTED
    assert _norm(A, dt=7) == E and _norm(A, dt=A.BDR_BF16_PACKED) == E
    assert _norm(A, rows=-1) == E and _norm(A, rows=1 << 24) == U
    assert _norm(A, hidden=0) == E
    assert _norm(A, hidden=68, stride=72) == U
    assert _norm(A, hidden=A.MAX_NORM_HIDDEN + 8, stride=A.MAX_NORM_HIDDEN + 8) == U
    assert _norm(A, stride=56) == E and _norm(A, stride=68) == E
    assert _norm(A, eps=-1.0) == E and _norm(A, eps=float("nan")) == E
    assert _norm(A, eps=float("inf")) == E
    assert _norm(A, x=None) == E and _norm(A, x=P + 8) == E
    assert _norm(A, w=None) == E and _norm(A, b=P + 2) == E
    assert _norm(A, rstd=None) == E
    assert _norm(A, y=P + 128) == E                      # overlaps x
    assert _norm(A, y=P, stride=72) == E                 # in place at another stride
    assert _norm(A, rows=0, x=None, y=None, w=None, rstd=None) == A.BDR_OK


def _norm_bwd(A, **k):
    a = dict(dy=P << 2, ds=64, x=P, xs=64, rows=4, hidden=64, dt=A.BDR_BF16, w=P, mean=P, rstd=P,
             dx=P << 1, dw=P, db=P, ws=P, n=1 << 30)
    a.update(k)
    return A.load().dspark_norm_backward(a["dy"], a["ds"], a["x"], a["xs"], a["rows"], a["hidden"],
                                         a["dt"], a["w"], a["mean"], a["rstd"], a["dx"], a["dw"],
                                         a["db"], a["ws"], a["n"], None)


def test_norm_backward_refusals(A):
    E, U, W = A.BDR_EINVAL, A.BDR_EUNSUPPORTED, A.BDR_EWORKSPACE
    assert _norm_bwd(A, ds=8) == E and _norm_bwd(A, xs=60) == E
    assert _norm_bwd(A, hidden=60, xs=64, ds=64) == U
    assert _norm_bwd(A, dx=None, dw=None, db=None) == E
    assert _norm_bwd(A, dx=P) == E                       # overlaps x
    assert _norm_bwd(A, dx=P << 2, ds=72) == E           # in place of dy at another stride
    assert _norm_bwd(A, rstd=None) == E and _norm_bwd(A, dw=P + 4) == E
    assert _norm_bwd(A, ws=None) == W and _norm_bwd(A, n=16) == W and _norm_bwd(A, ws=P + 16) == W
    assert _norm_bwd(A, rows=0, dw=None, db=None) == A.BDR_OK
    n = A.load().dspark_norm_backward_workspace_bytes
    assert n(4096, 5120) > 0 and n(4096, 5120) % 256 == 0 and n(0, 64) == 0 and n(4, 6) == 0


def _loss(A, distill=False, backward=False, **k):
    a = dict(x=P, rows=5, hidden=64, vocab=1000, dt=A.BDR_BF16, w=P, w1=P, w2=P, rank=8, prev=P,
             labels=P, ids=P, u=P, top=4, udt=A.BDR_F32, T=1.0, loss=P, lse=P, picked=P, g=P,
             dh=2 * P, dw=3 * P, d1=5 * P, d2=6 * P, ws=P, n=1 << 40)
    a.update(k)
    L = A.load()
    head = (a["x"], a["rows"], a["hidden"], a["vocab"], a["dt"], a["w"], a["w1"], a["w2"], a["rank"],
            a["prev"])
    mid = (a["ids"], a["u"], a["top"], a["udt"], a["T"]) if distill else (a["labels"],)
    if backward:
        saved = (a["lse"], a["picked"], a["g"]) if distill else (a["lse"], a["g"])
        tail = saved + (a["dh"], a["dw"], a["d1"], a["d2"], a["ws"], a["n"], None)
        f = L.dspark_distill_backward if distill else L.dspark_ce_backward
    else:
        tail = (a["loss"], a["lse"]) + ((a["picked"],) if distill else ()) + (a["ws"], a["n"], None)
        f = L.dspark_distill_loss if distill else L.dspark_ce_loss
    return f(*head, *mid, *tail)


@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_loss_refusals(A, distill, backward):
    E, U, W = A.BDR_EINVAL, A.BDR_EUNSUPPORTED, A.BDR_EWORKSPACE
    f = lambda **k: _loss(A, distill, backward, **k)
    assert f(dt=A.BDR_BF16_PACKED) == E and f(dt=9) == E
    assert f(rows=-1) == E and f(hidden=0) == E and f(vocab=0) == E and f(rank=-8) == E
    assert f(rows=(1 << 20) + 1) == U and f(hidden=(1 << 20) + 8) == U and f(vocab=(1 << 21) + 1) == U
    assert f(rows=1 << 20, vocab=1 << 16) == U and f(hidden=1 << 18, vocab=1 << 18) == U
    assert f(hidden=68) == U and f(rank=12) == U and f(rank=136) == U
    assert f(dt=A.BDR_F32, hidden=66) == U
    assert f(x=None) == E and f(x=P + 8) == E and f(w=None) == E
    assert f(w1=None) == E and f(w2=None) == E and f(prev=None) == E and f(w2=P + 8) == E
    assert f(ws=None) == W and f(n=64) == W and f(ws=P + 64) == W
    assert f(lse=None) == E
    if distill:
        assert f(top=0) == E and f(top=A.MAX_TEACHER + 1) == U and f(udt=5) == E
        assert f(T=0.0) == E and f(T=-1.0) == E and f(T=9e-5) == E and f(T=1.1e4) == E and f(T=float("inf")) == E and f(T=float("nan")) == E
        assert f(ids=None) == E and f(u=None) == E and f(u=P + 2) == E and f(picked=None) == E
    else:
        assert f(labels=None) == E and f(labels=P + 2) == E
    if backward:
        assert f(g=None) == E
        assert f(dh=None, dw=None, d1=None, d2=None) == E
        assert f(dh=P + 8) == E and f(dw=P + 8) == E
        assert f(dh=P) == E and f(dw=P + 1024) == E and f(d1=3 * P + 16) == E   # overlaps
        assert f(rank=0) == E                            # Markov gradients without a head
        assert f(rows=0, dw=None, d1=None, d2=None) == A.BDR_OK
    else:
        assert f(loss=None) == E
        assert f(rows=0, x=None, w=None, loss=None) == A.BDR_OK


def test_loss_workspaces(A):
    L = A.load()
    ce = L.dspark_ce_workspace_bytes
    assert ce(0, 5120, 151936, 64, A.BDR_BF16, 0) == 0 and ce(4, 12, 100, 0, A.BDR_BF16, 0) == 0
    fwd, bwd = (ce(4096, 5120, 151936, 64, A.BDR_BF16, b) for b in (0, 1))
    assert fwd % 256 == 0 and bwd % 256 == 0
    # forward: compacted hidden states and per-row statistics, nothing logits-sized; backward: one
    # piece of d logits and the fp32 partial sums of d hidden
    assert 4096 * 5120 * 2 <= fwd < 4096 * 151936 * 2 // 8
    assert bwd < 4096 * 151936 * 2
    d = L.dspark_distill_workspace_bytes
    assert d(4096, 5120, 151936, 64, 64, A.BDR_BF16, 0) >= fwd
    assert d(4096, 5120, 151936, 64, 0, A.BDR_BF16, 0) == 0


def test_binding_refuses_host_tensors_and_other_shapes():
    torch = pytest.importorskip("torch")
    import block_draft_readout_amd as bdr
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(100, 64, dtype=torch.bfloat16)
    lab = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        bdr.dspark_norm(x, torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        bdr.dspark_ce_loss(x, w, lab)
    with pytest.raises(ValueError):
        bdr.dspark_distill_loss(x, w, lab[:, None], torch.zeros(4, 1))


def test_training_names_are_public():
    import block_draft_readout_amd as bdr
    for n in ("dspark_norm", "dspark_norm_backward", "dspark_ce_loss", "dspark_ce_backward",
              "dspark_distill_loss", "dspark_distill_backward"):
        assert n in bdr.__all__ and callable(getattr(bdr, n))
    assert C.sizeof(C.c_void_p) == 8
