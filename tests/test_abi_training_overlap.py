"""Outputs and workspaces of the training calls that share memory with another argument are
refused before the device is touched.  The addresses are made up, far apart, and never
dereferenced: every call below has one pair that overlaps."""
import itertools
import os

import pytest

FAR = 1 << 32


@pytest.fixture(scope="module")
def A():
    from block_draft_readout_amd import _abi
    if not os.path.exists(_abi.LIB_PATH):
        from block_draft_readout_amd import build
        build.build()
    _abi.load()
    return _abi


def _places(names):
    return {n: FAR * (i + 1) for i, n in enumerate(names)}


def _refused(A, rc, what):
    text = A.load().bdr_last_error().decode()
    assert rc == A.BDR_EINVAL and "overlap" in text, (what, rc, text)


def _pairs(outs, ins, free=()):
    """(moved, onto): each output onto each input and each later output."""
    for o in outs:
        for q in itertools.chain(ins, outs[outs.index(o) + 1:]):
            if (o, q) not in free:
                yield o, q


ROWS, H, V, R, TOP = 4096, 64, 1000, 8, 4      # every tensor above 256 bytes


def test_norm(A):
    names = ("x", "w", "b", "y", "mean", "rstd")
    for o, q in _pairs(("y", "mean", "rstd"), ("x", "w", "b"), free={("y", "x")}):
        a = _places(names)
        a[o] = a[q] + 64
        _refused(A, A.load().dspark_norm(a["x"], ROWS, H, H, A.BDR_BF16, a["w"], a["b"], 1e-6, a["y"],
                                         a["mean"], a["rstd"], None), (o, q))
    a = _places(names)      # an input that begins inside the output
    a["b"] = a["y"] + ROWS * H * 2 - 16
    _refused(A, A.load().dspark_norm(a["x"], ROWS, H, H, A.BDR_BF16, a["w"], a["b"], 1e-6, a["y"],
                                     a["mean"], a["rstd"], None), "end of y")


def test_norm_backward(A):
    names = ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws")
    ins = ("dy", "x", "w", "mean", "rstd")
    n = A.load().dspark_norm_backward_workspace_bytes(ROWS, H)
    for o, q in _pairs(("dx", "dw", "db", "ws"), ins, free={("dx", "dy")}):
        a = _places(names)
        if o == "ws":
            a[q] = a[o] + n - 64     # a workspace stays aligned: the other one moves
        else:
            a[o] = a[q] + 64
        _refused(A, A.load().dspark_norm_backward(
            a["dy"], H, a["x"], H, ROWS, H, A.BDR_BF16, a["w"], a["mean"], a["rstd"], a["dx"], a["dw"],
            a["db"], a["ws"], n, None), (o, q))


@pytest.mark.parametrize("distill", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_losses(A, distill, backward):
    L = A.load()
    ins = ["x", "w", "w1", "w2", "prev"] + (["ids", "u"] if distill else ["labels"])
    saved = ["lse"] + (["picked"] if distill else [])
    if backward:
        ins += saved + ["g"]
        outs = ["dh", "dw", "d1", "d2", "ws"]
    else:
        outs = ["loss"] + saved + ["ws"]
    if distill:
        n = L.dspark_distill_workspace_bytes(ROWS, H, V, R, TOP, A.BDR_BF16, int(backward))
    else:
        n = L.dspark_ce_workspace_bytes(ROWS, H, V, R, A.BDR_BF16, int(backward))
    for o, q in _pairs(outs, ins):
        a = _places(dict.fromkeys(ins + outs))
        if "ws" in (o, q):
            other = q if o == "ws" else o
            a[other] = a["ws"] + n - 64
        else:
            a[o] = a[q] + 64
        head = (a["x"], ROWS, H, V, A.BDR_BF16, a["w"], a["w1"], a["w2"], R, a["prev"])
        mid = (a["ids"], a["u"], TOP, A.BDR_F32, 1.0) if distill else (a["labels"],)
        mids = tuple(a[k] for k in saved)
        if backward:
            f = L.dspark_distill_backward if distill else L.dspark_ce_backward
            rc = f(*head, *mid, *mids, a["g"], a["dh"], a["dw"], a["d1"], a["d2"], a["ws"], n, None)
        else:
            f = L.dspark_distill_loss if distill else L.dspark_ce_loss
            rc = f(*head, *mid, a["loss"], *mids, a["ws"], n, None)
        _refused(A, rc, (o, q))


@pytest.mark.gpu
def test_neighbours_are_accepted():
    """Buffers that touch without sharing a byte."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as m
    buf = torch.randn(2 * 37, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    want = m.dspark_norm(buf[:37].clone(), w)
    assert torch.equal(m.dspark_norm(buf[:37], w, out=buf[37:]), want)
    with pytest.raises(m.BdrError):
        m.dspark_norm(buf[:37], w, out=buf[36:73])
