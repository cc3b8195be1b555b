"""Arguments of the training calls that are no tensors (a packed weight among them) are refused
by name, before anything else is asked of them."""
import pytest

torch = pytest.importorskip("torch")


def _args():
    import block_draft_readout_amd as m
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(100, 64, dtype=torch.bfloat16)
    packed = m.PackedWeight(torch.zeros(16384, dtype=torch.uint8), 100, 64)
    rows = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    return m, x, w, packed, rows, f


def test_losses():
    m, x, w, packed, rows, f = _args()
    ids, u = rows[:, None], f[:, None]
    for bad in (packed, None, w.tolist()):
        for call in (lambda: m.dspark_ce_loss(x, bad, rows),
                     lambda: m.dspark_ce_backward(x, bad, rows, f, f),
                     lambda: m.dspark_distill_loss(x, bad, ids, u),
                     lambda: m.dspark_distill_backward(x, bad, ids, u, f, u, f)):
            with pytest.raises(TypeError, match="lm_head_w"):
                call()
    with pytest.raises(TypeError, match="hidden"):
        m.dspark_ce_loss(None, w, rows)
    with pytest.raises(TypeError, match="hidden"):
        m.dspark_ce_loss(packed, w, rows)
    with pytest.raises(TypeError, match="markov_w1"):
        m.dspark_ce_loss(x, w, rows, markov_w1=packed, markov_w2=w, prev_token=rows)
    with pytest.raises(TypeError, match="teacher_ids"):
        m.dspark_distill_loss(x, w, None, u)
    with pytest.raises(TypeError, match="teacher_logits"):
        m.dspark_distill_loss(x, w, ids, [0.0] * 4)


def test_norm():
    m, x, w, packed, rows, f = _args()
    with pytest.raises(TypeError, match="x must"):
        m.dspark_norm([1.0], w[0])
    with pytest.raises(TypeError, match="x must"):
        m.dspark_norm(packed, w[0])
    with pytest.raises(TypeError, match="grad must"):
        m.dspark_norm_backward(None, x, w[0], f, f)
