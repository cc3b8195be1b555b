"""The softmax's logarithm is rounded once, and fp32 gradients lose nothing more to it.

hidden = 0 (or every weight 0): the sum over the vocabulary is V exactly, so lse has to be ln V rounded
to fp32 (no V here is near a tie).  A feature that is 1 in the only row makes d W of an entry that is
not the label g p itself, p = 1 / V; u = 2^-24.  lse is off by half a step (2^-21 from 8 on, 2^-22
from 4 on), which is p's relative error; the exponential is good to a step (2 u), its correction, g and
their products to 4 u: 2^-21 + 6 u.  With every weight 0 at temperature T the distillation's p is the
same 1 / V and its d logits g T p.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
VS = [61, 100, 363, 1000, 2981, 3001, 4097, 5003, 7001, 9973, 12007, 17011, 20011, 24001, 30011, 37003, 44017,
      50021, 61501, 80021, 99991, 120011, 151936]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lse_of_equal_logits_is_rounded_once(dtype):
    import block_draft_readout_amd as m
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    for V in VS:
        x, w = torch.ones(2, 8, dtype=t, device="cuda"), torch.zeros(V, 8, dtype=t, device="cuda")
        lab = torch.tensor([0, V - 1], dtype=torch.int32, device="cuda")
        want = np.float32(np.log(np.float64(V)))
        loss, lse = m.dspark_ce_loss(x, w, lab)
        assert (lse.cpu().numpy() == want).all() and (loss.cpu().numpy() == want).all(), V
        _, lse, _ = m.dspark_distill_loss(x, w, lab[:, None].contiguous(),
                                          torch.zeros(2, 1, device="cuda"), temperature=1.7)
        assert (lse.cpu().numpy() == want).all(), V


@pytest.mark.parametrize("temp", [0.0, 1.7])
def test_gradient_of_equal_logits(temp):
    import block_draft_readout_amd as m
    for V in VS:
        x = torch.zeros(1, 8, device="cuda")
        x[0, 0] = 1.0
        w, lab = torch.zeros(V, 8, device="cuda"), torch.tensor([V // 2], dtype=torch.int32, device="cuda")
        one = torch.ones(1, device="cuda")
        if temp:
            ids, u = lab[:, None].contiguous(), torch.zeros(1, 1, device="cuda")
            _, lse, picked = m.dspark_distill_loss(x, w, ids, u, temperature=temp)
            d = m.dspark_distill_backward(x, w, ids, u, lse, picked, one, temperature=temp)["lm_head_w"]
        else:
            _, lse = m.dspark_ce_loss(x, w, lab)
            d = m.dspark_ce_backward(x, w, lab, lse, one)["lm_head_w"]
        d = np.delete(d[:, 0].double().cpu().numpy(), V // 2)
        want = (np.float64(np.float32(temp)) or 1.0) / V
        assert np.abs(d / want - 1).max() <= 2.0 ** -21 + 6 * U, (V, np.abs(d / want - 1).max())
