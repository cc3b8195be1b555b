"""Distillation from a single entry at T = 1 is cross entropy with that entry as the label: the same
loss, lse and gradients, bit for bit.  That holds only if the teacher's entries get the very
logits that the softmax is made of; a dot product summed in another order is off by several u zabs,
which the difference of lse and logit does not cancel (one confident row of 3528 features: its loss
was off by 5e-5 of it).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


CASES = [("f32", 1, 4, 3, 0), ("f32", 5, 64, 1000, 8), ("f32", 130, 260, 1031, 12), ("f32", 70, 1028, 5003, 128),
         ("bf16", 1, 8, 2, 0), ("bf16", 1, 5120, 30011, 32), ("bf16", 1, 3528, 9683, 88), ("bf16", 9, 72, 1000, 8),
         ("bf16", 40, 2568, 60001, 16), ("bf16", 100, 2552, 60001, 0), ("bf16", 128, 1000, 20011, 40),
         ("bf16", 300, 520, 20011, 128), ("bf16", 700, 136, 3001, 8), ("bf16", 2000, 264, 20011, 24),
         ("bf16", 26000, 64, 12000, 8)]


@pytest.mark.parametrize("dtype,N,H,V,r", CASES)
def test_one_entry_is_the_label(dtype, N, H, V, r):
    import block_draft_readout_amd as m
    g = torch.Generator(device="cuda").manual_seed(N + H)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    w = (rn(V, H) / H ** 0.5).to(t)
    lab = torch.randint(-V // 8, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    lab[0] = V - 1
    x = (rn(N, H) + 12 * torch.rand(N, 1, generator=g, device="cuda") * w[lab.long().clamp(min=0)].float()).to(t)
    lg = torch.rand(N, generator=g, device="cuda") + 0.2
    mk = {}
    if r:
        mk = dict(markov_w1=rn(V, r).to(t), markov_w2=(rn(V, r) * 0.3).to(t),
                  prev_token=torch.randint(-1, V, (N,), generator=g, device="cuda", dtype=torch.int32))
    loss, lse = m.dspark_ce_loss(x, w, lab, **mk)
    want = m.dspark_ce_backward(x, w, lab, lse, lg, **mk)
    # the entry stands at another place of each row's list, the others are not listed
    top = 21
    at = torch.randint(0, top, (N, 1), generator=g, device="cuda")
    ids = torch.full((N, top), -1, dtype=torch.int32, device="cuda").scatter_(1, at, lab[:, None])
    u = rn(N, top)
    l2, lse2, picked = m.dspark_distill_loss(x, w, ids, u, **mk)
    got = m.dspark_distill_backward(x, w, ids, u, lse2, picked, lg, **mk)
    assert torch.equal(lse2, lse) and torch.equal(l2, loss)
    assert set(got) == set(want)
    for k in want:
        assert torch.equal(got[k], want[k]), k
