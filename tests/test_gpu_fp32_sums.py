"""fp32 products of the losses sum a step of 32 products before they join the running sum.

One product is 2^12 and every other one 2^-14: four of them are half a step of 2^12 in fp32 (a tie, which
rounds to the even sum), so a chain that adds four products at a time to its running sum never moves.
Thirty-two are 2^-9, four steps: every join is exact but for the first step's, whose 31 small products
may be lost (2^-9.05), and the last one's where it is not whole; so a sum of K products is off by at
most 2 * 32 * 2^-14 = 2^-8 in all, where a chain of fours loses K 2^-14.
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


@pytest.mark.parametrize("N,H,V,r", [(1, 1024, 60, 0), (70, 1028, 130, 12), (5, 2052, 33, 128)])
def test_logits(N, H, V, r):
    """picked is the logit itself."""
    import block_draft_readout_amd as m
    x = torch.full((N, H), 2.0 ** -7, device="cuda")
    w = torch.full((V, H), 2.0 ** -7, device="cuda")
    x[:, 0], w[:, 0] = 2.0 ** 6, 2.0 ** 6
    mk = {}
    if r:
        mk = dict(markov_w1=torch.full((V, r), 2.0 ** -7, device="cuda"), markov_w2=torch.full((V, r), 2.0 ** -7, device="cuda"),
                  prev_token=torch.zeros(N, dtype=torch.int32, device="cuda"))
    ids = torch.arange(V, dtype=torch.int32, device="cuda").repeat(N, 1)[:, :20].contiguous()
    _, lse, picked = m.dspark_distill_loss(x, w, ids, torch.zeros(N, ids.shape[1], device="cuda"), **mk)
    want = 2.0 ** 12 + (H - 1 + r) * 2.0 ** -14
    # (the embedding starts a step of its own: two steps that are not whole)
    assert (picked.double() - want).abs().max() <= 3 * 2.0 ** -9, float(picked[0, 0]) - want
    # all logits are equal: lse is theirs plus ln V, rounded (2^-12) and off as they are
    assert (lse.double() - want - torch.tensor(float(V)).double().log().item()).abs().max() <= 3 * 2.0 ** -9 + 2.0 ** -12


def test_gradients():
    """d W of entry 0 sums the rows: 2^12 from the first, 2^-14 from each other one; d hidden of row
    0 sums the entries likewise.  hidden = 0 but for feature 0, and the head 0, so p = 1 / V."""
    import block_draft_readout_amd as m
    N, V = 1025, 2
    x = torch.zeros(N, 8, device="cuda")
    w = torch.zeros(V, 8, device="cuda")
    x[:, 0] = 2.0 ** -7
    lg = torch.full((N,), 2.0 ** -6, device="cuda")      # d logit of entry 0: -g / 2
    x[0, 0], lg[0] = 2.0 ** 6, 2.0 ** 7
    lab = torch.zeros(N, dtype=torch.int32, device="cuda")
    _, lse = m.dspark_ce_loss(x, w, lab)
    d = m.dspark_ce_backward(x, w, lab, lse, lg, grads=("lm_head_w",))["lm_head_w"]
    want = 2.0 ** 12 + 1024 * 2.0 ** -14
    # p = 1 / 2 is good to 4 u of 2^12
    assert abs(-float(d[0, 0]) - want) <= 2.0 ** -8 + 2.0 ** -10
    # one row, 2049 entries: W is 2^12 at the label's, 2^-3 ... (p - 1 and p = 2^-11 of 2048 entries)
    V = 2048
    x1, w1 = torch.zeros(1, 8, device="cuda"), torch.zeros(V, 8, device="cuda")
    w1[:, 0] = -(2.0 ** -3)          # times p: 2^-14 each
    w1[0, 0] = 2.0 ** 12
    _, lse = m.dspark_ce_loss(x1, w1, lab[:1])
    d = m.dspark_ce_backward(x1, w1, lab[:1], lse, torch.ones(1, device="cuda"), grads=("hidden",))["hidden"]
    want = (2.0 ** -11 - 1) * 2.0 ** 12 - 2047 * 2.0 ** -14
    assert abs(float(d[0, 0]) - want) <= 2.0 ** -8 + 2.0 ** -10
