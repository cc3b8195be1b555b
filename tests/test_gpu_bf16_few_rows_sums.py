"""bf16 logits of up to 64 rows: 256 products are summed before they join the running sum.

One product is 2^12 and every other one 2^-17: the thirty-two of an MFMA are half a step of 2^12 in fp32
(a tie, which rounds to the even sum), so a chain of MFMAs on one running sum never moves.  256 are
2^-9, four steps: every join is exact but the first one's, whose 255 small products may be lost, and the
last one's where it is not whole (half a step, 2^-12, each for the hidden state's and the embedding's
last step).  So a sum of K products is off by at most 2^-9 + 2^-11, where a chain loses K 2^-17."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_draft_readout_amd as bdr
    bdr.lib()


@pytest.mark.parametrize("N,H,V,r", [(1, 5120, 60, 0), (7, 2560, 151936, 32), (64, 4104, 9000, 8), (40, 2048, 33, 128),
                                     (3, 5120, 30011, 64)])
def test_logits(N, H, V, r):
    """picked is the logit itself; all logits are equal, so lse is theirs plus ln V, rounded (2^-12),
    and the cross entropy ln V."""
    import block_draft_readout_amd as m
    full = lambda n, k, v: torch.full((n, k), v, dtype=torch.bfloat16, device="cuda")
    x, w = full(N, H, 2.0 ** -8), full(V, H, 2.0 ** -9)
    x[:, 0], w[:, 0] = 2.0 ** 6, 2.0 ** 6
    mk = {}
    if r:
        mk = dict(markov_w1=full(V, r, 2.0 ** -8), markov_w2=full(V, r, 2.0 ** -9),
                  prev_token=torch.zeros(N, dtype=torch.int32, device="cuda"))
    ids = torch.arange(V, dtype=torch.int32, device="cuda").repeat(N, 1)[:, -20:].contiguous()
    want, ln = 2.0 ** 12 + (H - 1 + r) * 2.0 ** -17, torch.tensor(float(V)).double().log().item()
    off = 2.0 ** -9 + 2.0 ** -11
    assert (H - 1) * 2.0 ** -17 > 4 * off
    _, lse, picked = m.dspark_distill_loss(x, w, ids, torch.zeros(N, ids.shape[1], device="cuda"), **mk)
    assert (picked.double() - want).abs().max() <= off, float(picked[0, 0]) - want
    assert (lse.double() - want - ln).abs().max() <= off + 2.0 ** -12
    loss, lse2 = m.dspark_ce_loss(x, w, ids[:, 3].contiguous(), **mk)
    assert torch.equal(lse2, lse) and (loss.double() - ln).abs().max() <= 64 * 2.0 ** -24 * (1 + ln)
