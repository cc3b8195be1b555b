"""Calls of the paged attention's operators that their documentation allows and that lie off the usual ones."""
import pytest

from gpu_util import log
from test_gpu_paged_qk import _case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def bdr():
    import block_draft_readout_amd as m
    return m


@pytest.mark.parametrize("n,hq,hkv,d,dt", [(1, 40, 8, 128, torch.bfloat16), (1, 1, 1, 64, torch.float32),
                                           (5, 1, 1, 256, torch.bfloat16), (1, 3, 1, 128, torch.float32)])
def test_in_place_of_single_rows_and_heads(n, hq, hkv, d, dt):
    log(f"in place n={n} heads={hq}, {hkv} of {d}")
    q, k, _, wq, wk, f, pos = _case(n + hq, n, hq, hkv, d, d, dt)
    q, k = q.contiguous(), k.contiguous()
    want = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk)
    got = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
