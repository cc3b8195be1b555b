"""Calls of the paged attention's operators that their documentation allows and that lie off the usual ones."""
import pytest

from gpu_util import log
from test_gpu_paged_attention import Case
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


@pytest.mark.parametrize("page_size", [(1 << 32) + 16, -(1 << 32) + 16, 1 << 31])
def test_page_sizes_past_32_bits(page_size):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    with pytest.raises((ValueError, bdr().BdrError)):
        bdr().spec_slots(z(2), z(2), z(2, 1), z(2), z(2), z(1), page_size, 8)
    if page_size > 0:   # a cache whose positions lie over each other
        cache = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(1, page_size, 2, 64)
        with pytest.raises((ValueError, bdr().BdrError)):
            bdr().dflash_paged_attention(cache[0, :1], cache, cache, z(1, 1), z(2), z(1))


def test_windows_past_32_bits():
    c = Case(1, [(4, 200), (70, 90)], 4, 2, 64, 16)
    want = c.run()
    for window in (1 << 31, 1 << 32, (1 << 32) + 5, (1 << 40) - 1):   # past every context: none
        got = c.run(window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for window in (-1, -(1 << 32), -(1 << 32) + 7):
        with pytest.raises((ValueError, bdr().BdrError)):
            c.run(window=window)


@pytest.mark.parametrize("n,d,dt,inter", [(1, 128, torch.bfloat16, False), (2100, 64, torch.bfloat16, True),
                                          (7, 256, torch.float32, False)])
def test_weight_of_keys_without_queries(n, d, dt, inter):
    """A drafter's context has keys and values alone: no weight of queries is needed, and none is read."""
    q, k, v, wq, wk, f, pos = _case(n + d, n, 4, 2, d, d, dt)
    slots = torch.randperm(n + 5, device="cuda")[:n].int()
    caches = [[torch.zeros(n + 5, 1, 2, d, dtype=dt, device="cuda") for _ in range(2)] for _ in range(3)]
    for (kc, vc), weights in zip(caches, (dict(q_weight=wq, k_weight=wk), dict(k_weight=wk),
                                          dict(q_weight=torch.full_like(wk, float("nan")), k_weight=wk))):
        bdr().dspark_qk_norm_rope(None, k, v, pos, f, interleaved=inter, slots=slots, k_cache=kc, v_cache=vc, **weights)
    for kc, vc in caches[1:]:
        assert torch.equal(kc, caches[0][0]) and torch.equal(vc, caches[0][1])
    with_q = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk, interleaved=inter)[1]
    assert torch.equal(caches[1][0][slots.long(), 0], with_q)


@pytest.mark.parametrize("n,dt", [(2, torch.bfloat16), (50, torch.bfloat16), (90, torch.bfloat16), (5, torch.float32)])
def test_small_scales_of_large_queries(n, dt):
    """Every finite scale counts: queries 2^110 times as large with a scale 2^-110 of the usual one."""
    c = Case(n, [(n, 300), (1, 40)], 4, 2, 128, 16, dt)
    want = c.run(scale=0.0625)
    got = c.run(q=c.q * 2.0 ** 110, scale=0.0625 * 2.0 ** -110)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
