"""The binding of the paged attention's calls refuses device tensors of other shapes, types,
strides and devices, with nothing launched."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture()
def m():
    import block_draft_readout_amd
    return block_draft_readout_amd


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _refused(kinds, fn, good, **change):
    with pytest.raises(kinds):
        fn(**{**good, **change})


def test_slots(m):
    good = dict(cached=_ints(3, 5), new_tokens=_ints(1, 1), block_table=_ints(0, 1, 2, 3).view(2, 2),
                page_count=_ints(1, 2), free_pages=_ints(7, 8), free_count=_ints(2), page_size=4, max_rows=4)
    m.spec_slots(**good)
    bad = (ValueError, TypeError)
    for name in ("cached", "new_tokens", "page_count", "free_count", "block_table"):
        _refused(bad, m.spec_slots, good, **{name: good[name].long()})
        _refused(bad, m.spec_slots, good, **{name: None})
    for name in ("new_tokens", "page_count", "free_count"):
        _refused(bad, m.spec_slots, good, **{name: _ints(1, 2, 3)})
        _refused(bad, m.spec_slots, good, **{name: good[name].cpu()})
    _refused(bad, m.spec_slots, good, block_table=_ints(0, 1, 2, 3, 4, 5, 6, 7).view(2, 4)[:, ::2])
    _refused(bad, m.spec_slots, good, out={"slots": _ints(1)})
    _refused(bad, m.spec_slots, good, out={"other": _ints(1)})
    _refused(bad, m.spec_slots, good, max_rows=-1)
    _refused(m.BdrError, m.spec_slots, good, page_size=0)
    _refused(m.BdrError, m.spec_slots, good, out={"kv_len": good["cached"]})


def test_qk(m):
    x = torch.randn(3, 8, 64, device="cuda").to(torch.bfloat16)
    cache = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    good = dict(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], positions=_ints(0, 1, 2), inv_freq=torch.ones(32, device="cuda"),
                slots=_ints(0, 1, 2), k_cache=cache, v_cache=cache.clone())
    m.dspark_qk_norm_rope(**good)
    bad = (ValueError, TypeError, m.BdrError)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    _refused(bad, m.dspark_qk_norm_rope, good, q_weight=w)
    _refused(bad, m.dspark_qk_norm_rope, good, q_weight=w.float(), k_weight=w)
    _refused(bad, m.dspark_qk_norm_rope, good, q=good["q"].float())
    _refused(bad, m.dspark_qk_norm_rope, good, q=good["q"][:2])
    _refused(bad, m.dspark_qk_norm_rope, good, k=x[:, 4:6].transpose(1, 2))
    _refused(bad, m.dspark_qk_norm_rope, good, v=None)
    _refused(bad, m.dspark_qk_norm_rope, good, v=x[:, 6:7])
    _refused(bad, m.dspark_qk_norm_rope, good, slots=None)
    _refused(bad, m.dspark_qk_norm_rope, good, positions=_ints(0, 1))
    _refused(bad, m.dspark_qk_norm_rope, good, inv_freq=torch.ones(40, device="cuda"))
    _refused(bad, m.dspark_qk_norm_rope, good, inv_freq=torch.ones(32, device="cuda").double())
    _refused(bad, m.dspark_qk_norm_rope, good, k_cache=None)
    _refused(bad, m.dspark_qk_norm_rope, good, v_cache=good["k_cache"])
    _refused(bad, m.dspark_qk_norm_rope, good, v_cache=cache.transpose(0, 1).contiguous().transpose(0, 1))
    _refused(bad, m.dspark_qk_norm_rope, good, k_cache=cache.view(torch.uint8))
    one = torch.ones(2, device="cuda")
    _refused(bad, m.dspark_qk_norm_rope, good, k_scale=one, v_scale=one)
    _refused(bad, m.dspark_qk_norm_rope, good, k_scale=one)
    _refused(bad, m.dspark_qk_norm_rope, good, q=None, q_out=torch.empty_like(x[:, :4]))
    _refused(bad, m.dspark_qk_norm_rope, good, q_out=x[:, :4])
    # one entry expanded over the positions would be written many times
    _refused(bad, m.dspark_qk_norm_rope, good, k_cache=cache[:1].expand(4, -1, -1, -1),
             v_cache=good["v_cache"][:1].expand(4, -1, -1, -1))


def test_attention(m):
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    cache = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, k_cache=cache, v_cache=cache, block_table=_ints(0, 1, 2, 3).view(2, 2),
                query_offsets=_ints(0, 1, 3), kv_len=_ints(4, 9))
    m.dflash_paged_attention(**good)
    bad = (ValueError, TypeError, m.BdrError)
    _refused(bad, m.dflash_paged_attention, good, q=q.float())
    _refused(bad, m.dflash_paged_attention, good, q=q.half())
    _refused(bad, m.dflash_paged_attention, good, q=q.transpose(1, 2))
    _refused(bad, m.dflash_paged_attention, good, q=q[:, :3])
    _refused(bad, m.dflash_paged_attention, good, k_cache=cache[..., :32])
    _refused(bad, m.dflash_paged_attention, good, v_cache=cache[:3])
    _refused(bad, m.dflash_paged_attention, good, block_table=good["block_table"].long())
    _refused(bad, m.dflash_paged_attention, good, query_offsets=_ints(0, 1))
    _refused(bad, m.dflash_paged_attention, good, kv_len=_ints(4))
    _refused(bad, m.dflash_paged_attention, good, kv_len=good["kv_len"].cpu())
    _refused(bad, m.dflash_paged_attention, good, scale=0.0)
    _refused(bad, m.dflash_paged_attention, good, window=-2)
    _refused(bad, m.dflash_paged_attention, good, out=q)
    _refused(bad, m.dflash_paged_attention, good, out=q.float())
    _refused(bad, m.dflash_paged_attention, good, k_scale=torch.ones(2, device="cuda"))
    wide = torch.zeros(2, 300, dtype=torch.int32, device="cuda")
    _refused(bad, m.dflash_paged_attention, good, block_table=wide,
             workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
