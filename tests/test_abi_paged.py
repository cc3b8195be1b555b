"""Host-side checks of the paged attention's calls: sizes, strides, pointers, overlaps and
workspaces are refused with the documented codes before the device is touched, and the
binding refuses tensors of other shapes, types and places."""
import os

import pytest

P = 1 << 24     # aligned addresses far apart; never dereferenced: every call below fails before that


def at(i):
    return P * (i + 1) << 6


@pytest.fixture(scope="module")
def A():
    from block_draft_readout_amd import _abi
    if not os.path.exists(_abi.LIB_PATH):
        from block_draft_readout_amd import build
        build.build()
    _abi.load()
    return _abi


def _call(fn, defaults, changes):
    unknown = set(changes) - set(defaults)
    assert not unknown, unknown
    return fn(*{**defaults, **changes}.values())


def _slots(A, **k):
    d = dict(cached=at(0), new=at(1), batch=4, width=8, page=16, table=at(2), count=at(3), free=at(4),
             capacity=100, top=at(5), rows=20, offsets=at(6), kv_len=at(7), positions=at(8), slots=at(9),
             count_out=at(10), top_out=at(11), status=at(12), stream=None)
    return _call(A.load().spec_slots, d, k)


def test_slots_refusals(A):
    E, U = A.BDR_EINVAL, A.BDR_EUNSUPPORTED
    assert _slots(A, batch=-1) == E and _slots(A, batch=(1 << 20) + 1) == U
    assert _slots(A, width=0) == E and _slots(A, page=0) == E
    assert _slots(A, width=1 << 27, page=16) == U
    assert _slots(A, capacity=-1) == E and _slots(A, capacity=1 << 31) == U
    assert _slots(A, rows=-1) == E and _slots(A, rows=(1 << 24) + 1) == U
    for name in ("cached", "new", "table", "count", "free", "top", "offsets", "kv_len", "positions", "slots",
                 "count_out", "top_out", "status"):
        assert _slots(A, **{name: None}) == E, name
        assert _slots(A, **{name: at(20) + 2}) == E, name
    # outputs over inputs and over each other; the two that may be their inputs shifted by one
    assert _slots(A, kv_len=at(0)) == E and _slots(A, slots=at(8) + 76) == E
    assert _slots(A, table=at(3) - 4) == E and _slots(A, free=at(5) - 396) == E
    assert _slots(A, count_out=at(3) + 4) == E and _slots(A, top_out=at(3)) == E
    assert _slots(A, count_out=at(1)) == E and _slots(A, count_out=at(5), top=at(5)) == E
    assert _slots(A, status=at(11)) == E and _slots(A, offsets=at(10)) == E


def _qk(A, **k):
    d = dict(q=at(0), qr=1024, qh=128, k=at(1), kr=256, kh=128, v=at(2), vr=256, vh=128, rows=10, hq=8, hkv=2,
             dim=128, dt=A.BDR_BF16, pos=at(3), freq=at(4), rot=128, inter=0, wq=at(5), wk=at(6), eps=1e-6,
             q_out=at(7), k_out=at(8), slots=at(9), kc=at(10), vc=at(11), pages=9, page=16,
             ps=16 * 256, ts=256, hs=128, ks=None, vs=None, stream=None)
    return _call(A.load().dspark_qk_norm_rope, d, k)


def test_qk_refusals(A):
    E, U = A.BDR_EINVAL, A.BDR_EUNSUPPORTED
    assert _qk(A, dt=7) == E and _qk(A, dt=A.BDR_BF16_PACKED) == E
    assert _qk(A, rows=-1) == E and _qk(A, rows=1 << 24) == U
    assert _qk(A, hq=-1) == E and _qk(A, hkv=0) == E and _qk(A, hq=1023) == U
    for dim in (0, 32, 96, 136, 512):
        assert _qk(A, dim=dim) == U
    for rot in (0, 8, 24, 144, -16):
        assert _qk(A, rot=rot) == E
    for eps in (-1.0, float("nan"), float("inf")):
        assert _qk(A, eps=eps) == E
    assert _qk(A, wq=None) == E and _qk(A, wk=None) == E and _qk(A, wq=at(5) + 8) == E
    for name in ("qr", "qh", "kr", "kh", "vr", "vh"):
        assert _qk(A, **{name: 132}) == E and _qk(A, **{name: -128}) == E, name
        assert _qk(A, **{name: 1 << 45}) == U, name
    for name in ("q", "k", "v", "q_out", "pos", "freq", "slots"):
        assert _qk(A, **{name: None}) == E, name
        assert _qk(A, **{name: at(20) + 2}) == E, name
    assert _qk(A, kc=None) == E and _qk(A, vc=None) == E and _qk(A, kc=at(10) + 8) == E
    assert _qk(A, k_out=None, kc=None, vc=None) == E            # keys would go nowhere
    assert _qk(A, kc=None, vc=None, ks=at(12), vs=at(13)) == E  # scales without a cache
    assert _qk(A, ks=at(12)) == E and _qk(A, vs=at(12)) == E
    assert _qk(A, dt=A.BDR_F32, ks=at(12), vs=at(13)) == E      # codes go with bf16
    assert _qk(A, pages=0) == E and _qk(A, page=0) == E and _qk(A, pages=1 << 28) == U
    assert _qk(A, ts=260) == E and _qk(A, hs=-128) == E and _qk(A, ks=at(12), vs=at(13), ts=264) == E
    assert _qk(A, ps=1 << 30) == U and _qk(A, ts=1 << 30) == U and _qk(A, hs=1 << 30) == U


def test_qk_overlaps(A):
    E = A.BDR_EINVAL
    # elements of the cache over each other: tokens, heads, pages, keys over values
    assert _qk(A, ts=128) == E and _qk(A, hs=64) == E and _qk(A, ps=16 * 256 - 128) == E
    assert _qk(A, vc=at(10)) == E and _qk(A, vc=at(10) + 256) == E and _qk(A, vc=at(10) + 9 * 8192 - 16) == E
    # outputs over inputs, over each other and over the cache
    assert _qk(A, q_out=at(0) + 16) == E and _qk(A, q_out=at(1)) == E and _qk(A, k_out=at(7)) == E
    assert _qk(A, q_out=at(0), qr=1088) == E and _qk(A, q_out=at(2)) == E
    assert _qk(A, k_out=at(1), kr=512) == E and _qk(A, k_out=at(0)) == E
    assert _qk(A, kc=at(0)) == E and _qk(A, vc=at(2) - 16) == E and _qk(A, kc=at(7)) == E
    for name in ("pos", "freq", "wq", "wk", "slots"):
        assert _qk(A, **{name: at(7) + 16}) == E, name
        assert _qk(A, **{name: at(11) + 32}) == E, name
    assert _qk(A, rows=0, q=None, k=None, v=None, q_out=None, pos=None, freq=None, slots=None) == A.BDR_OK


def _attn(A, **k):
    d = dict(q=at(0), qr=1024, qh=128, rows=10, hq=8, hkv=2, dim=128, dt=A.BDR_BF16, kc=at(1), vc=at(2), pages=9,
             page=16, ps=16 * 256, ts=256, hs=128, ks=None, vs=None, table=at(3), batch=3, width=300,
             offsets=at(4), kv_len=at(5), scale=0.1, causal=1, window=0, out=at(6), lse=at(7), ws=at(8),
             n=1 << 30, stream=None)
    return _call(A.load().dflash_paged_attention, d, k)


def test_attention_refusals(A):
    E, U, W = A.BDR_EINVAL, A.BDR_EUNSUPPORTED, A.BDR_EWORKSPACE
    assert _attn(A, dt=9) == E and _attn(A, rows=-1) == E and _attn(A, rows=1 << 28) == U
    assert _attn(A, hq=0) == E and _attn(A, hq=7) == E and _attn(A, hkv=0) == E and _attn(A, hq=1024) == U
    assert _attn(A, dim=80) == U
    assert _attn(A, batch=-1) == E and _attn(A, batch=(1 << 20) + 1) == U and _attn(A, width=0) == E
    assert _attn(A, width=1 << 27) == U
    assert _attn(A, pages=0) == E and _attn(A, page=0) == E and _attn(A, pages=1 << 28) == U
    assert _attn(A, ps=1 << 30) == U
    assert _attn(A, ts=4) == E and _attn(A, ps=-8) == E and _attn(A, ks=at(9)) == E
    assert _attn(A, dt=A.BDR_F32, ks=at(9), vs=at(10)) == E and _attn(A, ks=at(9) + 1, vs=at(10)) == E
    assert _attn(A, qr=1020) == E and _attn(A, qh=-8) == E
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(A, scale=scale) == E
    assert _attn(A, window=-1) == E
    for name in ("q", "kc", "vc", "table", "offsets", "kv_len", "out"):
        assert _attn(A, **{name: None}) == E, name
        assert _attn(A, **{name: at(20) + 2}) == E, name
    assert _attn(A, lse=at(7) + 1) == E
    assert _attn(A, ws=None) == W and _attn(A, ws=at(8) + 16) == W and _attn(A, n=1000) == W
    for name in ("out", "lse", "ws"):
        for i in (0, 1, 2, 3, 4, 5):
            assert _attn(A, **{name: at(i)}) == E, (name, i)
    assert _attn(A, lse=at(6)) == E and _attn(A, ws=at(6)) == E and _attn(A, ks=at(6), vs=at(9)) == E
    none = dict(q=None, kc=None, vc=None, table=None, offsets=None, kv_len=None, out=None, lse=None, ws=None, n=0)
    assert _attn(A, rows=0, **none) == A.BDR_OK and _attn(A, batch=0, **none) == A.BDR_OK


def test_attention_workspace(A):
    f = A.load().dflash_paged_attention_workspace_bytes
    need = f(10, 8, 2, 128, A.BDR_BF16, 3, 300, 16)
    assert 0 < need < 1 << 30 and need % 256 == 0
    assert f(0, 8, 2, 128, A.BDR_BF16, 3, 300, 16) == 0 and f(10, 8, 2, 128, A.BDR_BF16, 0, 300, 16) == 0
    assert f(10, 8, 3, 128, A.BDR_BF16, 3, 300, 16) == 0 and f(10, 8, 2, 100, A.BDR_BF16, 3, 300, 16) == 0


def test_binding_refusals(A):
    torch = pytest.importorskip("torch")
    import block_draft_readout_amd as m
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 64)
    cache = torch.zeros(3, 4, 2, 64)
    with pytest.raises(ValueError):     # not on a device
        m.spec_slots(i, i, i.view(2, 1), i, i, i[:1], 4, 8)
    with pytest.raises(TypeError):
        m.spec_slots([0, 1], i, i.view(2, 1), i, i, i[:1], 4, 8)
    with pytest.raises(ValueError):
        m.dspark_qk_norm_rope(x, x, None, i, torch.zeros(32))
    with pytest.raises(TypeError):
        m.dspark_qk_norm_rope(x, None, None, i, torch.zeros(32))
    with pytest.raises(ValueError):
        m.dflash_paged_attention(x, cache, cache, i.view(2, 1), i, i)
    with pytest.raises(TypeError):
        m.dflash_paged_attention(None, cache, cache, i.view(2, 1), i, i)
