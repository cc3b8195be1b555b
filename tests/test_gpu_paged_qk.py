"""dspark_qk_norm_rope against the oracle in float64.

Tolerances count roundings.  The norm's sum of D squares is off by at most (D / 16 + 4) 2^-24
relative (16 products of a lane one after another, then pairs), its root by half of that, and
quotient, weight and rotation add a few more: 64 * 2^-24 of |y1| + |y2| covers them with the angle's
2^-22.  The output's own rounding is half a step: 2^-8 of the value for bf16, 2^-24 for fp32, 2^-4
or 2^-10 below the normals for an E4M3 code."""
import numpy as np
import pytest

from gpu_util import log
from oracle import paged as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def bdr():
    import block_draft_readout_amd as m
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _case(seed, n, hq, hkv, d, rot, dt, norm=True, far=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda")
         * (0.1 + 3 * torch.rand(n, hq + 2 * hkv, 1, generator=g, device="cuda"))).to(dt)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if norm else None for _ in range(2)]
    f = 1e4 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) * 2 / rot)
    pos = torch.randint(-5, far, (n,), generator=g, device="cuda").int()
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], w[0], w[1], f, pos


def _ref(x, pos, f, w, inter):
    y = oracle.norm_rope(_f64(x), pos.cpu().numpy(), _f64(f), None if w is None else _f64(w), 1e-6, inter)
    # what a value is made of: |y1| + |y2| of its pair, before the rotation
    z = np.abs(oracle.norm_rope(_f64(x), [0] * x.shape[0], _f64(f), None if w is None else _f64(w), 1e-6, inter))
    half = len(f)
    s = z.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        s[..., a] = s[..., b] = z[..., a] + z[..., b]
    return y, s


def _near(got, y, s, dt):
    tol = HALF[dt] * np.abs(y) + 64 * 2.0 ** -24 * s * 1.01 + 1e-37
    bad = np.abs(_f64(got) - y) > tol
    assert not bad.any(), (bad.sum(), np.abs(_f64(got) - y)[bad][:5], tol[bad][:5])


def _near_codes(codes, y, s, scale):
    v = _f64(codes.view(torch.float8_e4m3fn).float())
    z = np.clip(y / scale, -448, 448)
    tol = np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + 70 * 2.0 ** -24 * s / scale
    assert (np.abs(v - z) <= tol).all()


@pytest.mark.parametrize("n,hq,hkv,d,rot,dt,inter,norm", [
    (1, 40, 8, 128, 128, torch.bfloat16, False, True), (1, 1, 1, 64, 16, torch.float32, True, True),
    (3, 5, 5, 64, 64, torch.bfloat16, True, True), (17, 6, 2, 64, 32, torch.float32, True, True),
    (33, 8, 1, 256, 256, torch.bfloat16, False, True), (9, 4, 2, 256, 64, torch.float32, False, True),
    (50, 7, 7, 128, 48, torch.bfloat16, False, False), (2, 33, 3, 128, 128, torch.float32, False, False),
    (2048, 2, 1, 64, 64, torch.bfloat16, False, True), (2051, 3, 1, 128, 96, torch.bfloat16, True, True),
])
def test_queries_and_keys(n, hq, hkv, d, rot, dt, inter, norm):
    log(f"qk n={n} hq={hq} hkv={hkv} d={d} rot={rot} {dt} inter={inter}")
    q, k, v, wq, wk, f, pos = _case(n + d, n, hq, hkv, d, rot, dt, norm)
    got_q, got_k = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk, interleaved=inter)
    _near(got_q, *_ref(q, pos, f, wq, inter), dt)
    _near(got_k, *_ref(k, pos, f, wk, inter), dt)


@pytest.mark.parametrize("layout", ["NHD", "HND", "pairs"])
@pytest.mark.parametrize("n,hq,hkv,d,page,dt,fp8", [
    (1, 2, 1, 128, 16, torch.bfloat16, False), (37, 5, 1, 64, 24, torch.bfloat16, True),
    (70, 0, 4, 128, 1, torch.bfloat16, True), (13, 4, 2, 256, 5, torch.float32, False),
    (2100, 0, 3, 64, 64, torch.bfloat16, False), (2049, 1, 1, 128, 16, torch.bfloat16, True),
])
def test_cache_writes(n, hq, hkv, d, page, dt, fp8, layout):
    q, k, v, wq, wk, f, pos = _case(n + page, n, hq, hkv, d, d, dt)
    g = np.random.default_rng(n)
    pages = -(-(n + 40) // page)
    ct = torch.uint8 if fp8 else dt
    if layout == "NHD":
        kc, vc = (torch.empty(pages, page, hkv, d, dtype=dt, device="cuda").normal_().to(ct) for _ in range(2))
    elif layout == "HND":
        kc, vc = (torch.empty(pages, hkv, page, d, dtype=dt, device="cuda").normal_().to(ct).transpose(1, 2)
                  for _ in range(2))
    else:   # keys and values of a page beside each other, room behind every page
        both = torch.empty(pages, 3, page, hkv, d, dtype=dt, device="cuda").normal_().to(ct)
        kc, vc = both[:, 0], both[:, 1]
    scales = [torch.tensor(0.02 + 0.05 * g.random(hkv), dtype=torch.float32, device="cuda") for _ in range(2)] \
        if fp8 else [None, None]
    slots = g.permutation(pages * page)[:n].astype(np.int32)
    slots[g.random(n) < 0.1] = -1
    slots[-1:] = pages * page      # outside
    before = [c.clone() for c in (kc, vc)]
    got_q, got_k = bdr().dspark_qk_norm_rope(
        q if hq else None, k, v, pos, f, q_weight=wq, k_weight=wk, slots=torch.from_numpy(slots).cuda(),
        k_cache=kc, v_cache=vc, k_scale=scales[0], v_scale=scales[1])
    assert got_k is None and (got_q is None) == (hq == 0)
    if hq:
        _near(got_q, *_ref(q, pos, f, wq, False), dt)
    fine = np.flatnonzero((slots >= 0) & (slots < pages * page))
    page_of, in_page = slots[fine] // page, slots[fine] % page
    wrote_k, wrote_v = kc[page_of, in_page], vc[page_of, in_page]
    y, s = _ref(k, pos, f, wk, False)
    rows = torch.from_numpy(fine).cuda()
    if fp8:
        for c, z, zs, sc in ((wrote_k, y, s, scales[0]), (wrote_v, _f64(v), np.abs(_f64(v)), scales[1])):
            _near_codes(c, z[fine], zs[fine], _f64(sc)[:, None])
    else:
        _near(wrote_k, y[fine], s[fine], dt)
        assert torch.equal(wrote_v, v[rows])
    for c, was in ((kc, before[0]), (vc, before[1])):   # and nothing else
        now = c.clone()
        now[page_of, in_page] = was[page_of, in_page]
        assert torch.equal(now, was)


def test_codes_of_large_values_and_infinities():
    n, d = 4, 64
    v = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    v[0] = 1e30
    v[1] = float("-inf")
    v[2, 0, :8] = torch.tensor([448.0, 449, 464, 465, 480, -1e4, 0.0, -0.0])
    v[3] = float("nan")
    k = torch.ones_like(v)
    kc, vc = (torch.zeros(1, 4, 1, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    one = torch.ones(1, device="cuda")
    i = torch.arange(4, dtype=torch.int32, device="cuda")
    bdr().dspark_qk_norm_rope(None, k, v, i, torch.zeros(32, device="cuda"), slots=i, k_cache=kc,
                              v_cache=vc, k_scale=one, v_scale=one)
    got = vc.view(torch.float8_e4m3fn).float().cpu()
    assert (got[0, 0] == 448).all() and (got[0, 1] == -448).all()
    assert got[0, 2, 0, :8].tolist() == [448.0, 448, 448, 448, 448, -448, 0, 0]
    assert torch.isnan(got[0, 3]).all()
    assert (kc.view(torch.float8_e4m3fn).float() == 1).all()


def test_norm_alone_of_zeros_and_in_place():
    q, k, _, wq, wk, f, pos = _case(3, 19, 4, 2, 128, 128, torch.bfloat16)
    q, k = q.contiguous(), k.contiguous()
    q[3] = 0
    want = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk)
    assert (want[0][3] == 0).all()
    got = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_no_rows():
    q, k, v, wq, wk, f, pos = _case(4, 0, 4, 2, 128, 128, torch.bfloat16)
    got = bdr().dspark_qk_norm_rope(q, k, None, pos, f, q_weight=wq, k_weight=wk)
    assert got[0].shape == (0, 4, 128) and got[1].shape == (0, 2, 128)
