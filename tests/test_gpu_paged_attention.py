"""dflash_paged_attention against the oracle in float64.

Tolerance of an output, from the roundings (eps = 2^-24, A = sum_t w_t |v_t|, s the largest sum of
|scale q_d k_d| of the row):
  output            half a step of its type: 2^-8 |out| (bf16), eps |out| (fp32)
  probabilities     bf16 products only: half a step each, 2^-8 A
  scores            a sum of D fp32 products: at most (D + 2) eps s, and 2 eps s more where the
                    exponent's argument is formed: a relative error of each weight and of their
                    sum, so twice that times A
  sums              of L weights and products: (L + 64) eps A, twice; the exponential 4 eps
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import paged as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 2.0 ** -24


def bdr():
    import block_draft_readout_amd as m
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Requests with (n, L) each over shuffled pages; everything that nobody sees is NaN."""

    def __init__(self, seed, lens, hq, hkv, d, page, dt=torch.bfloat16, fp8=False, layout="NHD", width=None,
                 before=0, behind=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.page, self.dt, self.fp8 = lens, hq, hkv, d, page, dt, fp8
        need = [-(-length // page) for _, length in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.width = width or max(1, max(need))
        table = np.full((len(lens), self.width), -1, dtype=np.int32)
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = order[at:at + c]
            at += c
        ct = torch.uint8 if fp8 else dt
        shape = (pages, page, hkv, d) if layout == "NHD" else (pages, hkv, page, d)

        def cache():
            c = torch.full(shape, 0x7F, dtype=ct, device="cuda") if fp8 else \
                torch.full(shape, float("nan"), dtype=ct, device="cuda")
            return c if layout == "NHD" else c.transpose(1, 2)

        self.kc, self.vc = cache(), cache()
        self.scales = [None, None]
        if fp8:
            self.scales = [torch.tensor(0.01 + 0.02 * rng.random(hkv), dtype=torch.float32, device="cuda")
                           for _ in range(2)]
        self.k, self.v = [], []
        for b, (_, length) in enumerate(lens):
            t = torch.arange(length)
            where = (torch.from_numpy(table[b][t.numpy() // page]).long().cuda(), (t % page).cuda())
            for c, held, scale in ((self.kc, self.k, self.scales[0]), (self.vc, self.v, self.scales[1])):
                x = torch.randn(length, hkv, d, generator=g, device="cuda") * 1.2 + 0.2
                if fp8:
                    x = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                    c[where] = x.view(torch.uint8)
                    held.append(_f64(x.float()) * _f64(scale)[:, None])
                else:
                    c[where] = x.to(dt)
                    held.append(_f64(x.to(dt)))
        self.offsets = np.cumsum([before] + [n for n, _ in lens]).astype(np.int32)
        self.rows = int(self.offsets[-1]) + behind
        q = torch.randn(self.rows, hq, d, generator=g, device="cuda")
        self.q = (q * (0.2 + spread * torch.rand(self.rows, hq, 1, generator=g, device="cuda"))).to(dt)
        self.table = torch.from_numpy(table).cuda()
        self.off = torch.from_numpy(self.offsets).cuda()
        self.kv_len = torch.tensor([length for _, length in lens], dtype=torch.int32, device="cuda")

    def run(self, **kw):
        kw = dict(dict(lse=True, k_scale=self.scales[0], v_scale=self.scales[1]), **kw)
        return bdr().dflash_paged_attention(kw.pop("q", self.q), kw.pop("k_cache", self.kc),
                                            kw.pop("v_cache", self.vc), kw.pop("table", self.table),
                                            kw.pop("offsets", self.off), kw.pop("kv_len", self.kv_len), **kw)

    def check(self, got, causal=True, window=0, scale=None, requests=None):
        out, lse = _f64(got[0]), _f64(got[1])
        scale = self.d ** -0.5 if scale is None else scale
        q = _f64(self.q)
        for b, (n, length) in enumerate(self.lens):
            if requests is not None and b not in requests:
                continue
            rows = slice(self.offsets[b], self.offsets[b] + n)
            ref, rl, mass, s = oracle.attention(q[rows], self.k[b], self.v[b], length - n, scale, causal, window)
            rel = 2 * ((self.d + 4) * EPS * s + (length + 70) * EPS)[..., None]
            if self.dt == torch.bfloat16:
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + rel) * mass
            else:
                tol = EPS * np.abs(ref) + rel * mass
            err = np.abs(out[rows] - ref)
            assert (err <= tol * 1.01 + 1e-37).all(), (b, n, length, float((err / (tol + 1e-37)).max()))
            none = rl == -np.inf
            assert np.array_equal(lse[rows] == -np.inf, none)
            assert (out[rows][none] == 0).all()
            # lse: the scores' error, the sum's, and its own rounding
            at = ~none
            tol = rel[..., 0] / 2 * 1.5 + 4 * EPS * np.abs(np.where(none, 0, rl)) + 4 * EPS
            assert (np.abs(lse[rows][at] - rl[at]) <= tol[at]).all()


SHAPES = [   # hq, hkv, d, page, dtype, fp8
    (40, 8, 128, 16, torch.bfloat16, False), (4, 4, 64, 24, torch.bfloat16, False),
    (6, 2, 256, 32, torch.bfloat16, False), (5, 1, 128, 1, torch.bfloat16, True),
    (8, 8, 64, 48, torch.bfloat16, True), (16, 2, 256, 16, torch.bfloat16, True),
    (6, 2, 64, 24, torch.float32, False), (3, 3, 128, 7, torch.float32, False),
    (4, 1, 256, 16, torch.float32, False),
]
LENS = {
    "one": [(1, 1)],
    "single": [(1, 1000)],
    "edges": [(1, 31), (1, 32), (1, 33), (2, 63), (3, 64), (1, 65), (1, 127), (4, 128), (1, 129), (1, 257)],
    "block": [(8, 8), (8, 300), (8, 77), (8, 1025)],
    "ragged": [(1, 5), (0, 40), (9, 9), (33, 500), (2, 0), (1, 640), (0, 0), (17, 18)],
    "chunk": [(150, 400), (1, 900)],
    "prompt": [(257, 257)],
}


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 40)])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(shape, lens, causal, window):
    hq, hkv, d, page, dt, fp8 = SHAPES[shape]
    log(f"attention {SHAPES[shape]} {lens} causal={causal} window={window}")
    c = Case(shape * 100 + len(lens), LENS[lens], hq, hkv, d, page, dt, fp8, layout="HND" if shape % 2 else "NHD",
             before=2 if lens == "ragged" else 0, behind=3)
    c.check(c.run(causal=causal, window=window), causal, window)


@pytest.mark.parametrize("n,group", [(1, 1), (1, 32), (1, 33), (2, 16), (8, 4), (8, 5), (9, 8), (16, 8), (13, 10),
                                     (40, 3), (200, 1)])
def test_rows_of_every_variant(n, group):
    log(f"attention n={n} group={group}")
    c = Case(n + group, [(n, 700), (n, 211)], 2 * group, 2, 128, 16)
    c.check(c.run())
    c.check(c.run(causal=False, window=65), False, 65)


def test_many_requests():
    """More requests than lanes, few of them long, some without tokens."""
    g = np.random.default_rng(3)
    lens = [(int(g.integers(0, 4)), int(g.integers(0, 40))) for _ in range(150)]
    lens = [(min(n, length), length) for n, length in lens]
    lens[70], lens[149] = (3, 2000), (2, 1500)
    c = Case(4, lens, 4, 2, 64, 16)
    c.check(c.run())


@pytest.mark.parametrize("dt,fp8", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
def test_long_context_of_one_request(dt, fp8):
    """The keys of one row tile spread over many workgroups."""
    c = Case(6, [(3, 30000)], 4, 1, 128, 16, dt, fp8)
    c.check(c.run())
    c.check(c.run(window=9000), True, 9000)


def test_long_prompt_in_pairs_of_row_tiles():
    c = Case(7, [(700, 900), (650, 650)], 2, 1, 64, 16)
    c.check(c.run())


def test_scale_and_strided_queries():
    c = Case(8, [(5, 90), (2, 300)], 6, 2, 128, 16)
    wide = torch.full((c.rows, 3, 6, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1, :, 16:144] = c.q
    view = wide[:, 1, :, 16:144]
    assert not view.is_contiguous()
    got = c.run(q=view, scale=0.3)
    c.check(got, scale=0.3)
    same = c.run(scale=0.3)
    assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])


def test_rows_of_no_request_stay():
    c = Case(9, [(3, 50), (0, 9), (4, 4)], 4, 4, 64, 16, before=5, behind=6)
    out = torch.full((c.rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(out=out)
    c.check(got)
    assert (out[:5] == 7).all() and (out[-6:] == 7).all()


def test_tokens_before_the_first_position_see_nothing():
    """More new tokens than positions (a request that was cut short): the first ones see nothing."""
    for n, length in ((9, 4), (40, 0), (300, 130)):
        c = Case(10, [(n, length), (2, 33)], 4, 2, 128, 16)
        c.check(c.run())


def test_bad_pages_read_as_zeros():
    c = Case(11, [(4, 200), (4, 130)], 4, 2, 64, 16)
    table = c.table.clone()
    for b, col, entry in ((0, 3, -1), (0, 7, 1 << 30), (1, 8, c.kc.shape[0])):
        table[b, col] = entry
        c.k[b][16 * col:16 * col + 16] = 0
        c.v[b][16 * col:16 * col + 16] = 0
    c.check(c.run(table=table))


def test_lengths_past_the_table_are_cut():
    c = Case(12, [(2, 64), (3, 48)], 2, 1, 64, 16)
    long = c.kv_len.clone()
    long[0] = 1 << 30                       # the table has four columns
    c.check(c.run(kv_len=long))


def test_large_and_small_scores():
    """Scores of hundreds in both directions: the running maximum rises late and by much."""
    c = Case(13, [(1, 900), (8, 400)], 4, 2, 128, 16, spread=0.0)
    ramp = torch.linspace(-30, 30, c.kc.shape[0] * 16, device="cuda").view(-1, 16, 1, 1)
    seen = ~torch.isnan(c.kc)
    c.kc = torch.where(seen, c.kc + ramp.to(c.kc.dtype), c.kc)
    for b, (_, length) in enumerate(c.lens):
        t = np.arange(length)
        c.k[b] = _f64(c.kc[c.table[b][torch.from_numpy(t // 16).cuda()].long(), torch.from_numpy(t % 16).cuda()])
    c.q = torch.randn(c.rows, 4, 128, device="cuda").mul_(2).to(torch.bfloat16)
    c.check(c.run())


@pytest.mark.parametrize("rate", [0.04, 0.17, 0.6, -0.3])   # scores' growth with a key
@pytest.mark.parametrize("n, hq, hkv, d, dt", [(1, 4, 1, 128, torch.bfloat16), (9, 5, 1, 64, torch.bfloat16),
                                               (90, 2, 2, 128, torch.bfloat16), (300, 1, 1, 128, torch.bfloat16),
                                               (150, 1, 1, 256, torch.bfloat16), (40, 2, 1, 128, torch.float32),
                                               (7, 2, 2, 64, torch.float32)])
def test_scores_that_grow(n, hq, hkv, d, dt, rate):
    c = Case(hq * d + n, [(n, 700), (min(n, 33), 33)], hq, hkv, d, 16, dt, spread=0.5)
    c.q[..., 0] = d ** 0.5
    for b, (_, length) in enumerate(c.lens):
        t = torch.arange(length, device="cuda")
        ramp = (rate * t).to(dt)
        c.kc[c.table[b].long()[t // c.page], t % c.page, :, 0] = ramp[:, None]
        c.k[b][:, :, 0] = _f64(ramp)[:, None]
    for causal, window in ((True, 0), (False, 0), (True, 97)):
        c.check(c.run(causal=causal, window=window), causal=causal, window=window)


def test_caches_beyond_32_bit_offsets():
    """Pages of 4 MB apart: the last ones lie past 2^32 elements."""
    hkv, d, page = 1, 128, 16
    lens = [(4, 300)]
    c = Case(14, lens, 4, hkv, d, page)
    pages = 2100
    big = torch.empty(pages * (1 << 21) + 4096, dtype=torch.bfloat16, device="cuda")
    place = torch.randperm(60)[:c.kc.shape[0]] + 2040
    views = []
    for i, cache in enumerate((c.kc, c.vc)):
        view = big[2048 * i:].as_strided((pages, page, hkv, d), (1 << 21, d, d, 1), 2048 * i + big.storage_offset())
        view[place.cuda()] = cache
        views.append(view)
    table = torch.where(c.table >= 0, place.int().cuda()[c.table.clamp(min=0).long()], -1).int()
    c.check(c.run(k_cache=views[0], v_cache=views[1], table=table))
    # and written there
    m = bdr()
    slots = torch.tensor([pages * page - 1, 2050 * page + 3], dtype=torch.int32, device="cuda")
    k = torch.randn(2, 1, d, device="cuda").to(torch.bfloat16)
    v = torch.randn(2, 1, d, device="cuda").to(torch.bfloat16)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    m.dspark_qk_norm_rope(None, k, v, zero, torch.ones(64, device="cuda"), slots=slots, k_cache=views[0],
                          v_cache=views[1])
    for s, x, y in zip(slots.tolist(), k, v):
        assert torch.equal(views[0][s // page, s % page], x) and torch.equal(views[1][s // page, s % page], y)


def test_same_bits_again():
    c = Case(15, [(8, 3000), (8, 90), (8, 1234)], 10, 2, 128, 16)
    a, b = c.run(causal=False), c.run(causal=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows_or_requests():
    c = Case(16, [(0, 20)], 4, 2, 64, 16)
    assert c.run()[0].shape == (0, 4, 64)
    c = Case(17, [(3, 20)], 4, 2, 64, 16)
    out = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    c.run(table=c.table[:0], offsets=c.off[:1], kv_len=e, out=out)
    assert (out == 5).all()
