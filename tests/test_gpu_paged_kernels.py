"""Every kernel of dflash_paged_attention, with weights that are exact: powers of two.

Queries have four features of 1 or -1, keys small whole numbers, and the scale is log 2, so that a
score is a whole power of two of at most 8 and its weight one to within a few eps = 2^-24, which no
rounding to bf16 or fp16 loses.  Tolerance of an output, A = sum_t w_t |v_t|, L keys:
  output    half a step of its type: 2^-8 |out| (bf16), eps |out| (fp32)
  weights   scale log2 e is off by 2 eps, a score of 8 and its reference by 8 times that and a
            rounding of 8 eps each, the exponential by 4: 60 eps
  sums      of L weights and products: (L + 70) eps; with the weights twice, out being a quotient
An output of many values of both signs is small: a key that is missed, taken twice or mistaken shows."""
import math

import numpy as np
import pytest

from gpu_util import log
from oracle import paged as oracle
from test_gpu_paged_attention import EPS, Case, _f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
SCALE = float(np.float32(math.log(2)))
# 16-row tiles of a few-row kernel, tiles of 128 and of 256 rows -> tokens of a request, 3 heads a kv head
TOKENS = {1: 5, 2: 9, 3: 14, 4: 19, "128": 33, "256": 90}
KERNELS = [(BF, False, d, rows) for d in (64, 128) for rows in TOKENS] + \
          [(BF, False, 256, rows) for rows in (1, 2, "128")] + \
          [(BF, True, 64, rows) for rows in (1, 2, 3, 4, "128")] + [(BF, True, 128, rows) for rows in TOKENS] + \
          [(BF, True, 256, rows) for rows in (1, 2, "128")] + \
          [(F32, False, d, rows) for d in (64, 128) for rows in (1, 2, "128")] + [(F32, False, 256, "128")]


def _whole_numbers(c, g):
    """Keys and queries of few whole numbers in place of a case's own."""
    if c.fp8:
        c.scales[0].fill_(0.5)
    for b, (_, length) in enumerate(c.lens):
        t = torch.arange(length, device="cuda")
        k = torch.randint(-2, 3, (length, c.hkv, c.d), generator=g, device="cuda").float()
        x = (k / 0.5).to(torch.float8_e4m3fn).view(torch.uint8) if c.fp8 else k.to(c.dt)
        c.kc[c.table[b].long()[t // c.page], t % c.page] = x
        c.k[b] = _f64(k)
        v = torch.randn(length, c.hkv, c.d, generator=g, device="cuda")
        x = (v / c.scales[1][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) if c.fp8 else v.to(c.dt)
        c.vc[c.table[b].long()[t // c.page], t % c.page] = x.view(torch.uint8) if c.fp8 else x
        c.v[b] = _f64(x.float()) * (_f64(c.scales[1])[:, None] if c.fp8 else 1)
    order = torch.rand(c.rows, c.hq, c.d, generator=g, device="cuda").argsort(-1)
    c.q = torch.where(order < 2, 1.0, torch.where(order < 4, -1.0, 0.0)).to(c.dt)


def _check(c, got, causal, window):
    out, lse = _f64(got[0]), _f64(got[1])
    q = _f64(c.q)
    half = 2.0 ** -8 if c.dt == BF else EPS
    for b, (n, length) in enumerate(c.lens):
        rows = slice(c.offsets[b], c.offsets[b] + n)
        ref, rl, mass, _ = oracle.attention(q[rows], c.k[b], c.v[b], length - n, SCALE, causal, window)
        rel = 2 * (60 + length + 70) * EPS
        err = np.abs(out[rows] - ref)
        tol = half * np.abs(ref) + rel * mass
        assert (err <= 1.01 * tol + 1e-37).all(), (b, n, length, float((err / (tol + 1e-37)).max()))
        none = rl == -np.inf
        assert np.array_equal(lse[rows] == -np.inf, none)
        # lse: the sum's error, and those of 8 log 2 and of itself
        at = ~none
        assert (np.abs(lse[rows][at] - rl[at]) <= rel / 2 + 40 * EPS).all()


@pytest.mark.parametrize("page", [16, 64, 7])
@pytest.mark.parametrize("shared", [False, True])   # one workgroup a row tile, or shares that are joined
@pytest.mark.parametrize("dt,fp8,d,rows", KERNELS)
def test_every_kernel(dt, fp8, d, rows, shared, page):
    log(f"kernel {dt} e4m3={fp8} d={d} rows={rows} shared={shared} page={page}")
    n = TOKENS[rows]
    few = isinstance(rows, int)
    longest = (1530 if few else 700) if shared else (450 if few else 230)
    c = Case(d + n, [(n, longest), (n, n + 3)], 6, 2, d, page, dt, fp8, layout="HND" if page == 64 else "NHD", width=None)
    m = pytest.importorskip("block_draft_readout_amd")
    need = m.lib().dflash_paged_attention_workspace_bytes(c.rows, c.hq, c.hkv, d, 0 if dt == F32 else 1, 2, c.width, page)
    assert (need > 0) == shared
    _whole_numbers(c, torch.Generator(device="cuda").manual_seed(n))
    for causal, window in ((True, 0), (False, 0), (True, 97)):
        _check(c, c.run(causal=causal, window=window, scale=SCALE), causal, window)
