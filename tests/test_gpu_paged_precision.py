"""How many bits of its weights dflash_paged_attention keeps in the product with the values.

Tolerance of an output, A = sum_t w_t |v_t|, s the largest sum of |scale q_d k_d| of the row, L keys,
v the largest value, eps = 2^-24:
  output     half a step of bf16: 2^-8 |out|
  weights    half a step each, W A: 2^-11 (fp16, for e4m3 caches), 2^-15 (few rows of bf16: the
             upper 8 bits leave at most 2^-7, which is rounded, 2^-8 of it)
  fp16       weights below 2^-21 of the reference's have a step of 2^-31 of it, the reference's own
             weight is 1 of the sum: half a step of L weights, L 2^-32 v
  the rest   scores, exponentials and fp32 sums: 2 ((D + 4) eps s + (L + 70) eps) A
Values of both signs nearly cancel in many outputs, whose own rounding then hides nothing."""
import numpy as np
import pytest

from gpu_util import log
from oracle import paged as oracle
from test_gpu_paged_attention import EPS, Case, _f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _balance(c):
    """Values of both signs, the same magnitudes, every second key the negative of the one before."""
    for b, (_, length) in enumerate(c.lens):
        t = torch.arange(length, device="cuda")
        where = (c.table[b].long()[t // c.page], t % c.page)
        x = c.vc[where].clone()
        x[1::2] = x[0:2 * (length // 2):2]
        if c.fp8:
            x[1::2] ^= 0x80
            c.v[b] = _f64(x.view(torch.float8_e4m3fn).float()) * _f64(c.scales[1])[:, None]
        else:
            x[1::2] *= -1
            c.v[b] = _f64(x)
        c.vc[where] = x


def _check(c, got, weights, causal=True):
    out = _f64(got[0])
    q = _f64(c.q)
    for b, (n, length) in enumerate(c.lens):
        rows = slice(c.offsets[b], c.offsets[b] + n)
        ref, _, mass, s = oracle.attention(q[rows], c.k[b], c.v[b], length - n, c.d ** -0.5, causal, 0)
        rel = 2 * ((c.d + 4) * EPS * s + (length + 70) * EPS)[..., None]
        tol = 2.0 ** -8 * np.abs(ref) + (weights + rel) * mass
        if c.fp8:
            tol = tol + length * 2.0 ** -32 * np.abs(c.v[b]).max()
        err = np.abs(out[rows] - ref)
        assert (err <= tol * 1.01 + 1e-37).all(), (b, n, length, float((err / (tol + 1e-37)).max()))


# one token; 16-row tiles 1 to 4; row tiles of 128 and of 256
ROWS = [(1, 4), (2, 8), (4, 8), (5, 8), (6, 10), (20, 5), (40, 4)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,group", ROWS)
def test_weights_of_codes(n, group, d):
    log(f"weights of codes n={n} group={group} d={d}")
    for lens in ([(n, n + 6), (n, n + 1)], [(n, 1500), (n, 333)]):   # one launch; shares and their join
        c = Case(n + d, lens, 2 * group, 2, d, 16, fp8=True, spread=0.3)
        _balance(c)
        _check(c, c.run(causal=False), 2.0 ** -11, False)


@pytest.mark.parametrize("n,group,d", [(n, group, d) for n, group in ROWS[:4] for d in (64, 128, 256)
                                       if n * group <= (48 if d == 128 else 32 if d == 256 else 64)] + [(6, 10, 64)])
def test_weights_of_few_rows(n, group, d):
    log(f"weights of few rows n={n} group={group} d={d}")
    for lens in ([(n, n + 6), (n, n + 1)], [(n, 1500), (n, 333)]):
        c = Case(n + d, lens, 2 * group, 2, d, 16, spread=0.3)
        _balance(c)
        _check(c, c.run(causal=False), 2.0 ** -15, False)


@pytest.mark.parametrize("down", [20, 22, 26])
@pytest.mark.parametrize("n", [1, 50, 200])
def test_small_weights_of_codes(n, down):
    """One key's score lies 2^down above all others', whose values make the output."""
    c = Case(n + down, [(n, 3000 + n)], 1, 1, 128, 16, fp8=True)
    t = torch.arange(3000 + n, device="cuda")
    where = (c.table[0].long()[t // 16], t % 16)
    code = lambda x: torch.full((len(t), 1, 128), x, device="cuda").to(torch.float8_e4m3fn)
    k, v = code(0.0), code(1.125)
    k[7] = code(64.0)[0]
    v[7] = 0
    c.kc[where], c.vc[where] = k.view(torch.uint8), v.view(torch.uint8)
    c.k[0] = _f64(k.float()) * _f64(c.scales[0])[:, None]
    c.v[0] = _f64(v.float()) * _f64(c.scales[1])[:, None]
    top = 64 * _f64(c.scales[0])[0] * 128
    c.q.fill_(down * np.log(2) * 128 ** 0.5 / top)
    _check(c, c.run(causal=False), 2.0 ** -11, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_sine_and_cosine_are_rounded_once(interleaved):
    """Pairs of (1, 0) turn into (cos a, sin a): half a step of fp32, where the angle's own 2^-53 of at
    most 2^20 quarter turns, taken for its product and for 2 / pi, leaves 2^-32."""
    import block_draft_readout_amd as m
    n, d = 3000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(n, 1, d, device="cuda")
    one, zero = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    x[..., one] = 1
    pos = torch.randint(-(1 << 20), 1 << 20, (n,), generator=g, device="cuda").int()
    pos[0] = 0
    f = 1e4 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float32) * 2 / d)
    got = _f64(m.dspark_qk_norm_rope(x, x, None, pos, f, interleaved=interleaved)[0][:, 0])
    a = _f64(pos)[:, None] * _f64(f)
    for y, ref in ((got[:, one], np.cos(a)), (got[:, zero], np.sin(a))):
        step = np.spacing(np.abs(ref).astype(np.float32)).astype(np.float64)
        assert (np.abs(y - ref) <= 0.51 * step + 2.0 ** -32).all()
