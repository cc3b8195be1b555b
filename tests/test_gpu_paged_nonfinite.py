"""dflash_paged_attention on scores that are no numbers: a row that sees one has out and lse NaN, every
other row what it has without it.  A score of -inf is a weight of 0."""
import pytest

from gpu_util import log
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
# n, hq, hkv, d, type, e4m3: 16-row tiles, tiles of 128 and of 256 rows; each over a context of one launch and
# over one that is shared and joined
KINDS = [(1, 4, 2, 128, BF, False), (9, 10, 2, 128, BF, False), (3, 4, 1, 64, BF, True), (9, 8, 2, 128, BF, True),
         (5, 4, 2, 256, BF, False), (7, 6, 2, 64, F32, False), (40, 4, 2, 128, BF, False), (30, 6, 2, 64, BF, True),
         (90, 4, 2, 128, BF, False), (80, 6, 2, 128, BF, True), (50, 4, 1, 256, BF, False), (30, 4, 2, 128, F32, False)]
LENGTHS = [180, 2100]


def _case(kind, length):
    n, hq, hkv, d, dt, fp8 = KINDS[kind]
    log(f"nonfinite {KINDS[kind]} over {length}")
    return Case(kind + length, [(n, length), (2, 40)], hq, hkv, d, 16, dt, fp8, behind=1)


def _same(a, b, rows):
    assert torch.equal(a[0][rows], b[0][rows]) and torch.equal(a[1][rows], b[1][rows])


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_query(kind, length):
    c = _case(kind, length)
    n, hq = c.lens[0][0], c.hq
    want = c.run()
    c.check(want)
    q = c.q.clone()
    q[n - 1, hq - 1, 5] = float("nan")
    out, lse = c.run(q=q)
    assert out[n - 1, hq - 1].isnan().all() and lse[n - 1, hq - 1].isnan()
    rest = torch.ones(c.rows - 1, hq, dtype=torch.bool, device="cuda")
    rest[n - 1, hq - 1] = False
    _same((out[:-1], lse[:-1]), (want[0][:-1], want[1][:-1]), rest)


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_key(kind, length, at):
    """A NaN key of one kv head: only rows that see it, of that head's queries."""
    c = _case(kind, length)
    n, group = c.lens[0][0], c.hq // c.hkv
    want = c.run()
    t = {"first": 0, "middle": length - n + n // 2, "last": length - 1}[at]
    c.kc[c.table[0, t // 16].long(), t % 16, 0, 3] = 0x7F if c.fp8 else float("nan")
    out, lse = c.run()
    hit = torch.zeros(c.rows - 1, c.hq, dtype=torch.bool, device="cuda")
    hit[max(0, t - (length - n)):n, :group] = True
    out, lse = out[:-1], lse[:-1]
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    _same((out, lse), (want[0][:-1], want[1][:-1]), ~hit)


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", [k for k in range(len(KINDS)) if not KINDS[k][5]])
def test_infinite_keys(kind, length):
    """A score of -inf weighs nothing, one of +inf leaves no number."""
    c = _case(kind, length)
    n, group = c.lens[0][0], c.hq // c.hkv
    c.q[..., 0] = c.q[..., 0].abs() + 0.5
    where = c.table[0, 1].long(), 5          # position 21, which all rows see
    c.kc[where[0], where[1], 0, 0] = -1e30
    want = c.run()
    c.kc[where[0], where[1], 0, 0] = float("-inf")
    got = c.run()
    _same((got[0][:-1], got[1][:-1]), (want[0][:-1], want[1][:-1]), slice(None))
    c.kc[where[0], where[1], 0, 0] = float("inf")
    out, lse = c.run()
    assert out[:n, :group].isnan().all() and lse[:n, :group].isnan().all()
    _same((out[:-1], lse[:-1]), (want[0][:-1], want[1][:-1]), (slice(None), slice(group, None)))
    _same((out, lse), want, slice(n, n + 2))


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", [k for k in range(len(KINDS)) if not KINDS[k][5]])
def test_infinite_values(kind, length):
    """An infinite value that all rows of a request see is infinite in its feature, and only there; two
    of both signs leave no number."""
    n, hq, hkv, d, dt, _ = KINDS[kind]
    c = Case(kind + length, [(n, length), (2, 40)], hq, hkv, d, 16, dt, spread=0.5, behind=1)
    group = hq // hkv
    want = c.run(causal=False)
    inf = float("inf")
    at = lambda t: (c.table[0, t // 16].long(), t % 16, 0)
    c.vc[at(0)][3], c.vc[at(length - 1)][4] = inf, -inf
    c.vc[at(11)][5], c.vc[at(length // 2)][5] = inf, -inf
    out, lse = c.run(causal=False)
    assert (out[:n, :group, 3] == inf).all() and (out[:n, :group, 4] == -inf).all()
    assert out[:n, :group, 5].isnan().all()
    out, one = out.clone(), want[0].clone()
    out[:n, :group, 3:6] = one[:n, :group, 3:6] = 0
    _same((out[:-1], lse[:-1]), (one[:-1], want[1][:-1]), slice(None))


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", [k for k in range(len(KINDS)) if not KINDS[k][5] and KINDS[k][0] > 1])
def test_large_values_that_others_see(kind, length):
    """Values near the largest number, of positions that a row does not see, do not reach it."""
    c = _case(kind, length)
    n, group = c.lens[0][0], c.hq // c.hkv
    want = c.run()
    c.vc[c.table[0, (length - 1) // 16].long(), (length - 1) % 16, 0] = 3e38
    got = c.run()
    for a, b in zip(got, want):   # all but the last token's rows of that head
        a[n - 1, :group] = b[n - 1, :group] = 0
    _same((got[0][:-1], got[1][:-1]), (want[0][:-1], want[1][:-1]), slice(None))


def test_rows_with_no_weight():
    """All scores that a row sees are -inf: no weight, as where it sees nothing."""
    for n, length in ((2, 100), (90, 100), (2, 3000)):
        c = Case(n + length, [(n, length), (2, 40)], 4, 2, 128, 16)
        c.q[..., 0] = 1
        t = torch.arange(length, device="cuda")
        c.kc[c.table[0].long()[t // 16], t % 16, 1, 0] = float("-inf")
        want = c.run()
        assert (want[0][:n, 2:] == 0).all() and (want[1][:n, 2:] == float("-inf")).all()
        c.check(want, requests=[1])


E4M3 = [k for k in range(len(KINDS)) if KINDS[k][5]]


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", E4M3)
def test_scale_that_is_no_number(kind, length, scale):
    """Of one kv head's keys: its rows are NaN where they see something, the others as they were."""
    c = _case(kind, length)
    group = c.hq // c.hkv
    lens = [(n, length) for n, length in c.lens]
    c.kv_len[1] = 0                          # request 1 sees nothing
    want = c.run()
    c.scales[0][0] = scale
    out, lse = c.run()
    n = lens[0][0]
    assert out[:n, :group].isnan().all() and lse[:n, :group].isnan().all()
    assert (out[n:n + 2] == 0).all() and (lse[n:n + 2] == float("-inf")).all()
    _same((out, lse), want, (slice(0, n), slice(group, None)))


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("kind", E4M3)
def test_negative_scales(kind, length):
    c = _case(kind, length)
    for scale, held in zip(c.scales, (c.k, c.v)):
        scale[0] *= -1
        for x in held:
            x[:, 0] *= -1
    for causal, window in ((True, 0), (False, 70)):
        c.check(c.run(causal=causal, window=window), causal, window)
