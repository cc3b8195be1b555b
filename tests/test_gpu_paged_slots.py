"""spec_slots against the oracle: whole numbers, equal."""
import numpy as np
import pytest

from gpu_util import dev, log
from oracle import paged as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def bdr():
    import block_draft_readout_amd as m
    return m


def _case(seed, batch, width, page, new, over=0.0, spare=None, ahead=True, ragged=True):
    """Requests with distinct pages, some of them over, and the other pages on the stack."""
    g = np.random.default_rng(seed)
    room = width * page
    fresh = g.integers(0, new + 1, batch) if ragged else np.full(batch, new)
    cached = np.array([g.integers(0, max(1, room - int(n) + 1)) for n in fresh])
    held = -(-cached // page)
    if ahead:
        held = np.minimum(width, held + (g.random(batch) < 0.3))
    cached = np.where(g.random(batch) < over, -1, cached)
    total = batch * width
    order = g.permutation(total)
    table = np.full((batch, width), -5)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    left = order[at:] if spare is None else order[at:at + spare]
    stack = np.full(total, -9)
    stack[:len(left)] = left
    i32 = lambda x: np.ascontiguousarray(x, dtype=np.int32)
    return [i32(x) for x in (cached, fresh, table, held, stack, [len(left)])]


def _check(args, page, max_rows, in_place=False):
    ref = oracle.slots(*[a[0] if i == 5 else a for i, a in enumerate(args)], page, max_rows)
    t = [dev(a) for a in args]
    out = {"page_count": t[3], "free_count": t[5]} if in_place else None
    got = bdr().spec_slots(*t, page, max_rows, out=out)
    torch.cuda.synchronize()
    for name in ("query_offsets", "kv_len", "positions", "slots", "page_count", "free_count", "status"):
        assert np.array_equal(got[name].cpu().numpy(), ref[name]), name
    assert np.array_equal(t[2].cpu().numpy(), ref["block_table"])
    assert np.array_equal(t[4].cpu().numpy(), ref["free_pages"])
    if in_place:
        assert got["page_count"] is t[3] and got["free_count"] is t[5]
    return ref


CASES = [
    # batch, width, page, new, over, ragged
    (1, 1, 1, 1, 0.0, False), (1, 4, 16, 9, 0.0, False), (16, 64, 16, 9, 0.0, False),
    (16, 64, 16, 9, 0.4, True), (63, 7, 24, 30, 0.1, True), (64, 33, 1, 5, 0.2, True),
    (65, 3, 128, 200, 0.5, True), (1000, 9, 64, 64, 0.1, True), (1024, 5, 16, 3, 0.0, True),
    (1025, 5, 16, 7, 0.3, True), (2500, 4, 32, 11, 0.2, True), (3, 300, 16, 4700, 0.0, False),
    (7, 130, 3, 390, 1.0, True),
]


@pytest.mark.parametrize("batch,width,page,new,over,ragged", CASES)
def test_slots_match_the_oracle(batch, width, page, new, over, ragged):
    args = _case(batch * 31 + width, batch, width, page, new, over, ragged=ragged)
    rows = int(np.where(args[0] < 0, 0, args[1]).sum())
    log(f"slots B={batch} width={width} P={page} rows={rows}")
    for extra in (0, 5):
        ref = _check(args, page, rows + extra, in_place=extra > 0)
        assert ref["status"][0] == 0


@pytest.mark.parametrize("rows", [4095, 4096, 4097, 9000])
def test_both_ways_of_filling_the_rows(rows):
    args = _case(rows, 40, 20, 16, 200, 0.1)
    _check(args, 16, rows)


def test_too_few_pages_or_columns_or_rows():
    args = _case(5, 20, 8, 16, 60, 0.0, spare=7, ragged=False)
    n = 20 * 60
    ref = _check(args, 16, n)
    assert ref["status"][0] > 0 and ref["free_count"][0] == 0
    _check(args, 16, n - 333)
    _check(args, 16, 0)
    # more tokens than the row of the table has columns for
    args = _case(6, 20, 8, 16, 20, 0.0)
    args[1][::3] = 500
    assert _check(args, 16, int(args[1].sum()))["status"][0] > 0


def test_odd_device_values():
    args = _case(7, 12, 6, 8, 10, 0.2)
    args[1][[2, 5]] = [-4, -2147483648]      # negative counts are none
    args[3][4] = 99                          # more pages than columns: all columns
    args[2][4] = np.arange(1000, 1006)
    _check(args, 8, 120)
    full = _case(8, 12, 6, 8, 10, 1.0)       # everything is over: pages past the capacity are dropped
    full[4] = full[4][:int(full[5][0]) + 5].copy()
    _check(full, 8, 16)


def test_no_requests():
    m = bdr()
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    one = torch.full((1,), 3, dtype=torch.int32, device="cuda")
    r = m.spec_slots(z, z, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), z,
                     torch.arange(5, dtype=torch.int32, device="cuda"), one, 16, 9)
    assert r["query_offsets"].tolist() == [0] and r["slots"].tolist() == [-1] * 9
    assert r["positions"].tolist() == [0] * 9 and r["free_count"].tolist() == [3]
    assert r["status"].tolist() == [0]


def test_many_steps_in_place():
    """Tokens come, are accepted in part, requests end and others take their rows."""
    g = np.random.default_rng(11)
    B, width, page, k = 9, 12, 4, 5
    cached = np.zeros(B, dtype=np.int32)
    state = [np.full((B, width), -1, dtype=np.int32), np.zeros(B, dtype=np.int32),
             g.permutation(B * width).astype(np.int32), np.array([B * width], dtype=np.int32)]
    t = [dev(x) for x in state]
    outs = {"page_count": t[1], "free_count": t[3]}
    fresh = np.full(B, k, dtype=np.int32)
    for step in range(40):
        table, count, stack, top = state
        ref = oracle.slots(cached, fresh, table, count, stack, top[0], page, B * k + 3)
        got = bdr().spec_slots(dev(cached), dev(fresh), *t, page, B * k + 3, out=dict(outs))
        for name in ("query_offsets", "kv_len", "positions", "slots", "status"):
            assert np.array_equal(got[name].cpu().numpy(), ref[name]), (step, name)
        state = [ref["block_table"], ref["page_count"], ref["free_pages"], ref["free_count"]]
        for a, b in zip(t, state):
            assert np.array_equal(a.cpu().numpy(), b), step
        held = np.concatenate([state[2][:state[3][0]]] + [state[0][b, :state[1][b]] for b in range(B)])
        assert sorted(held) == list(range(B * width))    # no page lost or held twice
        cached = np.where(cached < 0, 0, cached + g.integers(1, k + 1, B)).astype(np.int32)
        cached = np.where((cached > width * page - k) | (g.random(B) < 0.05), -1, cached).astype(np.int32)
