"""Pins of oracle/paged.py: facts other than itself."""
import numpy as np

from oracle import paged


def test_slots_by_hand():
    # pages of 4; request 0 holds 5 tokens in 2 pages, 1 is over with 2 pages, 2 is new
    table = np.array([[7, 3, -1], [5, 6, -1], [-1, -1, -1]])
    r = paged.slots([5, -1, 0], [4, 9, 5], table, [2, 2, 0], [1, 2, 0, 0], 2, 4, 12)
    # request 1's pages come back last page first: stack 1 2 6 5; request 0 needs a third page (5),
    # request 2 two (6, 2)
    assert r["block_table"].tolist() == [[7, 3, 5], [5, 6, -1], [6, 2, -1]]
    assert r["query_offsets"].tolist() == [0, 4, 4, 9] and r["kv_len"].tolist() == [9, 0, 5]
    assert r["positions"].tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, 0, 0, 0]
    assert r["slots"].tolist() == [13, 14, 15, 20, 24, 25, 26, 27, 8, -1, -1, -1]
    assert r["page_count"].tolist() == [3, 0, 2] and r["free_count"].tolist() == [1]
    assert r["status"].tolist() == [0]


def test_slots_run_out():
    r = paged.slots([0, 0], [5, 3], np.full((2, 2), -1), [0, 0], [9], 1, 4, 6)
    # one page for the first request's first four tokens; rows past six have no place
    assert r["slots"].tolist() == [36, 37, 38, 39, -1, -1] and r["status"].tolist() == [4]


def test_rotation_keeps_lengths_and_relative_angles():
    g = np.random.default_rng(1)
    f = np.array([1.0, 0.25, 1e-3, 3e-6])
    for inter in (False, True):
        x, y = g.standard_normal((2, 1, 1, 8))
        at = lambda v, p: paged.norm_rope(v, [p], f, None, 0.0, inter)[0, 0]
        assert np.isclose(np.linalg.norm(at(x, 77)), np.linalg.norm(x))
        # the product of two rotated vectors depends on the difference of their positions
        assert np.isclose(at(x, 500) @ at(y, 480), at(x, 20) @ at(y, 0))
        assert np.allclose(at(x, 0), x[0, 0])
    # a quarter turn of the pair (0, 4) and of (0, 1)
    e = np.zeros((1, 1, 8))
    e[0, 0, 0] = 1
    quarter = [np.pi / 2, 0, 0, 0]
    assert np.allclose(paged.norm_rope(e, [1], quarter, None, 0.0, False)[0, 0], np.eye(8)[4])
    assert np.allclose(paged.norm_rope(e, [1], quarter, None, 0.0, True)[0, 0], np.eye(8)[1])


def test_norm_of_constant_heads():
    x = np.full((1, 2, 16), -3.0)
    y = paged.norm_rope(x, [0], [0.0] * 8, np.arange(16.0), 0.0, False)
    assert np.allclose(y[0, 1], -np.arange(16.0))


def test_attention_closed_forms():
    g = np.random.default_rng(2)
    k = np.zeros((5, 1, 4))
    v = g.standard_normal((5, 1, 4))
    q = g.standard_normal((2, 3, 4))
    out, lse, *_ = paged.attention(q, k, v, 3, 0.5, True, 0)      # equal weights: means
    assert np.allclose(out[0], v[:4, 0].mean(0)) and np.allclose(out[1], v[:, 0].mean(0))
    assert np.allclose(lse[1], np.log(5))
    out, *_ = paged.attention(q, k, v, 3, 0.5, True, 2)           # the last two positions
    assert np.allclose(out[0], v[2:4, 0].mean(0)) and np.allclose(out[1], v[3:, 0].mean(0))
    out, *_ = paged.attention(q, k, v, 3, 0.5, False, 0)
    assert np.allclose(out, v[:, 0].mean(0))
    out, lse, *_ = paged.attention(q, k, v, -1, 0.5, True, 0)     # before the first position: nothing
    assert np.all(out[0] == 0) and np.all(lse[0] == -np.inf) and np.allclose(out[1], v[0, 0])
    # one key far above the others takes all; scores shifted together change nothing
    k[:, 0, 0] = [0, 0, 900, 0, 0]
    q[..., 0] = 1
    out, *_ = paged.attention(q, k, v, 3, 1.0, False, 0)
    assert np.allclose(out, v[2, 0])
