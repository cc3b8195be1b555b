"""Host-side checks of the paged attention's calls that their documentation allows, by what is refused
behind them: nothing is launched."""
import pytest

from test_abi_paged import A, _attn, _qk, at  # noqa: F401


def _refusal(A, **k):
    assert _qk(A, **k) == A.BDR_EINVAL
    return A.load().bdr_last_error().decode()


# rows, heads, row stride, head stride: contiguous ones (an axis of one entry has any stride)
CONTIGUOUS = [(10, 8, 1024, 128), (1, 8, 1024, 128), (1, 8, 0, 128), (1, 8, 4096, 128), (10, 1, 128, 0),
              (10, 1, 128, 512), (1, 1, 0, 0), (1, 1, 64, 256)]
STRIDED = [(10, 8, 2048, 128), (2, 8, 0, 128), (10, 8, 1024, 256), (1, 8, 0, 256), (10, 1, 256, 128)]


@pytest.mark.parametrize("rows,heads,row,head", CONTIGUOUS)
def test_in_place_where_contiguous(A, rows, heads, row, head):  # noqa: F811
    # the queries over themselves pass; the keys over the values, looked at later, do not
    q = dict(rows=rows, hq=heads, qr=row, qh=head, q_out=at(0), k_out=at(2))
    assert _refusal(A, **q) == "k_out overlaps v"
    k = dict(rows=rows, hkv=heads, kr=row, kh=head, k_out=at(1), q_out=at(2), ps=16 * 1024, ts=1024)
    assert _refusal(A, **k) == "q_out overlaps v"


@pytest.mark.parametrize("rows,heads,row,head", STRIDED)
def test_in_place_where_strided(A, rows, heads, row, head):  # noqa: F811
    assert _refusal(A, rows=rows, hq=heads, qr=row, qh=head, q_out=at(0)) == "q_out overlaps q"
    assert _refusal(A, rows=rows, hkv=heads, kr=row, kh=head, k_out=at(1), ps=16 * 1024, ts=1024) == "k_out overlaps k"


def test_weights_without_queries(A):  # noqa: F811
    """The keys' weight alone passes (the keys over the values do not), the queries' alone does not."""
    none = dict(hq=0, q=None, q_out=None)
    assert _refusal(A, **none, wq=None, k_out=at(2)) == "k_out overlaps v"
    assert _refusal(A, **none, wq=at(5) + 2, k_out=at(2)) == "k_out overlaps v"
    assert "weight" in _refusal(A, **none, wk=None)
    assert "k_weight" in _refusal(A, **none, wq=None, wk=at(6) + 2)
    assert "k_weight" in _refusal(A, **none, wq=None, k_out=at(6))
    assert "weight" in _refusal(A, wq=None) and "weight" in _refusal(A, wk=None)


def test_caches_past_all_memory(A):  # noqa: F811
    """Pages and strides whose product passes 63 bits of bytes: what lies in such a cache is not seen."""
    far = dict(dt=A.BDR_F32, page=1, pages=(1 << 31) - 1, ps=(1 << 30) - 4, ts=(1 << 30) - 4, hs=(1 << 30) - 4, hkv=2)
    assert _attn(A, out=at(1), **far) == A.BDR_EUNSUPPORTED
    assert _qk(A, k_out=at(10), **far) == A.BDR_EUNSUPPORTED
    wide = dict(dt=A.BDR_F32, page=(1 << 31) - 1, pages=1, ps=0, ts=(1 << 30) - 4, hs=128, hkv=2)
    assert _attn(A, out=at(1), **wide) == A.BDR_EUNSUPPORTED
    assert _qk(A, k_out=at(10), **wide) == A.BDR_EUNSUPPORTED
