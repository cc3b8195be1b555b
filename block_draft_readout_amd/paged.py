"""The drafter's attention over its paged context: the slots of a step's new tokens, the
norms of queries and keys with their rotation and the cache write, and the attention itself
(``include/bdr.h``, last section).

A cache is a pair of tensors [pages, page_size, kv_heads, D] (any strides along the first three
axes, the same for both), of the queries' dtype or uint8 E4M3 codes with one fp32 scale per kv
head.  Request b's position t is at ``block_table[b, t // page_size]``, place ``t % page_size``.
"""
from __future__ import annotations

from typing import Dict, Optional

import torch

from . import _abi
from .training import _dtype, _need, _on, _ptr, _space, _stream, _tensor

__all__ = ["spec_slots", "dspark_qk_norm_rope", "dflash_paged_attention"]


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _ints(t, name: str, shape, device) -> torch.Tensor:
    _tensor(t, name)
    return _need(t, name, shape, _I32, device)


# The calls serve single tokens, where the host's time is the call's: what is right is seen by one
# expression, and only what is not goes through the checks that say why.
def _is(t, dtype, shape, device) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous())


def _call(name: str, fn, device, *args) -> None:
    if torch._C._cuda_getDevice() == device.index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with _on(device):
            rc = fn(*args, _stream(device))
    if rc:
        _abi.check(name, rc)


def spec_slots(cached: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor,
               page_count: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
               page_size: int, max_rows: int,
               out: Optional[Dict[str, torch.Tensor]] = None) -> Dict[str, torch.Tensor]:
    """Pages and slots of a step's new tokens (all int32 on one device).

    Request b holds cached[b] tokens in page_count[b] pages, the first columns of block_table
    [B, max_pages], and gets new_tokens[b] more; cached[b] < 0: the request is over and gives its
    pages back.  Pages come from and go to the top of the stack free_pages, whose first
    free_count[0] entries are free.  block_table and free_pages are changed in place.

    Returns query_offsets [B+1], kv_len [B], positions and slots [max_rows] (position 0 and slot -1
    behind the last token), page_count [B] and free_count [1] as they are now, and status [1]: the
    number of new tokens without a slot, 0 when the step can run.  Pass tensors in ``out`` to
    have them filled; page_count and free_count may be the inputs."""
    L = _abi.load()
    _tensor(cached, "cached")
    if not cached.is_cuda or cached.dim() != 1:
        raise ValueError("cached must be a device tensor [B]")
    _tensor(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    _tensor(free_pages, "free_pages")
    dev, B, width, capacity = cached.device, cached.shape[0], block_table.shape[1], free_pages.numel()
    for t, name, shape in ((cached, "cached", (B,)), (new_tokens, "new_tokens", (B,)),
                           (block_table, "block_table", (B, width)), (page_count, "page_count", (B,)),
                           (free_pages, "free_pages", (capacity,)), (free_count, "free_count", (1,))):
        if not _is(t, _I32, shape, dev):
            _ints(t, name, shape, dev)
    if max_rows < 0:
        raise ValueError("max_rows must be >= 0")
    if not -0x80000000 <= page_size <= 0x7FFFFFFF:   # (ctypes would cut it to 32 bits)
        raise ValueError("page_size must be < 2^31")
    if out is None:
        # one allocation for all of them
        parts = torch.empty(3 * B + 2 * max_rows + 3, dtype=_I32, device=dev).split_with_sizes(
            (B + 1, B, max_rows, max_rows, B, 1, 1))
        res = dict(zip(("query_offsets", "kv_len", "positions", "slots", "page_count", "free_count", "status"),
                       parts))
    else:
        res = dict(out)
        shapes = {"query_offsets": (B + 1,), "kv_len": (B,), "positions": (max_rows,),
                  "slots": (max_rows,), "page_count": (B,), "free_count": (1,), "status": (1,)}
        for name in res:
            if name not in shapes:
                raise ValueError(f"unknown output {name!r}: one of {', '.join(shapes)}")
        for name, shape in shapes.items():
            if name not in res:
                res[name] = torch.empty(shape, dtype=_I32, device=dev)
            elif not _is(res[name], _I32, shape, dev):
                _ints(res[name], f"out[{name!r}]", shape, dev)
    _call("spec_slots", L.spec_slots, dev, cached.data_ptr(), new_tokens.data_ptr(), B, width, page_size,
          block_table.data_ptr(), page_count.data_ptr(), free_pages.data_ptr(), capacity,
          free_count.data_ptr(), max_rows, res["query_offsets"].data_ptr(), res["kv_len"].data_ptr(),
          res["positions"].data_ptr(), res["slots"].data_ptr(), res["page_count"].data_ptr(),
          res["free_count"].data_ptr(), res["status"].data_ptr())
    return res


def _heads(t, name: str, rows, dim, dtype, device):
    """[rows, heads, D] with unit stride along D: (heads, row stride, head stride)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.dim() == 3):
        _tensor(t, name)
        if t.device != device or t.dim() != 3:
            raise ValueError(f"{name} must be [{rows}, heads, {dim}] on {device}")
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    n, heads, d = t.shape
    row, head, one = t.stride()
    if n != rows or d != dim or one != 1:
        raise ValueError(f"{name} must be [{rows}, heads, {dim}] with unit stride along D")
    # (the stride of an axis of one entry says nothing)
    return heads, (row if n > 1 else 0), (head if heads > 1 else d)


def _cache(k_cache, v_cache, k_scale, v_scale, heads: int, dim: int, dtype, device):
    """Checked cache arguments: pages, page_size, strides."""
    want = dtype if k_scale is None else _U8
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not (isinstance(t, torch.Tensor) and t.dtype is want and t.device == device and t.dim() == 4):
            _tensor(t, name)
            if t.device != device or t.dim() != 4:
                raise ValueError(f"{name} must be [pages, page_size, {heads}, {dim}] on {device}")
            raise TypeError(f"{name} must be {want}, got {t.dtype}")
    shape, stride = k_cache.shape, k_cache.stride()
    pages, page, h, d = shape
    if h != heads or d != dim or stride[3] != 1:
        raise ValueError(f"k_cache must be [pages, page_size, {heads}, {dim}] with unit stride along D")
    if page > 0x7FFFFFFF:
        raise ValueError("page_size must be < 2^31")
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape")
    if 1 in shape:   # the stride of an axis of one entry says nothing
        stride = tuple(0 if n == 1 else s for n, s in zip(shape, stride))
        same = stride == tuple(0 if n == 1 else s for n, s in zip(shape, v_cache.stride()))
    else:
        same = stride == v_cache.stride()
    if not same:
        raise ValueError("k_cache and v_cache must have the same strides")
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale must both be given or both be None")
    if k_scale is not None:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if not _is(t, _F32, (heads,), device):
                _tensor(t, name)
                _need(t, name, (heads,), _F32, device)
    return pages, page, stride[0], stride[1], stride[2]


def dspark_qk_norm_rope(q: Optional[torch.Tensor], k: torch.Tensor, v: Optional[torch.Tensor],
                        positions: torch.Tensor, inv_freq: torch.Tensor, *,
                        q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        interleaved: bool = False, slots: Optional[torch.Tensor] = None,
                        k_cache: Optional[torch.Tensor] = None,
                        v_cache: Optional[torch.Tensor] = None,
                        k_scale: Optional[torch.Tensor] = None,
                        v_scale: Optional[torch.Tensor] = None,
                        q_out: Optional[torch.Tensor] = None,
                        k_out: Optional[torch.Tensor] = None):
    """Root-mean-square norm of each head of q [N, Hq, D] and k [N, Hkv, D] (weights [D], k_weight
    alone without queries; None: no norm), then the rotation of the first 2 * len(inv_freq)
    features by positions[n] * inv_freq (fp32), in pairs (i, i + half) or interleaved (2 i, 2 i + 1).
    q, k and v may be views of one projection's output (unit stride along D).

    With a cache, k and v [N, Hkv, D] are written at slots [N] of k_cache and v_cache (a slot
    outside the cache is skipped; uint8 caches take E4M3 codes of x / scale[head]).  Returns
    (q, k): q is None without queries (q=None: a drafter's context), k None with a cache unless
    k_out is given."""
    L = _abi.load()
    _tensor(k, "k")
    if not k.is_cuda or k.dim() != 3:
        raise ValueError("k must be a device tensor [N, Hkv, D]")
    dev, dtype = k.device, k.dtype
    dt = _dtype(k, "k")
    n, _, d = k.shape
    hkv, kr, kh = _heads(k, "k", n, d, dtype, dev)
    hq = qr = qh = vr = vh = 0
    qp = qo = vp = ko = sp = kc = vc = None
    if q is not None:
        hq, qr, qh = _heads(q, "q", n, d, dtype, dev)
        qp = q.data_ptr()
        if q_out is None:
            q_out = torch.empty((n, hq, d), dtype=dtype, device=dev)
        elif not _is(q_out, dtype, (n, hq, d), dev):
            _tensor(q_out, "q_out")
            _need(q_out, "q_out", (n, hq, d), dtype, dev)
        qo = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    if not _is(positions, _I32, (n,), dev):
        _ints(positions, "positions", (n,), dev)
    _tensor(inv_freq, "inv_freq")
    half = inv_freq.numel()
    if not _is(inv_freq, _F32, (half,), dev):
        _need(inv_freq, "inv_freq", (half,), _F32, dev)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and not _is(w, dtype, (d,), dev):
            _tensor(w, name)
            _need(w, name, (d,), dtype, dev)
    cache = (1, 1, 0, 0, 0)
    if k_cache is not None or v_cache is not None:
        if v is None or slots is None:
            raise ValueError("v and slots are needed with a cache")
        hv, vr, vh = _heads(v, "v", n, d, dtype, dev)
        if hv != hkv:
            raise ValueError(f"v must be [{n}, {hkv}, {d}]")
        cache = _cache(k_cache, v_cache, k_scale, v_scale, hkv, d, dtype, dev)
        if not _is(slots, _I32, (n,), dev):
            _ints(slots, "slots", (n,), dev)
        vp, sp, kc, vc = v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales are given without a cache")
    elif k_out is None:
        k_out = torch.empty((n, hkv, d), dtype=dtype, device=dev)
    if k_out is not None:
        if not _is(k_out, dtype, (n, hkv, d), dev):
            _tensor(k_out, "k_out")
            _need(k_out, "k_out", (n, hkv, d), dtype, dev)
        ko = k_out.data_ptr()
    _call("dspark_qk_norm_rope", L.dspark_qk_norm_rope, dev, qp, qr, qh, k.data_ptr(), kr, kh, vp, vr, vh,
          n, hq, hkv, d, dt, positions.data_ptr(), inv_freq.data_ptr(), 2 * half, interleaved,
          _ptr(q_weight), _ptr(k_weight), eps, qo, ko, sp, kc, vc, *cache, _ptr(k_scale), _ptr(v_scale))
    return q_out, k_out


def dflash_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_table: torch.Tensor, query_offsets: torch.Tensor,
                           kv_len: torch.Tensor, *, scale: Optional[float] = None,
                           causal: bool = True, window: int = 0,
                           k_scale: Optional[torch.Tensor] = None,
                           v_scale: Optional[torch.Tensor] = None, lse: bool = False,
                           out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None):
    """Attention of the new tokens q [N, Hq, D] over the cached positions of their requests.

    Rows query_offsets[b] .. query_offsets[b + 1] (int32 [B+1]) are the last of request b's
    kv_len[b] positions; they see its positions up to their own (causal=False: all of them), of
    those the last ``window`` (0: all).  scale defaults to D ** -0.5.  A row that sees nothing is
    0; rows of no request (behind the last one, in a padded batch) are not written.

    lse=True returns (out, lse): fp32 [N, Hq] logarithms of the sums of exponentials."""
    L = _abi.load()
    _tensor(q, "q")
    if not q.is_cuda or q.dim() != 3:
        raise ValueError("q must be a device tensor [N, Hq, D]")
    dev, dtype = q.device, q.dtype
    dt = _dtype(q, "q")
    n, _, d = q.shape
    hq, qr, qh = _heads(q, "q", n, d, dtype, dev)
    _tensor(k_cache, "k_cache")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, Hkv, D]")
    hkv = k_cache.shape[2]
    cache = _cache(k_cache, v_cache, k_scale, v_scale, hkv, d, dtype, dev)
    _tensor(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    b, width = block_table.shape
    for t, name, shape in ((block_table, "block_table", (b, width)),
                           (query_offsets, "query_offsets", (b + 1,)), (kv_len, "kv_len", (b,))):
        if not _is(t, _I32, shape, dev):
            _ints(t, name, shape, dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=dtype, device=dev)
    elif not _is(out, dtype, (n, hq, d), dev):
        _tensor(out, "out")
        _need(out, "out", (n, hq, d), dtype, dev)
    if window < 0:
        raise ValueError("window must be >= 0")
    sums = torch.empty((n, hq), dtype=_F32, device=dev) if lse else None
    need = L.dflash_paged_attention_workspace_bytes(n, hq, hkv, d, dt, b, width, cache[1])
    wp, wn, _keep = _space(need, dev, workspace)
    _call("dflash_paged_attention", L.dflash_paged_attention, dev, q.data_ptr(), qr, qh, n, hq, hkv, d, dt,
          k_cache.data_ptr(), v_cache.data_ptr(), *cache, _ptr(k_scale), _ptr(v_scale),
          block_table.data_ptr(), b, width, query_offsets.data_ptr(), kv_len.data_ptr(),
          d ** -0.5 if scale is None else scale, causal, min(window, 0x7FFFFFFF), out.data_ptr(), _ptr(sums), wp, wn)
    return (out, sums) if lse else out
