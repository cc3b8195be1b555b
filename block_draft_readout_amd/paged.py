"""The drafter's attention over its paged context: the slots of a step's new tokens, the
norms of queries and keys with their rotation and the cache write, and the attention itself
(``include/bdr.h``, last section).

A cache is a pair of tensors [pages, page_size, kv_heads, D] (any strides along the first three
axes, the same for both), of the queries' dtype or uint8 E4M3 codes with one fp32 scale per kv
head.  Request b's position t is at ``block_table[b, t // page_size]``, place ``t % page_size``.
"""
from __future__ import annotations

import math
from typing import Dict, Optional

import torch

from . import _abi
from .training import _dtype, _need, _on, _ptr, _space, _stream, _tensor

__all__ = ["spec_slots", "dspark_qk_norm_rope", "dflash_paged_attention"]


def _ints(t, name: str, shape, device) -> torch.Tensor:
    _tensor(t, name)
    return _need(t, name, shape, torch.int32, device)


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
    dev, B = cached.device, cached.shape[0]
    _ints(cached, "cached", (B,), dev)
    _ints(new_tokens, "new_tokens", (B,), dev)
    _tensor(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    width = block_table.shape[1]
    _ints(block_table, "block_table", (B, width), dev)
    _ints(page_count, "page_count", (B,), dev)
    _tensor(free_pages, "free_pages")
    capacity = free_pages.numel()
    _ints(free_pages, "free_pages", (capacity,), dev)
    _ints(free_count, "free_count", (1,), dev)
    res = dict(out) if out is not None else {}
    shapes = {"query_offsets": (B + 1,), "kv_len": (B,), "positions": (max_rows,),
              "slots": (max_rows,), "page_count": (B,), "free_count": (1,), "status": (1,)}
    for name in res:
        if name not in shapes:
            raise ValueError(f"unknown output {name!r}: one of {', '.join(shapes)}")
    if max_rows < 0:
        raise ValueError("max_rows must be >= 0")
    missing = [n for n in shapes if n not in res]
    for name in res:
        _ints(res[name], f"out[{name!r}]", shapes[name], dev)
    if missing:
        # one allocation for all of them, each at a 16-byte boundary
        sizes = [math.prod(shapes[n]) for n in missing]
        flat = torch.empty(sum((s + 3) & ~3 for s in sizes), dtype=torch.int32, device=dev)
        at = 0
        for name, s in zip(missing, sizes):
            res[name] = flat[at:at + s]
            at += (s + 3) & ~3
    with _on(dev):
        _abi.check("spec_slots", L.spec_slots(
            cached.data_ptr(), new_tokens.data_ptr(), B, width, page_size, block_table.data_ptr(),
            page_count.data_ptr(), free_pages.data_ptr(), capacity, free_count.data_ptr(), max_rows,
            res["query_offsets"].data_ptr(), res["kv_len"].data_ptr(), res["positions"].data_ptr(),
            res["slots"].data_ptr(), res["page_count"].data_ptr(), res["free_count"].data_ptr(),
            res["status"].data_ptr(), _stream(dev)))
    return res


def _heads(t: torch.Tensor, name: str, rows, dtype, device):
    """[rows, heads, D] with unit stride along D: (row stride, head stride)."""
    _tensor(t, name)
    if t.device != device or t.dim() != 3 or t.shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}, heads, D] on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    row, head, one = t.stride()
    if t.shape[2] != 1 and one != 1:
        raise ValueError(f"{name} must have unit stride along D")
    # the stride of an axis of one entry says nothing
    return (row if t.shape[0] > 1 else 0), (head if t.shape[1] > 1 else t.shape[2])


def _cache(k_cache, v_cache, k_scale, v_scale, heads: int, dim: int, dtype, device):
    """Checked cache arguments: (pages, page_size, strides, k_scale, v_scale pointers)."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _tensor(t, name)
        if t.device != device or t.dim() != 4 or t.shape[2:] != (heads, dim):
            raise ValueError(f"{name} must be [pages, page_size, {heads}, {dim}] on {device}")
        want = dtype if k_scale is None else torch.uint8
        if t.dtype != want:
            raise TypeError(f"{name} must be {want}, got {t.dtype}")
        if t.stride(3) != 1:
            raise ValueError(f"{name} must have unit stride along D")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    pages, page = k_cache.shape[:2]
    # (the stride of an axis of one entry says nothing: the tightest place is as good)
    stride = [s for s in k_cache.stride()[:3]]
    for i, n in enumerate(k_cache.shape[:3]):
        if n == 1:
            stride[i] = 0
        elif v_cache.stride(i) != stride[i]:
            raise ValueError("k_cache and v_cache must have the same strides")
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale must both be given or both be None")
    if k_scale is not None:
        _tensor(k_scale, "k_scale")
        _tensor(v_scale, "v_scale")
        _need(k_scale, "k_scale", (heads,), torch.float32, device)
        _need(v_scale, "v_scale", (heads,), torch.float32, device)
    return pages, page, stride


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
    """Root-mean-square norm of each head of q [N, Hq, D] and k [N, Hkv, D] (weights [D]; None: no
    norm), then the rotation of the first 2 * len(inv_freq) features by positions[n] * inv_freq
    (fp32), in pairs (i, i + half) or interleaved (2 i, 2 i + 1).  q, k and v may be views of one
    projection's output (unit stride along D).

    With a cache, k and v [N, Hkv, D] are written at slots [N] of k_cache and v_cache (a slot
    outside the cache is skipped; uint8 caches take E4M3 codes of x / scale[head]).  Returns
    (q, k): q is None without queries (q=None: a drafter's context), k None with a cache unless
    k_out is given."""
    L = _abi.load()
    _tensor(k, "k")
    if not k.is_cuda or k.dim() != 3:
        raise ValueError("k must be a device tensor [N, Hkv, D]")
    dev, dt = k.device, _dtype(k, "k")
    n, hkv, d = k.shape
    kr, kh = _heads(k, "k", n, k.dtype, dev)
    hq = qr = qh = vr = vh = 0
    if q is not None:
        qr, qh = _heads(q, "q", n, k.dtype, dev)
        hq = q.shape[1]
        if q.shape[2] != d:
            raise ValueError(f"q must be [{n}, Hq, {d}]")
        if q_out is None:
            q_out = torch.empty((n, hq, d), dtype=k.dtype, device=dev)
        else:
            _tensor(q_out, "q_out")
            _need(q_out, "q_out", (n, hq, d), k.dtype, dev)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    _ints(positions, "positions", (n,), dev)
    _tensor(inv_freq, "inv_freq")
    half = inv_freq.numel()
    _need(inv_freq, "inv_freq", (half,), torch.float32, dev)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _tensor(w, name)
            _need(w, name, (d,), k.dtype, dev)
    pages = page = 1
    strides = (0, 0, 0)
    if k_cache is not None or v_cache is not None:
        if v is None or slots is None:
            raise ValueError("v and slots are needed with a cache")
        vr, vh = _heads(v, "v", n, k.dtype, dev)
        if v.shape != k.shape:
            raise ValueError(f"v must be [{n}, {hkv}, {d}]")
        pages, page, strides = _cache(k_cache, v_cache, k_scale, v_scale, hkv, d, k.dtype, dev)
        _ints(slots, "slots", (n,), dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales are given without a cache")
    elif k_out is None:
        k_out = torch.empty((n, hkv, d), dtype=k.dtype, device=dev)
    if k_out is not None:
        _tensor(k_out, "k_out")
        _need(k_out, "k_out", (n, hkv, d), k.dtype, dev)
    with _on(dev):
        _abi.check("dspark_qk_norm_rope", L.dspark_qk_norm_rope(
            _ptr(q), qr, qh, k.data_ptr(), kr, kh, _ptr(v), vr, vh, n, hq, hkv, d, dt,
            positions.data_ptr(), inv_freq.data_ptr(), 2 * half, int(interleaved), _ptr(q_weight),
            _ptr(k_weight), eps, _ptr(q_out), _ptr(k_out), _ptr(slots), _ptr(k_cache),
            _ptr(v_cache), pages, page, *strides, _ptr(k_scale), _ptr(v_scale), _stream(dev)))
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
    dev, dt = q.device, _dtype(q, "q")
    n, hq, d = q.shape
    qr, qh = _heads(q, "q", n, q.dtype, dev)
    _tensor(k_cache, "k_cache")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, Hkv, D]")
    hkv = k_cache.shape[2]
    pages, page, strides = _cache(k_cache, v_cache, k_scale, v_scale, hkv, d, q.dtype, dev)
    _tensor(block_table, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    b, width = block_table.shape
    _ints(block_table, "block_table", (b, width), dev)
    _ints(query_offsets, "query_offsets", (b + 1,), dev)
    _ints(kv_len, "kv_len", (b,), dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=q.dtype, device=dev)
    else:
        _tensor(out, "out")
        _need(out, "out", (n, hq, d), q.dtype, dev)
    sums = torch.empty((n, hq), dtype=torch.float32, device=dev) if lse else None
    need = L.dflash_paged_attention_workspace_bytes(n, hq, hkv, d, dt, b, width, page)
    wp, wn, _keep = _space(need, dev, workspace)
    with _on(dev):
        _abi.check("dflash_paged_attention", L.dflash_paged_attention(
            q.data_ptr(), qr, qh, n, hq, hkv, d, dt, k_cache.data_ptr(), v_cache.data_ptr(), pages,
            page, *strides, _ptr(k_scale), _ptr(v_scale), block_table.data_ptr(), b, width,
            query_offsets.data_ptr(), kv_len.data_ptr(), d ** -0.5 if scale is None else scale,
            int(causal), window, out.data_ptr(), _ptr(sums), wp, wn, _stream(dev)))
    return (out, sums) if lse else out
