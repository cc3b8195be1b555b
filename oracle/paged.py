"""Oracle of the drafter's attention over its paged cache: slots from lengths, norms and
rotation of queries and keys, attention.  Plain loops and float64."""
from __future__ import annotations

import numpy as np


def slots(cached, new_tokens, block_table, page_count, free_pages, free_count, page_size, max_rows):
    """The step's plan as a dict (arrays), with block_table and free_pages as they are after it."""
    table = np.array(block_table, dtype=np.int64)
    stack = np.array(free_pages, dtype=np.int64)
    count = [min(max(int(c), 0), table.shape[1]) for c in page_count]
    top = min(max(int(free_count), 0), len(stack))
    width = table.shape[1]
    for b in reversed(range(len(cached))):
        if cached[b] < 0:
            for c in reversed(range(count[b])):
                if top < len(stack):
                    stack[top] = table[b, c]
                    top += 1
            count[b] = 0
    offsets, kv_len, positions, slot = [0], [], [], []
    for b in range(len(cached)):
        n = 0 if cached[b] < 0 else max(int(new_tokens[b]), 0)
        start = max(int(cached[b]), 0)
        while top > 0 and count[b] < min(-(-(start + n) // page_size), width):
            if cached[b] < 0:
                break
            top -= 1
            table[b, count[b]] = stack[top]
            count[b] += 1
        for p in range(start, start + n):
            positions.append(p)
            c = p // page_size
            slot.append(int(table[b, c]) * page_size + p % page_size if c < count[b] else -1)
        offsets.append(offsets[-1] + n)
        kv_len.append(start + n if cached[b] >= 0 else 0)
    fine = sum(s >= 0 for s in slot[:max_rows])
    status = offsets[-1] - fine
    pad = max(0, max_rows - len(slot))
    positions = (positions + [0] * pad)[:max_rows]
    slot = (slot + [-1] * pad)[:max_rows]
    i32 = lambda x: np.array(x, dtype=np.int32)
    return dict(query_offsets=i32(offsets), kv_len=i32(kv_len), positions=i32(positions),
                slots=i32(slot), page_count=i32(count), free_count=i32([top]), status=i32([status]),
                block_table=table.astype(np.int32), free_pages=stack.astype(np.int32))


def norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    """x [N, heads, D] float64 -> normalised (weight None: not) and rotated by position."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(inv_freq)
    out = x.copy()
    for n, p in enumerate(positions):
        for i, f in enumerate(inv_freq):
            a = float(p) * float(f)
            i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[n, :, i1] = x[n, :, i1] * np.cos(a) - x[n, :, i2] * np.sin(a)
            out[n, :, i2] = x[n, :, i2] * np.cos(a) + x[n, :, i1] * np.sin(a)
    return out


def attention(q, k, v, first_position, scale, causal, window):
    """Tokens q [n, Hq, D], the first at first_position, over k, v [L, Hkv, D] (float64).

    Returns (out, lse, weighted, largest): weighted = sum_t w_t |v_t| and the largest |scale q . k|
    of a row and head, from which the tests derive their tolerances."""
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out = np.zeros((n, hq, d))
    weighted = np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    largest = np.zeros((n, hq))
    for j in range(n):
        p = first_position + j
        lo = max(0, p - window + 1) if window else 0
        hi = min(length, p + 1) if causal else length
        if hi <= lo:
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            s = scale * (k[lo:hi, g] @ q[j, h])
            m = s.max()
            w = np.exp(s - m)
            lse[j, h] = m + np.log(w.sum())
            w /= w.sum()
            out[j, h] = w @ v[lo:hi, g]
            weighted[j, h] = w @ np.abs(v[lo:hi, g])
            largest[j, h] = scale * np.max(np.abs(k[lo:hi, g]) @ np.abs(q[j, h]))
    return out, lse, weighted, largest
