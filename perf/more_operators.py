"""Timed cases of the drafter's attention over a paged cache: the slots of a step's new tokens
from the requests' lengths, the norms of queries and keys with their rotation and the cache
write, and the attention of the new tokens over the cache.

Where ``own`` is false ``run`` computes them in their plain form with elementary torch
operations in 32 bits (angles in 64); where it is true it makes the calls a user makes of
``block_draft_readout_amd``.

Formulas (request b, page size P, head features D):

    slots     a request with cached[b] < 0 is over: its pages go back on the free stack.  The
              others hold cached[b] tokens and get new[b] more: pages for ceil((cached + new) / P)
              columns of the block table, taken from the top of the stack in the order of the
              requests.  New tokens lie behind one another in the order of the requests; the one
              at position p has slot table[b, p / P] * P + p % P, or -1 where there is no page
    norm      y = x * (mean(x^2) + eps)^-1/2 * w for each head of q and of k
    rotation  by the angle a = position * inv_freq[i] of the pair i of the first 2 * len(inv_freq)
              features: (x1 cos a - x2 sin a, x2 cos a + x1 sin a), the pairs (i, i + half) or,
              interleaved, (2 i, 2 i + 1)
    cache     k and v at their token's slot (a slot outside the cache: nowhere), in 8 bits as
              e4m3(x / scale of the head)
    attention token j of request b's n, at position p = kv_len - n + j, sees the cached positions
              t < kv_len, of those t <= p where causal and t > p - window where there is one:
              out = sum_t softmax_t(scale q . k[t]) v[t], a token that sees nothing gets 0
"""
import math

import torch

own = False

EPS = 1e-6
FAR = 262144   # positions of a long context


def _bdr():
    import block_draft_readout_amd
    return block_draft_readout_amd


def _slots(name, batch, new, ragged, page, max_len, over):
    return dict(name=name, op="slots", batch=batch, new=new, ragged=ragged, page=page,
                max_len=max_len, over=over)


def _qk(name, rows, heads, kv_heads, dim, rot, dtype, cache, interleaved=False, norm=True):
    return dict(name=name, op="qk", rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                dtype=dtype, cache=cache, interleaved=interleaved, norm=norm)


def _attn(name, batch, new, ragged, max_len, heads, kv_heads, dim, page, dtype, cache, causal,
          window=0):
    return dict(name=name, op="attn", batch=batch, new=new, ragged=ragged, max_len=max_len,
                heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, cache=cache,
                causal=causal, window=window)


def listed():
    return [
        # the 16 x 9 positions of one batched block-step: latency
        _slots("slots_16x9_p16", 16, 9, False, 16, 32768, 0.0),
        # a large server's step: prompts and drafts of many requests, a tenth of them over
        _slots("slots_1000_ragged_p64", 1000, 64, True, 64, 8192, 0.1),
        # one token of one sequence
        _qk("qk_1x40_bf16", 1, 40, 8, 128, 128, "bf16", "bf16"),
        # the 16 x 9 positions of a block-step, 8-bit cache
        _qk("qk_144x40_fp8", 144, 40, 8, 128, 128, "bf16", "fp8"),
        # a prompt's chunk
        _qk("qk_8192x40_bf16", 8192, 40, 8, 128, 128, "bf16", "bf16"),
        # an fp32 model: odd rows, interleaved pairs, half of the features rotated, no cache
        _qk("qk_1023x6_f32", 1023, 6, 2, 64, 32, "f32", "none", True),
        # one token over a short context: latency
        _attn("attn_1x1_l1000_bf16", 1, 1, False, 1000, 40, 8, 128, 16, "bf16", "bf16", True),
        # the drafter's block of 8 positions that see one another, 16 requests of unequal length
        _attn("attn_block_16x8_l32768_bf16", 16, 8, False, 32768, 40, 8, 128, 16, "bf16", "bf16",
              False),
        # the 9 verified positions of each request over long 8-bit caches
        _attn("attn_verify_16x9_l65536_fp8", 16, 9, False, 65536, 40, 8, 128, 64, "bf16", "fp8",
              True),
        # a chunk of a long prompt
        _attn("attn_chunk_2048_l16384_bf16", 1, 2048, False, 16384, 32, 8, 128, 16, "bf16", "bf16",
              True),
        # prompts' chunks among decoding requests, wide heads, a sliding window
        _attn("attn_mixed_24_l12000_d256_bf16", 24, 700, True, 12000, 16, 2, 256, 32, "bf16",
              "bf16", True, 4096),
        # an fp32 model: odd lengths and pages
        _attn("attn_5x7_l1001_f32", 5, 7, True, 1001, 6, 2, 64, 24, "f32", "f32", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("slots", "qk", "qk", "attn", "attn", "attn"))
    if op == "slots":
        batch = _log_int(rng, 1, 1000)
        return dict(op=op, batch=batch, new=_log_int(rng, 1, 64), ragged=rng.random() < 0.5,
                    page=rng.choice((1, 16, 16, 24, 32, 64, 128)), max_len=_log_int(rng, 64, 8192),
                    over=rng.choice((0.0, 0.1, 0.5)))
    f32 = rng.random() < 0.2
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8))
    if op == "qk":
        rows = _log_int(rng, 1, 8192)
        if dim == 256:
            kv_heads = min(kv_heads, 4)
        # no query heads: the keys and values of a drafter's context
        heads = 0 if rng.random() < 0.2 else kv_heads * group
        return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice((dim, dim, dim // 2)), dtype="f32" if f32 else "bf16",
                    cache=rng.choice(("none", "f32")) if f32 else rng.choice(("none", "bf16", "fp8")),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8)
    batch = _log_int(rng, 1, 32)
    new = _log_int(rng, 1, 512)
    max_len = max(new, _log_int(rng, 16, 16384))
    if f32:   # fp32 models are small ones
        batch, new, max_len = min(batch, 4), min(new, 64), min(max_len, 2048)
    new = min(new, max_len)
    # no more query positions than the largest case has
    batch = max(1, min(batch, 2048 // new, 262144 // max_len))
    if new > 64:
        group, kv_heads = min(group, 4), min(kv_heads, 4)
    return dict(op=op, batch=batch, new=new, ragged=rng.random() < 0.5, max_len=max_len,
                heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                page=rng.choice((1, 16, 16, 24, 32, 64, 128)), dtype="f32" if f32 else "bf16",
                cache="f32" if f32 else rng.choice(("bf16", "bf16", "fp8")),
                causal=rng.random() < 0.7, window=rng.choice((0, 0, 0, 128, 1000)))


# ------------------------------------------------------------------------- a step's requests
def _spread(i):
    return (0.5 + i * 0.6180339887498949) % 1.0   # in [0, 1), spread evenly whatever the count


def _lengths(case):
    """(tokens in the cache with the new ones, new tokens) of each request: the first the longest,
    the others down to an eighth of it; ragged: from one new token up."""
    out = []
    for b in range(case["batch"]):
        total = max(1, round(case["max_len"] * (0.125 ** _spread(b) if b else 1)))
        new = case["new"] if not case["ragged"] or b == 0 else max(1, round(case["new"] ** _spread(3 * b + 1)))
        out.append((total, min(new, total)))
    return out


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_slots(case, g):
    page = case["page"]
    width = -(-(case["max_len"] + case["new"]) // page)
    lens = _lengths(case)
    over = [_spread(7 * b + 2) < case["over"] for b in range(len(lens))]
    cached = [total - new for total, new in lens]
    # a page ahead is held where drafts were rejected
    held = [min(width, -(-c // page) + (b % 5 == 1)) for b, c in enumerate(cached)]
    total = width * len(lens)
    order = torch.randperm(total, generator=g, device="cuda").int()
    used = sum(held)
    cols = torch.arange(width, device="cuda")
    count = _ints(held)
    first = count.cumsum(0) - count
    index = (first[:, None] + cols).clamp(max=total - 1)
    table = torch.where(cols < count[:, None], order[index.long()], 0).int()
    free = torch.zeros(total, dtype=torch.int32, device="cuda")
    free[:total - used] = order[used:]
    rows = sum(new for _, new in lens)
    return dict(case=case, cached=torch.where(torch.tensor(over, device="cuda"), -1, _ints(cached)).int(),
                new=_ints([new for _, new in lens]), table=table, count=count, free=free,
                top=_ints([total - used]), rows=rows + 7)


def _prepare_qk(case, g):
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n, hq, hkv, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    # one projection's output: queries, keys and values side by side, a few large features
    x = normal(n, hq + 2 * hkv, d)
    x[:, :, ::max(1, d // 4)] *= 4
    x = x.to(dt)
    s = dict(case=case, q=x[:, :hq] if hq else None, k=x[:, hq:hq + hkv], v=x[:, hq + hkv:],
             wq=None, wk=None, k_cache=None, v_cache=None, slots=None, k_scale=None, v_scale=None)
    if case["norm"]:
        s["wq"], s["wk"] = ((1 + normal(d, std=0.1)).to(dt) for _ in range(2))
    half = case["rot"] // 2
    s["inv_freq"] = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
    s["positions"] = torch.randint(0, FAR, (n,), generator=g, device="cuda").int()
    if case["cache"] != "none":
        page = 16
        pages = -(-2 * n // page) + 1
        fp8 = case["cache"] == "fp8"
        for name in ("k", "v"):
            c = normal(pages, page, hkv, d).to(dt)
            s[name + "_cache"] = c.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else c
            if fp8:   # without calibration the codes are the values
                s[name + "_scale"] = torch.ones(hkv, device="cuda")
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].int()
        # the rows of a padded batch have no slot
        s["slots"] = torch.where(torch.arange(n, device="cuda") % 50 == 49, -1, slots).int()
    return s


def _prepare_attn(case, g):
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hq, hkv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case)
    n = sum(new for _, new in lens)
    need = [-(-total // page) for total, _ in lens]
    pages, width = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device="cuda")
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    cols = torch.arange(width, device="cuda")
    held = torch.tensor(need, device="cuda")
    table = torch.where(cols < held[:, None], order[(first[:, None] + cols).clamp(max=pages - 1)], -1)
    s = dict(case=case, table=table.int(), kv_len=_ints([total for total, _ in lens]),
             k_scale=None, v_scale=None)
    offsets = [0]
    for _, new in lens:
        offsets.append(offsets[-1] + new)
    s["offsets"] = _ints(offsets)
    # normalised queries and keys: the keys share a direction, some queries find few of them
    q = torch.randn(n, hq, d, generator=g, device="cuda") * (0.5 + 2 * torch.rand(n, hq, 1, generator=g, device="cuda"))
    s["q"] = q.to(dt)
    for name in ("k", "v"):
        c = torch.empty(pages, page, hkv, d, dtype=dt, device="cuda").normal_(generator=g)
        c += torch.randn(hkv, d, generator=g, device="cuda").to(dt) * 0.5
        if case["cache"] == "fp8":
            scale = 0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
            c = (c / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = scale
        s[name + "_cache"] = c
    return s


def prepare(case, seed):
    return dict(slots=_prepare_slots, qk=_prepare_qk, attn=_prepare_attn)[case["op"]](case, _gen(seed))


# ------------------------------------------------------------------------- the framework's calls
def _run_own(s):
    bdr, c = _bdr(), s["case"]
    if c["op"] == "slots":
        r = bdr.spec_slots(s["cached"], s["new"], s["table"], s["count"], s["free"], s["top"],
                           c["page"], s["rows"])
        return dict(r, table=s["table"], free=s["free"])
    if c["op"] == "qk":
        r = bdr.dspark_qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"],
                                    q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                    interleaved=c["interleaved"], slots=s["slots"],
                                    k_cache=s["k_cache"], v_cache=s["v_cache"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        if c["cache"] == "none":
            return dict(q=r[0], k=r[1])
        return dict(q=r[0], **_caches(s))
    return bdr.dflash_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["offsets"],
                                      s["kv_len"], causal=c["causal"], window=c["window"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])


def _caches(s):
    if s["case"]["cache"] != "fp8":
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    return dict(k_cache=s["k_cache"].view(torch.float8_e4m3fn),
                v_cache=s["v_cache"].view(torch.float8_e4m3fn))


# ------------------------------------------------------------------------- plain forms
def _plain_slots(s):
    page, rows = s["case"]["page"], s["rows"]
    table, free = s["table"], s["free"]
    batch, width = table.shape
    cols = torch.arange(width, device=table.device)
    over = s["cached"] < 0
    held = s["count"].clamp(0, width)
    back = over[:, None] & (cols < held[:, None])
    # the last page of the last request that is over goes back first
    rank = back.flip(0, 1).reshape(-1).cumsum(0).reshape(batch, width).flip(0, 1) - 1
    to = torch.where(back, s["top"] + rank, free.numel()).clamp(max=free.numel())
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, to.reshape(-1).long(), table.reshape(-1))
    top = s["top"] + back.sum()
    have = torch.where(over, 0, held)
    new = torch.where(over, 0, s["new"].clamp(min=0))
    start = s["cached"].clamp(min=0)
    total = start + new
    grow = (((total + page - 1) // page).clamp(max=width) - have).clamp(min=0)
    first = grow.cumsum(0) - grow
    granted = torch.minimum((top - first).clamp(min=0), grow)
    count = have + granted
    take = (cols >= have[:, None]) & (cols < count[:, None])
    at = (top - 1 - first)[:, None] - (cols - have[:, None])
    table.copy_(torch.where(take, stack[at.clamp(0, free.numel()).long()], table))
    free.copy_(stack[:-1])
    ends = new.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    i = torch.arange(rows, device=table.device)
    b = torch.searchsorted(ends, i, right=True).clamp(max=batch - 1)
    live = i < ends[-1]
    pos = torch.where(live, start[b] + i - offsets[b], 0)
    col = pos // page
    fine = live & (col < count[b])
    slot = table[b, col.clamp(max=width - 1).long()] * page + pos % page
    lost = ends[-1] - fine.sum()
    return dict(query_offsets=offsets.int(), kv_len=torch.where(over, 0, total).int(),
                positions=pos.int(), slots=torch.where(fine, slot, -1).int(),
                page_count=count.int(), free_count=(top - granted.sum()).int().reshape(1),
                status=lost.int().reshape(1), table=table, free=free)


def _plain_head(x, w, cos, sin, interleaved):
    x = x.float()
    if w is not None:
        x = x * ((x * x).mean(dim=-1, keepdim=True) + EPS).rsqrt() * w.float()
    half = cos.shape[-1]
    if interleaved:
        x1, x2 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        x1, x2 = x[..., :half], x[..., half:2 * half]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1)


def _plain_qk(s):
    c = s["case"]
    dt = s["k"].dtype
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = None if s["q"] is None else _plain_head(s["q"], s["wq"], cos, sin, c["interleaved"]).to(dt)
    k = _plain_head(s["k"], s["wk"], cos, sin, c["interleaved"])
    if c["cache"] == "none":
        return dict(q=q, k=k.to(dt))
    slots = s["slots"].long()
    flat = s["k_cache"].shape[0] * s["k_cache"].shape[1]
    fine = (slots >= 0) & (slots < flat)
    for name, x in (("k", k), ("v", s["v"].float())):
        if c["cache"] == "fp8":
            x = (x / s[name + "_scale"][:, None]).clamp(-448, 448)
            x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        cache = s[name + "_cache"]
        cache.view(flat, *cache.shape[2:])[slots[fine]] = x[fine].to(cache.dtype)
    return dict(q=q, **_caches(s))


def _values(cache, scale):
    if scale is None:
        return cache.float()
    return cache.view(torch.float8_e4m3fn).float() * scale[:, None]


def _plain_attn(s):
    c = s["case"]
    q, table, offsets, kv_len = s["q"], s["table"].long(), s["offsets"].long(), s["kv_len"].long()
    n, hq, d = q.shape
    hkv, page = c["kv_heads"], c["page"]
    batch, longest = c["batch"], table.shape[1] * page
    longest_new = c["new"]
    dev = q.device
    t = torch.arange(longest, device=dev)
    pages = table[:, t // page].clamp(min=0)
    inside = t < kv_len[:, None]
    # the requests' keys and values side by side, zeros behind their ends
    k = torch.where(inside[:, :, None, None], _values(s["k_cache"][pages, t % page], s["k_scale"]), 0.0)
    v = torch.where(inside[:, :, None, None], _values(s["v_cache"][pages, t % page], s["v_scale"]), 0.0)
    j = torch.arange(longest_new, device=dev)
    new = offsets[1:] - offsets[:-1]
    row = (offsets[:-1, None] + j).clamp(max=n - 1)
    qs = q.float()[row].reshape(batch, longest_new, hkv, hq // hkv, d)
    qs = qs.permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, d)
    z = qs @ k.permute(0, 2, 3, 1)
    z *= 1 / math.sqrt(d)
    p = (kv_len - new)[:, None] + j
    sees = inside[:, None, :].expand(batch, longest_new, longest)
    if c["causal"]:
        sees = sees & (t <= p[:, :, None])
    if c["window"]:
        sees = sees & (t > p[:, :, None] - c["window"])
    sees = sees[:, None, :, None, :]
    z = z.view(batch, hkv, longest_new, hq // hkv, longest)
    z = torch.where(sees, z, -math.inf)
    top = z.max(dim=-1, keepdim=True).values
    z -= torch.where(top == -math.inf, 0.0, top)
    z.exp_()
    total = z.sum(dim=-1, keepdim=True)
    z = z.reshape(batch, hkv, -1, longest) @ v.permute(0, 2, 1, 3)
    z = z.view(batch, hkv, longest_new, hq // hkv, d) / torch.where(total > 0, total, 1.0)
    z = z.permute(0, 2, 1, 3, 4).reshape(batch, longest_new, hq, d)
    i = torch.arange(n, device=dev)
    b = torch.searchsorted(offsets[1:], i, right=True)
    return z[b, i - offsets[b]].to(q.dtype)


def run(state):
    if own:
        return _run_own(state)
    return dict(slots=_plain_slots, qk=_plain_qk, attn=_plain_attn)[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "slots":
        lens = _lengths(c)
        rows = sum(new for _, new in lens)
        # four numbers of a request in, four out; a token's position and slot; the pages of new tokens
        return dict(bytes=32 * c["batch"] + 8 * rows + 8 * (rows // c["page"] + 1), flops=8.0 * rows)
    e = 2 if c["dtype"] == "bf16" else 4
    d, hkv, hq = c["dim"], c["kv_heads"], c["heads"]
    if c["op"] == "qk":
        out = dict(none=e, bf16=2, f32=4, fp8=1)[c["cache"]]
        vectors = (hq + hkv) * e + hkv * out + hq * e
        if c["cache"] != "none":
            vectors += hkv * (e + out)
        return dict(bytes=c["rows"] * (vectors * d + 8), flops=c["rows"] * (hq + hkv) * d * 9.0)
    lens = _lengths(c)
    eb = dict(bf16=2, f32=4, fp8=1)[c["cache"]]
    seen = pairs = rows = 0
    for total, new in lens:
        lo = max(0, total - new - c["window"] + 1) if c["window"] else 0
        seen += total - lo
        rows += new
        if c["window"]:
            for j in range(new):
                p = total - new + j
                pairs += (p + 1 if c["causal"] else total) - max(0, p - c["window"] + 1)
        elif c["causal"]:
            pairs += new * total - new * (new - 1) // 2
        else:
            pairs += new * total
    return dict(bytes=2 * seen * hkv * d * eb + 2 * rows * hq * d * e, flops=4.0 * pairs * hq * d)


# ------------------------------------------------------------------------- in 64 bits
def _exact_qk(s):
    c = s["case"]
    d64 = torch.float64
    angle = torch.outer(s["positions"].to(d64), s["inv_freq"].to(d64))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    half = angle.shape[1]

    def head(x, w):
        x = x.to(d64)
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.to(d64)
        r = x[..., :2 * half]
        pairs = r.unflatten(-1, (half, 2)) if c["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        r = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([r, x[..., 2 * half:]], dim=-1)

    q = None if s["q"] is None else head(s["q"], s["wq"])
    k = head(s["k"], s["wk"])
    if c["cache"] == "none":
        return dict(q=q, k=k)
    out = dict(q=q)
    slots = s["slots"].tolist()
    rows = [i for i, t in enumerate(slots) if t >= 0]
    at = [slots[i] for i in rows]
    for name, x in (("k", k), ("v", s["v"].to(d64))):
        cache = s[name + "_cache"]
        if c["cache"] == "fp8":
            cache = cache.view(torch.float8_e4m3fn).float()
            x = x.clamp(-448, 448)
        full = cache.to(d64).flatten(0, 1)
        full[at] = x[rows]
        out[name + "_cache"] = full.view(cache.shape)
    return out


def _exact_attn(s):
    c = s["case"]
    d64 = torch.float64
    q = s["q"].to(d64)
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros_like(q)
    offsets, lens = s["offsets"].tolist(), s["kv_len"].tolist()
    for b, total in enumerate(lens):
        lo, hi = offsets[b], offsets[b + 1]
        t = torch.arange(total, device=q.device)
        page = s["table"][b].long()[t // c["page"]]
        k, v = (s[x + "_cache"][page, t % c["page"]] for x in ("k", "v"))
        if c["cache"] == "fp8":
            k, v = k.view(torch.float8_e4m3fn).float(), v.view(torch.float8_e4m3fn).float()
        k, v = k.to(d64), v.to(d64)
        if c["cache"] == "fp8":
            k, v = k * s["k_scale"].to(d64)[:, None], v * s["v_scale"].to(d64)[:, None]
        p = torch.arange(total - (hi - lo), total, device=q.device)[:, None]
        gone = torch.zeros(hi - lo, total, dtype=torch.bool, device=q.device)
        if c["causal"]:
            gone |= t > p
        if c["window"]:
            gone |= t <= p - c["window"]
        empty = gone.all(dim=1, keepdim=True)
        for h in range(c["heads"]):
            logits = (q[lo:hi, h] @ k[:, h // group].T) / math.sqrt(c["dim"])
            weights = torch.softmax(logits.masked_fill(gone, -math.inf), dim=1).masked_fill(empty, 0.0)
            out[lo:hi, h] = weights @ v[:, h // group]
    return out


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions (slots are whole numbers: none)."""
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    return _exact_qk(s) if case["op"] == "qk" else _exact_attn(s)
