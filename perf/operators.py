"""The paged-cache operators as they are measured: their cases, inputs, plain forms and exact values.

A serving program keeps the keys and values of its sequences in a pool of pages.  Each
step it rotates the new queries and keys by their positions and appends keys and values
to the pages (``fa_kv_append``), then attends over the pages (``fa_fwd_paged``); a prompt
that continues a cached prefix reads the pages back as packed rows (``fa_kv_gather``) and
runs the variable-length forward on them.  A pool holds 16-bit values, or 4-bit codes
with a 16-bit scale and zero per 32 head dims.

Pool layout: 16-bit [pages, Hkv, page_size, d]; 4-bit uint8 [pages, Hkv, page_size, 5d/8],
whose page_size * 5d/8 bytes per (page, head) are first the codes, page_size rows of d/2
bytes (dim 2i in the low four bits of byte i, dim 2i + 1 in the high four), then
page_size rows of d/32 (scale, zero) pairs in the 16-bit type.  A code c stands for
scale * c + zero.
"""
import random

import torch

own = False

GROUP = 32  # head dims that share a scale and a zero

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------
def _case(name, op, fmt, dtype, heads, page, batch, ctx, new, rot=1.0, interleaved=False, even=False):
    hq, hkv, d = heads
    c = dict(op=op, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, batch=batch, ctx=ctx, new=new,
             rot=int(d * rot) // 16 * 16, interleaved=interleaved, even=even)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a serving batch: one token per sequence, where the launch is the cost
        _case("append step b32", "append", "16", "bf16", (32, 8, 128), 16, 32, 2048, 1),
        # prompts of a prefill batch, packed, appended to fresh pages
        _case("append prompts", "append", "16", "bf16", (32, 8, 128), 64, 8, 4096, 4096),
        # the same for a 4-bit pool, half the head dims rotated as interleaved pairs, and
        # the sequences read back as the chunk's attention needs them
        _case("append + read prompts int4", "append", "int4", "bf16", (32, 4, 128), 32, 8, 4100, 4100, 0.5, True),
        # cached prefixes read back for the next chunk of their prompts
        _case("read prefixes d256", "gather", "16", "fp16", (16, 2, 256), 64, 16, 8192, 1),
        _case("read prefixes int4", "gather", "int4", "bf16", (32, 8, 128), 16, 16, 16384, 1),
        # a single user's next token: latency
        _case("decode b1 1k", "attend", "16", "bf16", (32, 8, 128), 16, 1, 1000, 1),
        # a serving batch of ragged lengths
        _case("decode b64 ragged", "attend", "16", "bf16", (32, 4, 128), 64, 64, 8192, 1),
        # few long documents, wide heads
        _case("decode b4 128k d256", "attend", "16", "fp16", (16, 2, 256), 128, 4, 131072, 1, even=True),
        # a single user's next token over a 4-bit pool, widest heads
        _case("decode int4 b1 d512", "attend", "int4", "bf16", (8, 1, 512), 32, 1, 777, 1),
        # the serving batch over a 4-bit pool
        _case("decode int4 b64 ragged", "attend", "int4", "bf16", (32, 8, 128), 16, 64, 8192, 1),
        # drafted tokens verified in one call
        _case("verify 4 int4 b16", "attend", "int4", "bf16", (32, 8, 128), 32, 16, 16384, 4),
        # few long documents over a 4-bit pool
        _case("decode int4 b4 128k", "attend", "int4", "fp16", (32, 4, 128), 64, 4, 131072, 1, even=True),
    ]


HEADS = [(32, 8, 128), (32, 4, 128), (16, 16, 128), (8, 2, 192), (8, 8, 256), (16, 2, 256), (8, 2, 384), (8, 1, 512)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "gather", "attend", "attend"])
    fmt = rng.choice(["16", "int4"])
    dtype = rng.choice(["bf16", "fp16"])
    heads = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    batch = _log(rng, 1, 64)
    new = _log(rng, 1, 16) if op == "attend" else 1
    # at most the values per pool, and for attention the products, of the largest listed case
    room = (1 << 25 if op == "append" else 1 << 28) // (batch * heads[1] * heads[2])
    room //= -(-new * heads[0] // heads[1] // 48)
    ctx = _log(rng, 1, min(131072, room))
    if op == "append":
        new = _log(rng, 1, min(ctx, max(1, (1 << 24) // (batch * heads[0] * heads[2])), 8192))
    new = min(new, ctx)
    return _case(None, op, fmt, dtype, heads, page, batch, ctx, new, rng.choice([0.25, 0.5, 1.0]),
                 rng.choice([False, True]), rng.choice([False, True]))


def _lens(c):
    """(cached length with this call's tokens, this call's tokens) of each sequence: from the case alone."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    lens, news = [], []
    for b in range(c["batch"]):
        n = c["ctx"] if c["even"] or b == 0 else _log(r, max(1, c["ctx"] // 8), c["ctx"])
        m = min(n, c["new"]) if c["even"] or b == 0 else min(n, r.randint(max(1, c["new"] // 2), c["new"]))
        lens.append(n)
        news.append(m)
    return lens, news


# ---------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------
def _quantise(x, dt):
    """fp64 [..., d] -> codes uint8 [..., d], scale and zero (type dt) [..., d / 32].  The zero is
    the group's least value and the scale a fifteenth of the rest, each rounded to dt; a code is
    the nearest whole number of scales above the zero, ties to even."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    zero = g.amin(-1).float().to(dt)
    scale = ((g.amax(-1) - zero.double()).clamp_min(0) / 15).float().to(dt)
    z, s = zero.double()[..., None], scale.double()[..., None]
    codes = torch.where(s > 0, ((g - z) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), torch.zeros_like(g))
    return codes.to(torch.uint8).reshape(x.shape), scale, zero


def _int4_views(pool, dt):
    """The code bytes [pages, Hkv, page, d / 2] and the (scale, zero) pairs [pages, Hkv, page, d / 32, 2] of a pool."""
    p, h, n, w = pool.shape
    d = w * 8 // 5
    flat = pool.view(p, h, n * w)
    codes = flat[:, :, : n * d // 2].view(p, h, n, d // 2)
    pairs = flat[:, :, n * d // 2:].view(dt).view(p, h, n, d // GROUP, 2)
    return codes, pairs


def _pool(c, pages, gen):
    dt, dev = DTYPES[c["dtype"]], "cuda"
    shape = (pages, c["hkv"], c["page"], c["d"])
    if c["fmt"] == "16":
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)
    pool = torch.empty(pages, c["hkv"], c["page"], 5 * c["d"] // 8, dtype=torch.uint8, device=dev)
    codes, pairs = _int4_views(pool, dt)
    step = max(1, (1 << 26) // (c["hkv"] * c["page"] * c["d"]))
    for p in range(0, pages, step):
        x = torch.randn((min(step, pages - p),) + shape[1:], generator=gen, device=dev, dtype=dt)
        q, s, z = _quantise(x.double(), dt)
        codes[p: p + step] = q[..., 0::2] | (q[..., 1::2] << 4)
        pairs[p: p + step] = torch.stack([s, z], -1)
    return pool


def prepare(case, seed):
    c = case
    dt, dev = DTYPES[c["dtype"]], "cuda"
    lens, news = _lens(c)
    gen = torch.Generator(device=dev).manual_seed(seed)
    width = -(-max(lens) // c["page"])
    pages = sum(-(-n // c["page"]) for n in lens)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(c["batch"], width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // c["page"])
        table[b, :k] = order[at: at + k]
        at += k
    s = dict(case=dict(c), table=table, k_cache=_pool(c, pages, gen), v_cache=_pool(c, pages, gen),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu=torch.tensor([0] + news, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev),
             cu_k=torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev),
             total=sum(news), total_k=sum(lens), max_new=max(news), width=max(lens))
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "append":
        # a layer's fused projection: queries, keys and values side by side in each token's row
        qkv = torch.randn(sum(news), hq + 2 * hkv, d, generator=gen, device=dev).to(dt)
        s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], 1)
        rot = c["rot"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(rot, 1))).float()
    if c["op"] == "attend":
        s["q"] = torch.randn(sum(news), hq, d, generator=gen, device=dev).to(dt)
    return s


# ---------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import exact_attention_blackwell_fa_b200 as fa

    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "append":
        q = fa.fa_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["lens"], s["table"],
                            inv_freq=s["inv_freq"], interleaved=c["interleaved"])
        if c["fmt"] == "16":
            return q, s["k_cache"], s["v_cache"]
        k, v = fa.fa_kv_gather(s["k_cache"], s["v_cache"], s["cu_k"], s["table"], s["total_k"], dt)
        return q, k, v
    if c["op"] == "gather":
        return fa.fa_kv_gather(s["k_cache"], s["v_cache"], s["cu_k"], s["table"], s["total_k"], dt)
    return fa.fa_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["lens"], s["table"], s["max_new"],
                           causal=True)


def _rows(cu, total):
    """The sequence and the place in it of each packed row."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, t - cu[b].long()


def _rotate(x, pos, inv_freq, interleaved, wide):
    """Rows [T, H, d] turned by pos * inv_freq, rounded once to their type unless `wide`.  The angles
    are formed in 64 bits; so is all of it where a code's border decides."""
    ct = torch.float64 if wide else torch.float32
    y = x.to(ct)
    if inv_freq.numel():
        rot = 2 * inv_freq.numel()
        a = pos.double()[:, None] * inv_freq.double()
        cos, sin = a.cos().to(ct)[:, None], a.sin().to(ct)[:, None]
        r = y[..., :rot]
        if interleaved:
            u, w = r[..., 0::2], r[..., 1::2]
            r = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
        else:
            u, w = r[..., : rot // 2], r[..., rot // 2:]
            r = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
        y = torch.cat([r, y[..., rot:]], -1)
    return y if wide else y.to(x.dtype)


def _read(pool, page, slot, dt):
    """Rows [..., Hkv, d] of the pool in fp32, at page and slot [...]."""
    if pool.dtype != torch.uint8:
        return pool[page, :, slot].float()
    codes, pairs = _int4_views(pool, dt)
    b, p = codes[page, :, slot], pairs[page, :, slot].float()
    q = torch.stack([b & 15, b >> 4], -1).float().reshape(*b.shape[:-1], -1, GROUP)
    return (q * p[..., :1] + p[..., 1:]).flatten(-2)


def _run_plain(s):
    c, table = s["case"], s["table"].long()
    dt, page = DTYPES[c["dtype"]], c["page"]
    if c["op"] in ("append", "gather"):
        bk, jk = _rows(s["cu_k"], s["total_k"])
        if c["op"] == "append":
            b, i = _rows(s["cu"], s["total"])
            pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[b] + i
            q = _rotate(s["q"], pos, s["inv_freq"], c["interleaved"], False)
            k = _rotate(s["k"], pos, s["inv_freq"], c["interleaved"], c["fmt"] == "int4")
            pg, slot = table[b, pos // page], pos % page
            if c["fmt"] == "16":
                s["k_cache"][pg, :, slot] = k
                s["v_cache"][pg, :, slot] = s["v"]
                return q, s["k_cache"], s["v_cache"]
            _write(s["k_cache"], pg, slot, k, dt)
            _write(s["v_cache"], pg, slot, s["v"].double(), dt)
            at = table[bk, jk // page], jk % page
            return q, _read(s["k_cache"], *at, dt).to(dt), _read(s["v_cache"], *at, dt).to(dt)
        at = table[bk, jk // page], jk % page
        return _read(s["k_cache"], *at, dt).to(dt), _read(s["v_cache"], *at, dt).to(dt)
    # attention: every sequence padded to the longest, the padding masked
    hq, hkv, d, B = c["hq"], c["hkv"], c["d"], c["batch"]
    b, i = _rows(s["cu"], s["total"])
    nq = (s["cu"][1:] - s["cu"][:-1]).long()
    q = torch.zeros(B, s["max_new"], hq, d, device=table.device)
    q[b, i] = s["q"].float()
    j = torch.arange(s["width"], device=table.device)
    at = table[:, j // page], (j % page).expand(B, -1)
    k = _read(s["k_cache"], *at, dt)                                   # [B, S, Hkv, d]
    x = torch.einsum("bihgd,bjhd->bhgij", q.view(B, -1, hkv, hq // hkv, d), k) * d ** -0.5
    del k
    lens = s["lens"].long()
    last = (lens - nq)[:, None] + torch.arange(s["max_new"], device=table.device)
    seen = (j[None, None] <= last[..., None]) & (j[None, None] < lens[:, None, None])  # [B, i, S]
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp_min(torch.finfo(torch.float32).min)).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.where((j[None] < lens[:, None])[..., None, None], _read(s["v_cache"], *at, dt), 0.0)
    o = torch.einsum("bhgij,bjhd->bihgd", p / total, v).reshape(B, -1, hq, d)
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, -1, hq)
    return o[b, i].to(dt), lse[b, i].t().contiguous()


def _write(pool, page, slot, x, dt):
    codes, pairs = _int4_views(pool, dt)
    q, scale, zero = _quantise(x, dt)
    codes[page, :, slot] = q[..., 0::2] | (q[..., 1::2] << 4)
    pairs[page, :, slot] = torch.stack([scale, zero], -1)


# ---------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------
def work(case):
    c = case
    lens, news = _lens(c)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    row = hkv * (2 * d if c["fmt"] == "16" else 5 * d // 8)  # bytes of a token's keys in the pool
    T, K = sum(news), sum(lens)
    if c["op"] == "append":
        # q, k and v in, q out, keys and values into the pages (4 bits: and the packed rows out)
        out = 2 * row * T + (2 * hkv * d * 2 * K if c["fmt"] == "int4" else 0)
        return {"bytes": T * (2 * hq + 2 * hkv) * d * 2 + out, "flops": T * (hq + hkv) * c["rot"] * 3}
    if c["op"] == "gather":
        return {"bytes": K * (2 * row + 2 * hkv * d * 2), "flops": 0 if c["fmt"] == "16" else K * 2 * hkv * d * 2}
    seen = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, news))
    return {"bytes": K * 2 * row + T * hq * (2 * d * 2 + 4), "flops": 4 * hq * d * seen}


# ---------------------------------------------------------------------------------
# The same from the definition, in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------------
def _exact_rows(pool, pages, n, c):
    """Rows 0 .. n - 1 of a sequence whose pages are `pages`, fp64 [n, Hkv, d]."""
    d, hkv, page = c["d"], c["hkv"], c["page"]
    if c["fmt"] == "16":
        return pool[pages].transpose(1, 2).reshape(-1, hkv, d)[:n].double()
    raw = pool[pages].reshape(len(pages), hkv, -1)
    low = raw[:, :, : page * d // 2].reshape(len(pages), hkv, page, d // 2)
    out = torch.empty(len(pages), hkv, page, d, dtype=torch.float64, device=pool.device)
    out[..., 0::2] = (low % 16).double()
    out[..., 1::2] = (low // 16).double()
    tail = raw[:, :, page * d // 2:].contiguous().view(DTYPES[c["dtype"]]).double()
    tail = tail.reshape(len(pages), hkv, page, d // GROUP, 2)
    out = out * tail[..., 0].repeat_interleave(GROUP, -1) + tail[..., 1].repeat_interleave(GROUP, -1)
    return out.transpose(1, 2).reshape(-1, hkv, d)[:n]


def _exact_turn(x, first, c, inv_freq):
    """fp64 [n, H, d] with pair r of row i multiplied by exp(1j * (first + i) * inv_freq[r])."""
    y, rot = x.clone(), c["rot"]
    if rot:
        pos = torch.arange(first, first + x.shape[0], device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), torch.outer(pos, inv_freq.double()))
        re, im = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., re], x[..., im]) * turn[:, None]
        y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_held(x, dt):
    """What 4 bits hold of fp64 [n, H, d]."""
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], GROUP):
        part = x[..., g: g + GROUP]
        zero = part.min(-1, keepdim=True).values.float().to(dt).double()
        scale = ((part.max(-1, keepdim=True).values - zero).clamp(min=0) / 15).float().to(dt).double()
        steps = torch.nan_to_num(torch.round((part - zero) / scale), nan=0.0, posinf=0.0, neginf=0.0).clamp(0, 15)
        out[..., g: g + GROUP] = zero + scale * steps
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens, news = _lens(c)
    dt, page = DTYPES[c["dtype"]], c["page"]
    outs = [[], []]
    if c["op"] == "append":
        qs, at = [], 0
        kp, vp = (s["k_cache"].double(), s["v_cache"].double()) if c["fmt"] == "16" else (None, None)
        for b, (n, m) in enumerate(zip(lens, news)):
            rows = slice(at, at + m)
            at += m
            qs.append(_exact_turn(s["q"][rows].double(), n - m, c, s["inv_freq"]))
            k, v = _exact_turn(s["k"][rows].double(), n - m, c, s["inv_freq"]), s["v"][rows].double()
            pages = s["table"][b, : -(-n // page)].long()
            if c["fmt"] == "16":
                j = torch.arange(n - m, n, device=k.device)
                kp[pages[j // page], :, j % page] = k
                vp[pages[j // page], :, j % page] = v
            else:
                for o, pool, new in ((outs[0], s["k_cache"], k), (outs[1], s["v_cache"], v)):
                    o.append(torch.cat([_exact_rows(pool, pages, n, c)[: n - m], _exact_held(new, dt)]))
        q = torch.cat(qs)
        return (q, kp, vp) if c["fmt"] == "16" else (q, torch.cat(outs[0]), torch.cat(outs[1]))
    if c["op"] == "gather":
        for b, n in enumerate(lens):
            pages = s["table"][b, : -(-n // page)].long()
            outs[0].append(_exact_rows(s["k_cache"], pages, n, c))
            outs[1].append(_exact_rows(s["v_cache"], pages, n, c))
        return torch.cat(outs[0]), torch.cat(outs[1])
    at, group = 0, c["hq"] // c["hkv"]
    for b, (n, m) in enumerate(zip(lens, news)):
        pages = s["table"][b, : -(-n // page)].long()
        k, v = (_exact_rows(p, pages, n, c) for p in (s["k_cache"], s["v_cache"]))
        q = s["q"][at: at + m].double()
        at += m
        hidden = torch.arange(n, device=q.device)[None] > torch.arange(n - m, n, device=q.device)[:, None]
        o, lse = torch.empty_like(q), torch.empty(c["hq"], m, dtype=torch.float64, device=q.device)
        for h in range(c["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            x = torch.matmul(q[:, heads].transpose(0, 1), k[:, h].t()) / c["d"] ** 0.5  # [group, m, n]
            x = torch.where(hidden, -torch.inf, x)
            o[:, heads] = torch.matmul(torch.softmax(x, -1), v[:, h]).transpose(0, 1)
            lse[heads] = torch.logsumexp(x, -1)
        outs[0].append(o)
        outs[1].append(lse)
    return torch.cat(outs[0]), torch.cat(outs[1], 1)
