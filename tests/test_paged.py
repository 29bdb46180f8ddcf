"""Paged KV cache: fa_kv_append (rotation by position, 16-bit and 4-bit pools),
fa_kv_gather and fa_fwd_paged, each against its definition in 64 bits.

Host side (no GPU): refusals of every entry point and of the binding; the definition
written here against closed forms.
GPU: the pools' contents and the rotated queries; read-back; attention over ragged,
empty and causal sequences, bad pages, poisoned places that take no part, pools past
2^31 elements, streams and graphs; and the calls together as a serving loop makes them.
"""
import math

import pytest
import torch

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA = range(4)
FA_ERR_BAD_PAGE = 6
FAKE = 1 << 20
BF16, FP16 = torch.bfloat16, torch.float16
NAN = float("nan")


# ---------------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------------
def half(dt):
    """Half a step of the type, relative to the value: the most one rounding is off."""
    return torch.finfo(dt).eps / 2


def turn(x, pos, inv_freq, interleaved):
    """x [n, H, d] with pair r of row i turned by pos[i] * inv_freq[r]."""
    y, rot = x.double().clone(), 2 * inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    return y


def quantise(x, dt):
    """fp64 [..., d] -> codes [..., d / 32, 32], scale and zero [..., d / 32, 1], all fp64."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    zero = g.amin(-1, keepdim=True).float().to(dt).double()
    scale = ((g.amax(-1, keepdim=True) - zero).clamp_min(0) / 15).float().to(dt).double()
    bad = ~(g.isfinite().all(-1, keepdim=True) & zero.isfinite() & scale.isfinite())
    steps = ((g - zero) / torch.where(scale > 0, scale, 1.0)).round().clamp(0, 15)
    codes = torch.where((scale > 0) & ~bad, steps, 0.0)
    return codes, torch.where(bad, NAN, scale), torch.where(bad, NAN, zero)


def held(x, dt):
    codes, scale, zero = quantise(x, dt)
    return (codes * scale + zero).reshape(x.shape)


def attend(q, k, v, causal, scale):
    """fp64 q [m, Hq, d], k, v [n, Hkv, d] -> o [m, Hq, d], lse [Hq, m], sum_j p_j |v_j| [m, Hq, d]."""
    m, hq, d = q.shape
    n, hkv, _ = k.shape
    kk, vv = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
    x = torch.einsum("ihd,jhd->hij", q, kk) * scale
    if causal:
        i, j = torch.arange(m, device=q.device), torch.arange(n, device=q.device)
        x = x.masked_fill(j[None] > i[:, None] + n - m, -math.inf)
    lse = torch.logsumexp(x, -1) if n else torch.full((hq, m), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(lse.isneginf()[..., None], 0.0, (x - lse[..., None]).exp())
    return torch.einsum("hij,jhd->ihd", p, vv), lse, torch.einsum("hij,jhd->ihd", p, vv.abs())


def test_definition_against_closed_forms():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 128, generator=g, dtype=torch.float64)
    f = torch.tensor([1.0, 0.25] + [0.0] * 6)
    for inter in (False, True):
        y = turn(x, torch.tensor([0, 1, 7, 100, 1 << 30]), f, inter)
        assert torch.equal(y[0], x[0])                                   # position 0
        assert torch.equal(y[..., 16:], x[..., 16:])                     # past rot_dim
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1))    # a turn keeps the norm
        i, j = (2, 3) if inter else (1, 9)                               # pair 1
        z = torch.complex(x[2, 0, i], x[2, 0, j]) * complex(math.cos(1.75), math.sin(1.75))
        assert abs(z - torch.complex(y[2, 0, i], y[2, 0, j])) < 1e-14
    # whole steps are held exactly: 0 .. 15 in one group, and a constant group
    w = torch.cat([torch.arange(32) % 16, torch.full((32,), 2.5)]).double()
    assert torch.equal(held(w, BF16), w)
    # half a step (and the roundings of scale and zero) is the most a finite value is off
    for dt in (BF16, FP16):
        codes, s, z = quantise(x, dt)
        e = (held(x, dt) - x).abs().reshape(5, 2, 4, 32)
        assert (e <= s / 2 + 15 * s * half(dt) + z.abs() * half(dt)).all() and codes.max() == 15
    w[3] = math.inf
    assert held(w, BF16)[:32].isnan().all() and not held(w, BF16)[32:].isnan().any()
    # one key: O = v; equal scores: the mean
    q, v = torch.randn(1, 2, 128, dtype=torch.float64), torch.randn(3, 1, 128, dtype=torch.float64)
    o, lse, _ = attend(q, torch.zeros(3, 1, 128, dtype=torch.float64), v, False, 0.1)
    assert torch.allclose(o[0, 1], v.mean(0)[0]) and torch.allclose(lse, torch.tensor(math.log(3.0)).double())
    o, lse, _ = attend(q.expand(3, 2, 128), v[:1], v[:1], True, 0.1)     # rows 0 and 1 see nothing
    assert (o[:2] == 0).all() and lse[:, :2].isneginf().all() and torch.allclose(o[2, 0], v[0, 0])


# ---------------------------------------------------------------------------------
# Refusals (no GPU)
# ---------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from exact_attention_blackwell_fa_b200 import _lib, build

    build.build()
    return _lib.load()


def append_call(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, qo=2 * FAKE, kc=FAKE, vc=FAKE, cu=FAKE, sk=FAKE,
             bt=FAKE, fr=FAKE, rot=128, inter=0, B=2, total=2, Hq=4, Hkv=2, d=128, ps=16, np=8, mp=4, fmt=0, dt=0)
    a.update(kw)
    return lib.fa_kv_append(*a.values(), None)


def gather_call(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, k=FAKE, v=FAKE, cu=FAKE, bt=FAKE, B=2, total=2, Hkv=2, d=128, ps=16, np=8, mp=4,
             fmt=0, dt=0)
    a.update(kw)
    return lib.fa_kv_gather(*a.values(), None)


def paged_call(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, o=FAKE, lse=FAKE, cu=FAKE, sk=FAKE, bt=FAKE, B=2, mq=1, total=2, Hq=4, Hkv=2,
             d=128, ps=16, np=8, mp=4, fmt=0, causal=0, scale=0.088, dt=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.fa_fwd_paged(*a.values(), None)


POOL_REFUSALS = [
    (dict(kc=None), FA_ERR_INVALID_ARG), (dict(vc=FAKE + 8), FA_ERR_INVALID_ARG), (dict(bt=None), FA_ERR_INVALID_ARG),
    (dict(bt=FAKE + 2), FA_ERR_INVALID_ARG), (dict(cu=None), FA_ERR_INVALID_ARG), (dict(cu=FAKE + 1), FA_ERR_INVALID_ARG),
    (dict(B=0), FA_ERR_INVALID_ARG), (dict(total=-1), FA_ERR_INVALID_ARG), (dict(Hkv=0), FA_ERR_INVALID_ARG),
    (dict(np=0), FA_ERR_INVALID_ARG), (dict(mp=0), FA_ERR_INVALID_ARG), (dict(mp=1 << 27), FA_ERR_INVALID_ARG),
    (dict(d=64), FA_ERR_UNSUPPORTED), (dict(d=160), FA_ERR_UNSUPPORTED), (dict(dt=2), FA_ERR_UNSUPPORTED),
    (dict(fmt=2), FA_ERR_UNSUPPORTED), (dict(ps=8), FA_ERR_UNSUPPORTED), (dict(ps=48), FA_ERR_UNSUPPORTED),
    (dict(ps=512), FA_ERR_UNSUPPORTED), (dict(ps=0), FA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("call", [append_call, gather_call, paged_call])
@pytest.mark.parametrize("kw,code", POOL_REFUSALS)
def test_pool_arguments_refused(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(k=FAKE + 8), dict(q=FAKE + 4), dict(qo=FAKE + 2),
    dict(qs=504), dict(qs=516), dict(ks=128), dict(vs=260), dict(ks=-256), dict(Hq=3), dict(Hq=0), dict(rot=8),
    dict(rot=144), dict(rot=-16), dict(fr=None), dict(fr=FAKE + 1), dict(sk=None), dict(sk=FAKE + 3),
    dict(q=FAKE, qo=FAKE, qs=1024),
])
def test_append_arguments_refused(lib, kw):
    assert append_call(lib, **kw) == FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=FAKE + 8)])
def test_gather_arguments_refused(lib, kw):
    assert gather_call(lib, **kw) == FA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(o=None), dict(lse=None), dict(o=FAKE + 8), dict(sk=None), dict(sk=FAKE + 2), dict(mq=0),
    dict(Hq=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=math.inf),
    dict(total=1 << 29, Hq=4),
])
def test_paged_arguments_refused(lib, kw):
    assert paged_call(lib, **kw) == FA_ERR_INVALID_ARG


def test_no_rows_is_valid_and_launches_nothing(lib):
    assert append_call(lib, total=0, q=None, qo=None, k=None, v=None) == FA_OK
    assert gather_call(lib, total=0, k=None, v=None) == FA_OK
    assert paged_call(lib, total=0, q=None, o=None, lse=None) == FA_OK


def test_valid_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (append_call, gather_call, paged_call):
        for kw in (dict(), dict(fmt=1, dt=1, d=512), dict(ps=256, mp=(1 << 23) - 1)):
            if call is append_call and kw.get("d") == 512:
                kw = dict(kw, qs=2048, ks=1024, vs=1024)
            assert call(lib, **kw) in (FA_ERR_CUDA, FA_ERR_UNSUPPORTED)
    assert append_call(lib, q=None, qo=None) in (FA_ERR_CUDA, FA_ERR_UNSUPPORTED)


def test_sizes_and_status_string(lib):
    assert lib.fa_kv_cache_size(3, 16, 2, 128, 0) == 3 * 16 * 2 * 256
    assert lib.fa_kv_cache_size(3, 16, 2, 128, 1) == 3 * 16 * 2 * 80
    assert lib.fa_kv_cache_size(1 << 20, 256, 8, 512, 0) == 1 << 41
    for bad in ((0, 16, 2, 128, 0), (1, 24, 2, 128, 0), (1, 16, 0, 128, 0), (1, 16, 2, 96, 0), (1, 16, 2, 128, 2)):
        assert lib.fa_kv_cache_size(*bad) == 0
    assert lib.fa_status_string(FA_ERR_BAD_PAGE).decode().startswith("FA_ERR_BAD_PAGE")
    assert lib.fa_fwd_paged_workspace_size(0, 1, 4, 2, 128) == 0
    assert lib.fa_fwd_paged_workspace_size(1, 1, 3, 2, 128) == 0


def test_binding_refuses_cpu_tensors():
    import exact_attention_blackwell_fa_b200 as fa

    pool, i = torch.zeros(2, 1, 16, 128, dtype=BF16), torch.zeros(1, 1, dtype=torch.int32)
    x = torch.zeros(1, 1, 128, dtype=BF16)
    with pytest.raises(ValueError):
        fa.fa_kv_append(x, x, x, pool, pool, i, i[0], i)
    with pytest.raises(ValueError):
        fa.fa_kv_gather(pool, pool, i, i, 1)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(x, pool, pool, i, i[0], i, 1)


# ---------------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------------
def fa_mod():
    import exact_attention_blackwell_fa_b200 as fa

    return fa


def status_ok(fa):
    torch.cuda.synchronize()
    code, detail = fa.fa_last_device_status()
    assert code == 0, f"device status {code} ({detail:#x})"


class Cache:
    """Pools of `spare` more pages than the sequences need, every place poisoned, and a
    block table whose unused entries are no pages."""

    def __init__(self, caps, Hkv, d, page, int4, dt, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        need = [-(-c // page) for c in caps]
        self.caps, self.Hkv, self.d, self.page, self.int4, self.dt = caps, Hkv, d, page, int4, dt
        self.pages = max(1, sum(need) + spare)
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(1, max(need))
        table = torch.tensor([[-7, 1 << 30][(r + c) % 2] for r in range(len(caps)) for c in range(width)],
                             dtype=torch.int32).view(len(caps), width)
        for b, n in enumerate(need):
            for c in range(n):
                table[b, c] = order.pop()
        self.table = table.cuda()
        shape = (self.pages, Hkv, page, 5 * d // 8 if int4 else d)
        self.k, self.v = (torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda") if int4 else
                          torch.full(shape, NAN, dtype=dt, device="cuda") for _ in range(2))

    def rows(self, pool, b, n):
        """fp64 rows 0 .. n - 1 of sequence b, read from the layout's description."""
        j = torch.arange(n, device="cuda")
        pg, slot = self.table[b].long()[j // self.page], j % self.page
        if not self.int4:
            return pool[pg, :, slot].double()
        flat = pool.view(self.pages, self.Hkv, -1)
        codes = flat[..., : self.page * self.d // 2].reshape(self.pages, self.Hkv, self.page, self.d // 2)[pg, :, slot]
        pairs = flat[..., self.page * self.d // 2:].contiguous().view(self.dt)
        pairs = pairs.reshape(self.pages, self.Hkv, self.page, self.d // 32, 2)[pg, :, slot].double()
        c = torch.stack([codes % 16, codes // 16], -1).double().reshape(n, self.Hkv, self.d // 32, 32)
        return (c * pairs[..., :1] + pairs[..., 1:]).flatten(-2)

    def fill(self, lens, seed, amp=1.0):
        """Writes N(0, amp^2) tokens with the append itself, unrotated; returns the fp64 rows."""
        fa, g = fa_mod(), torch.Generator().manual_seed(seed)
        k, v = ((torch.randn(sum(lens), self.Hkv, self.d, generator=g) * amp).to(self.dt).cuda() for _ in range(2))
        fa.fa_kv_append(None, k, v, self.k, self.v, cu_of(lens), i32(lens), self.table)
        return [(self.rows(self.k, b, n), self.rows(self.v, b, n)) for b, n in enumerate(lens)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32([0] + torch.tensor(lens).cumsum(0).tolist())


def randn(*shape, seed, dt=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


APPEND = [
    # news, lens, Hq, Hkv, d, page, rot, interleaved, dtype
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16, 128, False, BF16),
    ([5, 0, 33, 1], [5, 9, 40, 64], 4, 4, 128, 32, 64, True, FP16),
    ([130, 7], [130, 500], 8, 1, 192, 64, 48, False, BF16),
    ([16, 3], [16, 259], 2, 2, 256, 128, 256, True, BF16),
    ([9], [9], 6, 3, 384, 256, 16, False, FP16),
    ([700, 600], [700, 600], 3, 1, 512, 16, 512, False, BF16),     # many tokens per block
    ([1], [1], 1, 1, 128, 16, 0, False, FP16),                     # no rotation
]


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, int4):
    fa = fa_mod()
    news, lens, Hq, Hkv, d, page, rot, inter, dt = APPEND[case]
    T, extra = sum(news), 3                       # `extra` rows behind the last sequence
    c = Cache(lens, Hkv, d, page, int4, dt, seed=case)
    qkv = randn(T + extra, Hq + 2 * Hkv, d, seed=case, dt=dt)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)        # slices of a fused projection
    freq = (10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float().cuda() if rot else None
    q_out = torch.full((T + extra, Hq, d), 7.0, dtype=dt, device="cuda")
    before = [c.k.clone(), c.v.clone()]
    got = fa.fa_kv_append(q, k, v, c.k, c.v, cu_of(news), i32(lens), c.table, inv_freq=freq, interleaved=inter,
                          q_out=q_out)
    status_ok(fa)
    assert got is q_out and (q_out[T:] == 7.0).all()
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(news, lens)]).cuda()
    f = freq if rot else torch.zeros(0, device="cuda")
    turned = lambda x: turn(x[:T], pos, f, inter)
    # fp32 arithmetic (angle, sine and two products: under 8 roundings of 2^-24 of the pair's
    # length), then one rounding to the type; 2^-25 is fp16's half step among its subnormals
    def near(got, ref, x):
        pair = ref.abs().amax(-1, keepdim=True) * 2 ** 0.5
        return ((got.double() - ref).abs() <= half(dt) * ref.abs() * 1.001 + 8 * 2.0 ** -24 * pair + 2.0 ** -25).all()

    assert near(q_out[:T], turned(q), q)
    touched = torch.zeros(c.pages, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, (m, n) in enumerate(zip(news, lens)):
        kr, vr = c.rows(c.k, b, n)[n - m:], c.rows(c.v, b, n)[n - m:]
        kx, vx = turned(k)[at: at + m], v[at: at + m].double()
        if int4:  # every border is decided in 64 bits: the same codes, scales and zeros
            assert torch.equal(kr, held(kx, dt)) and torch.equal(vr, held(vx, dt))
        else:
            assert near(kr, kx, k) and torch.equal(vr, vx)
        j = torch.arange(n - m, n, device="cuda")
        touched[c.table[b].long()[j // page], j % page] = True
        at += m
    # every other place is as it was
    for pool, old in zip((c.k, c.v), before):
        if not int4:
            keep = ~touched[:, None, :, None].expand_as(pool)
            assert torch.equal(pool[keep].view(torch.int16), old[keep].view(torch.int16))
        else:
            for lo, w in ((0, d // 2), (page * d // 2, d // 8)):
                part = lambda t: t.view(c.pages, Hkv, -1)[..., lo: lo + page * w].reshape(c.pages, Hkv, page, w)
                keep = ~touched[:, None, :, None].expand(c.pages, Hkv, page, w)
                assert torch.equal(part(pool)[keep], part(old)[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_append_far_positions_in_place_and_without_queries(int4):
    """Positions just under 2^31 turn as exactly as near ones; q may be overwritten; K and V alone."""
    fa = fa_mod()
    page, width, d = 256, (1 << 23) - 1, 128
    n = page * width
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    c = Cache([page, page], 1, d, page, int4, BF16)
    freq = (500000.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()
    freq[3], freq[5] = -2.5, 40.0                          # any finite frequency
    q, k, v = (randn(4, h, d, seed=s) for h, s in ((2, 1), (1, 2), (1, 3)))
    q0 = q.clone()
    for with_q in (False, True):
        out = fa.fa_kv_append(q if with_q else None, k, v, c.k, c.v, i32([0, 4]), i32([n]), table, inv_freq=freq,
                              q_out=q if with_q else None)
        status_ok(fa)
        assert out is (q if with_q else None)
    pos = torch.arange(n - 4, n, device="cuda")
    a = pos[:, None].double() * freq.double()
    # the angle is off by its own 2^-53 here and in the definition (2^31 * 40 * 2^-53 = 1e-5)
    # and by fp32's rounding of the reduced turn, sine and products; then one rounding
    off = 4e-5 * k.abs().max().double()
    ref = turn(q0, pos, freq, False)
    assert a.max() > 8e10
    assert ((q.double() - ref).abs() <= half(BF16) * 1.001 * ref.abs() + 4e-5 * q0.abs().max()).all()
    c.table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
    got, ref = c.rows(c.k, 0, page)[-4:], turn(k, pos, freq, False)
    if int4:  # half a step, and the roundings of scale and zero
        _, sc, z = quantise(ref, BF16)
        most = (sc * (0.5 + 16 * half(BF16)) * 1.01 + z.abs() * half(BF16) * 1.01 + off).expand(4, 1, 4, 32)
        assert ((got - ref).abs() <= most.reshape(4, 1, 128)).all()
    else:
        assert ((got - ref).abs() <= half(BF16) * 1.001 * ref.abs() + off).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_append_int4_borders_and_non_finite_groups(dt):
    """Exact ties between codes, constant groups, groups with an infinity or a NaN, and
    the type's extremes, in values and in keys at position 0 (the turn is the identity)."""
    fa = fa_mod()
    c = Cache([16], 1, 128, 16, True, dt)
    x = torch.zeros(8, 1, 128)
    x[0] = torch.arange(128) % 31 / 2                           # scale 1, every half code: ties to even
    x[1] = 3.140625
    x[2, 0, 40] = math.inf
    x[2, 0, 70] = -math.inf
    x[2, 0, 100] = NAN
    x[3] = torch.finfo(dt).max * torch.linspace(-1, 1, 128)
    x[4] = torch.finfo(dt).tiny * (torch.arange(128) % 7)
    x[5] = 1000 + (torch.arange(128) % 5)
    x[6] = torch.randn(128, generator=torch.Generator().manual_seed(5))
    x[7] = -x[0]
    x = x.to(dt).cuda()
    freq = torch.zeros(64, device="cuda")
    fa.fa_kv_append(None, x, x, c.k, c.v, i32([0, 8]), i32([8]), c.table, inv_freq=freq)
    status_ok(fa)
    # the turn by a zero angle is the identity, but for an infinity's 0 * inf in its partner
    refs = [held(turn(x, torch.arange(8, device="cuda"), freq, False), dt), held(x.double(), dt)]
    assert refs[0][2].isnan().all() and refs[1][2].isnan().sum() == 96
    got = fa.fa_kv_gather(c.k, c.v, i32([0, 8]), c.table, 8, dt)
    status_ok(fa)
    for pool, ref, back in zip((c.k, c.v), refs, got):
        assert torch.equal(c.rows(pool, 0, 8).nan_to_num(nan=1e30), ref.nan_to_num(nan=1e30))
        assert not ref[[0, 1, 3, 4, 5, 6, 7]].isnan().any() and torch.equal(ref[1], x[1].double())
        assert torch.equal(back.isnan(), ref.isnan())
        fin = ~ref.isnan()
        # scale * c + zero in fp32 (exact but for 2^-24), then one rounding to the type
        e = (back.double() - ref).abs()[fin]
        assert (e <= (half(dt) * 1.001 + 2.0 ** -24) * ref.abs()[fin] + torch.finfo(dt).smallest_normal * half(dt)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,page,dt", [(128, 16, BF16), (192, 64, FP16), (256, 32, BF16), (384, 256, FP16), (512, 128, BF16)])
def test_gather(d, page, dt, int4):
    fa = fa_mod()
    lens, take, Hkv = [1, 300, 64, 0, 129], [1, 257, 0, 0, 129], 3
    c = Cache(lens, Hkv, d, page, int4, dt, seed=d)
    rows = c.fill(lens, seed=d)
    total = sum(take)
    k, v = (torch.full((total + 2, Hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
    fa.fa_kv_gather(c.k, c.v, cu_of(take), c.table, total + 2, dt, k=k, v=v)
    status_ok(fa)
    assert (k[total:] == 7.0).all() and (v[total:] == 7.0).all()
    for got, i in ((k, 0), (v, 1)):
        ref = torch.cat([r[i][:n] for r, n in zip(rows, take)])
        if int4:
            assert ((got[:total].double() - ref).abs() <= (half(dt) * 1.001 + 2.0 ** -24) * ref.abs() + 2.0 ** -25).all()
        else:
            assert torch.equal(got[:total].double(), ref)


def check_paged(c, rows, q, news, lens, causal, scale, o, lse, max_q=None):
    """o, lse of one call against the definition over the rows the pools stand for."""
    dt, at = c.dt, 0
    for b, (m, n) in enumerate(zip(news, lens)):
        mm = m if max_q is None else min(m, max_q)
        qs, k, v = q[at: at + mm].double(), rows[b][0][:n], rows[b][1][:n]
        ro, rl, mass = attend(qs, k, v, causal, scale)
        go, gl = o[at: at + mm].double(), lse[:, at: at + mm].double()
        at += m
        empty = rl.isneginf()
        assert torch.equal(gl.isneginf(), empty)
        assert (go.transpose(0, 1)[empty] == 0).all()
        # scores: d products summed in fp32, each addition off by 2^-23 of the running sum at most;
        # 2^-21: the exponentials, the row sum and the logarithm
        if n:
            kn = k.abs().repeat_interleave(q.shape[1] // c.Hkv, 1)
            size = torch.einsum("ihd,jhd->hij", qs.abs(), kn).amax(-1) * scale
            tol = size * c.d * 2.0 ** -23 + 2.0 ** -21 * (1 + rl.masked_fill(empty, 0).abs())
            assert bool(((gl - rl).abs()[~empty] <= tol[~empty]).all()), (b, (gl - rl)[~empty].abs().max().item())
            # O: the output's rounding, and P's and V's to the type (half a step each), all
            # relative to what they act on, and the scores' error in every weight
            err = tol.transpose(0, 1)[..., None]
            bound = half(dt) * ro.abs() * 1.01 + (2.02 * half(dt) + 2 * err) * mass + 2.0 ** -24
            assert bool(((go - ro).abs() <= bound).all()), (b, ((go - ro).abs() - bound).max().item())
        else:
            assert (go == 0).all()


ATTEND = [
    # news, lens, Hq, Hkv, d, page, dtype
    ([1], [1], 1, 1, 128, 16, BF16),
    ([1, 1, 1, 1], [1, 15, 16, 17], 8, 1, 128, 16, FP16),
    ([1, 1, 1, 1, 1], [513, 0, 127, 2000, 64], 32, 4, 128, 32, BF16),
    ([3, 0, 8, 1], [100, 40, 5, 777], 8, 2, 128, 64, BF16),         # more queries than keys
    ([17, 40], [1030, 40], 12, 4, 128, 128, FP16),                   # groups of 3; several row blocks
    ([1, 5], [300, 1025], 16, 1, 192, 16, FP16),
    ([2, 1], [260, 1500], 8, 8, 256, 256, BF16),
    ([1, 4, 9], [33, 400, 9], 5, 1, 384, 32, BF16),
    ([1, 2], [777, 70], 8, 1, 512, 64, FP16),
    ([1] * 37, [(7 * i * i) % 211 for i in range(37)], 4, 2, 128, 16, BF16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_paged_forward(case, int4, causal):
    fa = fa_mod()
    news, lens, Hq, Hkv, d, page, dt = ATTEND[case]
    c = Cache(lens, Hkv, d, page, int4, dt, seed=case)
    rows = c.fill(lens, seed=case)
    T, extra = sum(news), 2
    q = randn(T + extra, Hq, d, seed=100 + case, dt=dt)
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, T + extra), 7.0, device="cuda")
    scale = d ** -0.5
    fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, max(news), causal=causal, out=o, lse=lse)
    status_ok(fa)
    assert (o[T:] == 7.0).all() and (lse[:, T:] == 7.0).all()       # rows behind the last sequence
    check_paged(c, rows, q, news, lens, causal, scale, o, lse)
    # the same bits again, on another stream with a workspace of its own
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        need = fa.fa_fwd_paged_workspace_size(len(lens), max(news), Hq, Hkv, d)
        ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")   # contents do not matter
        o2, lse2 = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, max(news), causal=causal,
                                   workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    status_ok(fa)
    assert torch.equal(o2[:T], o[:T]) and torch.equal(lse2[:, :T], lse[:, :T])


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_paged_forward_sharp_scores_and_large_values(int4):
    """Scores that grow along the keys (every tile raises the running maximum) and a scale
    far from 1/sqrt(d): the statistics stay those of the definition."""
    fa = fa_mod()
    news, lens, Hq, Hkv, d, dt = [1, 2], [900, 400], 8, 2, 128, BF16
    c = Cache(lens, Hkv, d, 16, int4, dt)
    k = randn(sum(lens), Hkv, d, seed=1) * torch.linspace(0.1, 6, sum(lens), device="cuda")[:, None, None].to(dt)
    v = randn(sum(lens), Hkv, d, seed=2) * 100
    fa.fa_kv_append(None, k, v, c.k, c.v, cu_of(lens), i32(lens), c.table)
    rows = [(c.rows(c.k, b, n), c.rows(c.v, b, n)) for b, n in enumerate(lens)]
    q = randn(3, Hq, d, seed=3)
    for scale in (0.5, 1e-6):
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, 2, causal=True, scale=scale)
        status_ok(fa)
        check_paged(c, rows, q, news, lens, True, scale, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("d", [128, 192, 256, 384, 512])
def test_paged_forward_every_head_dim_and_row_count(d, dt, int4):
    """One, two and four tiles of eight rows (and several blocks of them), short sequences
    kept whole and long ones cut into pieces, for every head dim, type and pool."""
    fa = fa_mod()
    Hq, Hkv, page = 10, 2, 64                                        # groups of 5
    for news, lens in (([1, 1], [70, 33]), ([3, 1], [300, 1200]), ([2, 6], [900, 17]), ([11], [513])):
        c = Cache(lens, Hkv, d, page, int4, dt, seed=d)
        rows = c.fill(lens, seed=d + 1)
        q = randn(sum(news), Hq, d, seed=d + 2, dt=dt)
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, max(news), causal=True)
        status_ok(fa)
        check_paged(c, rows, q, news, lens, True, d ** -0.5, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_paged_forward_many_sequences(int4):
    """More sequences than a block has threads, some without queries, some without keys."""
    fa = fa_mod()
    B, Hq, Hkv, d, dt = 700, 4, 1, 128, BF16
    lens = [(37 * b) % 151 for b in range(B)]
    news = [(b % 5 != 0) + (b % 7 == 0) for b in range(B)]
    lens[650] = 3000
    c = Cache(lens, Hkv, d, 16, int4, dt)
    rows = c.fill(lens, seed=1)
    q = randn(sum(news), Hq, d, seed=2, dt=dt)
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, max(news), causal=True)
    status_ok(fa)
    check_paged(c, rows, q, news, lens, True, d ** -0.5, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_paged_forward_query_magnitudes(dt):
    """4-bit pools scale each query row by a power of two: rows of zeros, of tiny and of
    large values, side by side in one tile."""
    fa = fa_mod()
    lens, d = [400], 128
    c = Cache(lens, 1, d, 32, True, dt)
    rows = c.fill(lens, seed=1)
    e = [0.0, 1.0, 2.0 ** -12, 2.0 ** 10, 2.0 ** -20 if dt == FP16 else 2.0 ** -100, 2.0 ** 13 if dt == FP16 else 2.0 ** 30]
    q = randn(1, len(e), d, seed=2, dt=dt).clamp(-3, 3) * torch.tensor(e, device="cuda").to(dt)[None, :, None]
    for scale in (d ** -0.5, 1e-5, 2.0 ** -40):
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1]), i32(lens), c.table, 1, scale=scale)
        status_ok(fa)
        # rows whose scores the definition's own softmax cannot tell apart in 32 bits are left out
        sizes = (torch.einsum("ihd,jhd->hij", q.double().abs(), rows[0][0].abs().expand(-1, len(e), -1)).amax(-1)[:, 0] * scale)
        fine = (sizes < 1e3).nonzero()[:, 0]
        assert fine.numel() >= 3 and o.isfinite().all()
        check_paged(c, rows, q[:, fine], [1], lens, False, scale, o[:, fine], lse[fine])


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_a_nan_stays_in_its_sequence(int4):
    """A NaN among a sequence's visible keys or values makes that sequence's outputs NaN
    and no other's; one past its end or behind the causal limit does nothing."""
    fa = fa_mod()
    lens, news, d, dt = [50, 700, 60], [1, 1, 2], 128, BF16
    for n in (49, 699, 3):                      # in a whole sequence, in a cut one's last piece
        for which in ("k", "v"):
            c = Cache(lens, 1, d, 16, int4, dt)
            k, v = randn(sum(lens), 1, d, seed=1), randn(sum(lens), 1, d, seed=2)
            b = 1 if n == 699 else 0
            at = sum(lens[:b]) + n
            (k if which == "k" else v)[at] = NAN
            fa.fa_kv_append(None, k, v, c.k, c.v, cu_of(lens), i32(lens), c.table)
            q = randn(sum(news), 4, d, seed=3)
            o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(lens), c.table, 2, causal=True)
            status_ok(fa)
            assert o[b].isnan().all() and o[[i for i in range(4) if i != b]].isfinite().all()
            assert lse[:, b].isnan().all() == (which == "k")
            assert lse[:, [i for i in range(4) if i != b]].isfinite().all()
            cut = list(lens)
            cut[b] = n                          # the NaN is the first token past the end
            if n:
                o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of(news), i32(cut), c.table, 2, causal=True)
                status_ok(fa)
                assert o.isfinite().all() and lse.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,group,dt", [(128, 4, BF16), (128, 1, FP16), (256, 3, FP16), (512, 2, BF16), (192, 8, BF16)])
def test_non_finite_values_behind_the_causal_limit(d, group, dt, int4):
    """A token's infinity or NaN, in its key or its values, reaches the queries that see it
    and none before it."""
    fa = fa_mod()
    news, n = [4], 70
    for at, bad in ((69, NAN), (68, math.inf), (67, NAN), (66, -math.inf)):  # the last new tokens
        for which in ("k", "v"):
            c = Cache([n], 1, d, 16, int4, dt)
            k, v = randn(n, 1, d, seed=1, dt=dt), randn(n, 1, d, seed=2, dt=dt)
            (k if which == "k" else v)[at, 0, 5] = bad
            q = randn(4, group, d, seed=3, dt=dt).abs() + 0.5
            fa.fa_kv_append(None, k, v, c.k, c.v, i32([0, n]), i32([n]), c.table)
            o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 4]), i32([n]), c.table, 4, causal=True)
            status_ok(fa)
            first = at - (n - 4)                 # the first query that sees it
            rows = [(c.rows(c.k, 0, n), c.rows(c.v, 0, n))]
            assert o[:first].isfinite().all() and lse[:, :first].isfinite().all()
            if first:
                clean = [(r[0][: n - 4 + first], r[1][: n - 4 + first]) for r in rows]
                check_paged(c, clean, q[:first], [first], [n - 4 + first], True, d ** -0.5, o[:first], lse[:, :first])
            seen = o[first:]
            if which == "v":                     # only the dims that hold it (4 bits: their group)
                dims = torch.zeros(d, dtype=torch.bool, device="cuda")
                dims[0 if int4 else 5: 32 if int4 else 6] = True
                want = torch.tensor(NAN if int4 else bad)
                got = seen[..., dims].float()
                assert got.isnan().all() if want.isnan() else (got == want.item()).all()
                assert seen[..., ~dims].isfinite().all() and lse.isfinite().all()
            elif int4 or bad != -math.inf:       # (a score of -inf takes no part)
                assert seen.isnan().all() and not lse[:, first:].isfinite().any()


@pytest.mark.gpu
def test_explicit_streams_and_two_calls_at_once():
    """stream= as a torch stream and as a raw handle; two calls in flight on two streams."""
    fa = fa_mod()
    lens, d, Hq = [3000, 500], 128, 8
    c = Cache(lens, 2, d, 16, False, BF16)
    c.fill(lens, seed=1)
    cu, sk = i32([0, 1, 2]), i32(lens)
    qs = [randn(2, Hq, d, seed=s) for s in (2, 3)]
    want = [fa.fa_fwd_paged(q, c.k, c.v, cu, sk, c.table, 1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        got = [fa.fa_fwd_paged(q, c.k, c.v, cu, sk, c.table, 1, stream=s if rep % 2 else s.cuda_stream)
               for q, s in zip(qs, streams)]
        k, v = fa.fa_kv_gather(c.k, c.v, cu_of(lens), c.table, sum(lens), stream=streams[0])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref = torch.cat([c.rows(c.k, b, n) for b, n in enumerate(lens)])
    assert torch.equal(k.double(), ref)
    for s in (0, torch.cuda.default_stream()):
        o, lse = fa.fa_fwd_paged(qs[0], c.k, c.v, cu, sk, c.table, 1, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    x = randn(2, 2, d, seed=5)
    fa.fa_kv_append(None, x, x, c.k, c.v, cu, sk, c.table, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(c.rows(c.v, 0, 3000)[-1], x[0].double())
    status_ok(fa)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_bad_pages_are_left_out_and_reported(int4):
    """Entries that are no pages: nothing is written for them, they read as zeros, take no
    part in attention, and the device status says so."""
    fa = fa_mod()
    lens, Hkv, d, page, dt = [100, 40], 2, 128, 16, BF16
    c = Cache(lens, Hkv, d, page, int4, dt)
    rows = c.fill(lens, seed=4)
    good = c.table.clone()
    c.table[0, 2], c.table[0, 6], c.table[1, 0] = -1, c.pages, 1 << 30
    gone = [torch.arange(n, device="cuda") // page for n in lens]
    keep = [(gone[0] != 2) & (gone[0] != 6), gone[1] != 0]
    q = randn(2, 4, d, seed=5)
    fa.fa_clear_device_status()
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1, 2]), i32(lens), c.table, 1)
    assert fa.fa_last_device_status()[0] == FA_ERR_BAD_PAGE
    fa.fa_clear_device_status()
    kept = [(r[0][m], r[1][m]) for r, m in zip(rows, keep)]
    check_paged(c, kept, q, [1, 1], [int(m.sum()) for m in keep], False, d ** -0.5, o, lse)
    k, _ = fa.fa_kv_gather(c.k, c.v, cu_of(lens), c.table, sum(lens), dt)
    assert fa.fa_last_device_status()[0] == FA_ERR_BAD_PAGE
    fa.fa_clear_device_status()
    mask = torch.cat(keep)
    assert (k[~mask] == 0).all() and (k[mask] != 0).any()
    # append: positions past the table, before it, and bad entries leave the pools alone
    before = c.k.clone()
    x = randn(9, Hkv, d, seed=6)
    fa.fa_kv_append(None, x, x, c.k, c.v, i32([0, 4, 9]), i32([7 * page + 4, 3]), c.table)
    assert fa.fa_last_device_status()[0] == FA_ERR_BAD_PAGE
    fa.fa_clear_device_status()
    assert torch.equal(c.k.view(torch.uint8), before.view(torch.uint8))
    # lengths beyond the table count as the table's; negative ones as none
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1, 2]), i32([1 << 30, -5]), good, 1)
    assert fa.fa_last_device_status()[0] == FA_ERR_BAD_PAGE
    fa.fa_clear_device_status()
    assert (o[1] == 0).all() and lse[:, 1].isneginf().all()
    status_ok(fa)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_pool_past_32_bit_offsets(int4):
    """Pages whose elements lie past 2^31 (16-bit) and bytes past 2^32."""
    fa = fa_mod()
    Hkv, d, page = 8, 512, 256
    block = Hkv * page * (320 if int4 else 1024)
    pages = (1 << 32) // block + 3
    shape = (pages, Hkv, page, 320 if int4 else 512)
    k_cache, v_cache = (torch.empty(shape, dtype=torch.uint8 if int4 else BF16, device="cuda") for _ in range(2))
    c = Cache([300], Hkv, d, page, int4, BF16)
    k, v = randn(300, Hkv, d, seed=1), randn(300, Hkv, d, seed=2)
    table = i32([[pages - 1, pages - 2]])
    for kc, vc, t in ((k_cache, v_cache, table), (c.k, c.v, c.table)):
        fa.fa_kv_append(None, k, v, kc, vc, i32([0, 300]), i32([300]), t)
    q = randn(1, 8, d, seed=3)
    a = fa.fa_fwd_paged(q, k_cache, v_cache, i32([0, 1]), i32([300]), table, 1)
    b = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1]), i32([300]), c.table, 1)
    x = fa.fa_kv_gather(k_cache, v_cache, i32([0, 300]), table, 300, BF16)
    y = fa.fa_kv_gather(c.k, c.v, i32([0, 300]), c.table, 300, BF16)
    status_ok(fa)
    for s, t in zip(a + x, b + y):
        assert torch.equal(s, t)
    check_paged(c, [(c.rows(c.k, 0, 300), c.rows(c.v, 0, 300))], q, [1], [300], False, d ** -0.5, *b)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_queries_past_max_seqlen_q_are_cut(int4):
    fa = fa_mod()
    c = Cache([50, 60], 1, 128, 16, int4, BF16)
    rows = c.fill([50, 60], seed=1)
    q = randn(7, 2, 128, seed=2)
    o, lse = torch.full_like(q, 7.0), torch.full((2, 7), 7.0, device="cuda")
    fa.fa_fwd_paged(q, c.k, c.v, i32([0, 5, 7]), i32([50, 60]), c.table, 2, causal=True, out=o, lse=lse)
    status_ok(fa)
    assert (o[2:5] == 7.0).all() and (lse[:, 2:5] == 7.0).all()
    check_paged(c, rows, q, [5, 2], [50, 60], True, 128 ** -0.5, o, lse, max_q=2)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
def test_captured_decode_step_replays_with_new_lengths(int4):
    """Append and attention of one step captured once; replayed while the sequences grow
    across page borders, the table gets new pages and an eager call runs in between."""
    fa = fa_mod()
    B, Hq, Hkv, d, page, dt, steps = 3, 8, 2, 128, 16, BF16, 20
    caps = [40, 300, 25]
    lens = [c - steps for c in caps]
    c = Cache(caps, Hkv, d, page, int4, dt)
    c.fill(lens, seed=1)
    freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()
    qkv = torch.zeros(B, Hq + 2 * Hkv, d, dtype=dt, device="cuda")
    cu, sk = i32(list(range(B + 1))), i32(lens)
    table = torch.full_like(c.table, -1)
    q_out, o = (torch.empty(B, Hq, d, dtype=dt, device="cuda") for _ in range(2))
    lse = torch.empty(Hq, B, device="cuda")
    ws = torch.empty(max(256, fa.fa_fwd_paged_workspace_size(B, 1, Hq, Hkv, d)), dtype=torch.uint8, device="cuda")

    def step():
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        fa.fa_kv_append(q, k, v, c.k, c.v, cu, sk, table, inv_freq=freq, q_out=q_out)
        fa.fa_fwd_paged(q_out, c.k, c.v, cu, sk, table, 1, causal=True, out=o, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        sk.zero_()
        step()                                   # outside any sequence's table: warm, writes nothing
    torch.cuda.synchronize()
    fa.fa_clear_device_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        new = randn(B, Hq + 2 * Hkv, d, seed=50 + i)
        now = [n + i + 1 for n in lens]
        qkv.copy_(new)
        sk.copy_(i32(now))
        for b in range(B):
            table[b, : -(-now[b] // page)] = c.table[b, : -(-now[b] // page)]
        graph.replay()
        if i % 7 == 0:                           # an eager call between replays
            fa.fa_fwd_paged(q_out.clone(), c.k, c.v, cu, sk, table, 1, causal=True)
        status_ok(fa)
        pos = i32(now).long() - 1
        ref_q = turn(new[:, :Hq], pos, freq, False)
        assert ((q_out.double() - ref_q).abs() <= half(dt) * 1.01 * ref_q.abs() + 2.0 ** -19).all()
        rows = [(c.rows(c.k, b, n), c.rows(c.v, b, n)) for b, n in enumerate(now)]
        check_paged(c, rows, q_out, [1] * B, now, True, d ** -0.5, o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (256, 4, 4)])
def test_serving_loop(oracle_mod, d, Hq, Hkv, int4):
    """The calls together: a prompt in two chunks (append, read back, variable-length
    forward), then single tokens (append, paged forward); every output against the
    oracle over the rows the cache stands for."""
    fa = fa_mod()
    dt, page, chunks, steps = BF16, 32, [[150, 1], [77, 130]], 3
    caps = [sum(x) + steps for x in zip(*chunks)]
    B, have = len(caps), [0] * len(caps)
    c = Cache(caps, Hkv, d, page, int4, dt)
    freq = (10000.0 ** (-torch.arange(0, d // 2, 2).double() / (d // 2))).float().cuda()
    stages = chunks + [[1] * B] * steps
    for n, news in enumerate(stages):
        have = [h + m for h, m in zip(have, news)]
        qkv = randn(sum(news), Hq + 2 * Hkv, d, seed=n)
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        cu, sk = cu_of(news), i32(have)
        q = fa.fa_kv_append(q, k, v, c.k, c.v, cu, sk, c.table, inv_freq=freq, interleaved=True)
        if n < len(chunks):
            ck = cu_of(have)
            kk, vv = fa.fa_kv_gather(c.k, c.v, ck, c.table, sum(have), dt)
            o, lse = fa.fa_fwd_varlen(q, kk, vv, cu, ck, max(news), max(have), causal=True)
        else:
            o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu, sk, c.table, 1, causal=True)
        status_ok(fa)
        at = 0
        for b, m in enumerate(news):
            kr, vr = (c.rows(p, b, have[b]).to(dt)[None] for p in (c.k, c.v))
            ro, rl = oracle_mod.fwd(q[None, at: at + m], kr, vr, causal=True)
            err = (o[at: at + m].cpu().double() - ro[0]).abs()
            # the library's forward bound (1e-2 before the output's rounding); 4-bit rows are
            # rounded to the type on read-back, one half step more
            assert (err <= 1e-2 + 2 * half(dt) * ro[0].abs() + (half(dt) * 4 if int4 else 0)).all()
            assert (lse[:, at: at + m].cpu().double() - rl[0]).abs().max() <= 1e-3 + (2e-2 if int4 else 0)
            at += m


@pytest.mark.gpu
def test_binding_refusals():
    fa = fa_mod()
    c = Cache([40], 2, 128, 16, False, BF16)
    i, s = i32([0, 1]), i32([1])
    q, k = randn(1, 4, 128, seed=0), randn(1, 2, 128, seed=1)
    ok = lambda **kw: fa.fa_kv_append(**{**dict(q=q, k=k, v=k, k_cache=c.k, v_cache=c.v, cu_seqlens=i, seqlens_k=s,
                                                block_table=c.table), **kw})
    ok()
    bad = [dict(q=q.half()), dict(v=k.half()), dict(k=randn(1, 3, 128, seed=2)), dict(seqlens_k=i),
           dict(cu_seqlens=i.long()), dict(block_table=c.table[0]), dict(block_table=c.table.t()),
           dict(inv_freq=torch.ones(64, device="cuda").double()), dict(q_out=torch.empty(2, 4, 128, device="cuda", dtype=BF16)),
           dict(q=q.expand(1, 4, 128)[..., ::2]), dict(k_cache=c.k.half()), dict(v_cache=c.v[1:]),
           dict(q=None, q_out=q), dict(v=randn(2, 2, 128, seed=3)), dict(seqlens_k=s.cpu()),
           dict(k=randn(1, 128, 2, seed=2).transpose(1, 2)), dict(v=k[0])]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            ok(**kw)
    for kw in (dict(inv_freq=torch.ones(4, device="cuda")), dict(inv_freq=torch.ones(72, device="cuda")),
               dict(q=torch.zeros(2, 8, 128, dtype=BF16, device="cuda")[:, :4][:1].expand(2, 4, 128),
                    k=randn(2, 2, 128, seed=1), v=randn(2, 2, 128, seed=1))):
        with pytest.raises(fa.FAError):
            ok(**kw)
    with pytest.raises(ValueError):
        fa.fa_kv_gather(c.k.view(torch.uint8), c.v.view(torch.uint8), i, c.table, 1)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(randn(1, 4, 256, seed=1), c.k, c.v, i, s, c.table, 1)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged(randn(1, 3, 128, seed=1), c.k, c.v, i, s, c.table, 1)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged(q, c.k, c.v, i, s, c.table, 0)
    e = q[:0]
    o, lse = fa.fa_fwd_paged(e, c.k, c.v, i32([0, 0]), s, c.table, 1)
    assert o.shape == e.shape and lse.shape == (4, 0)
    status_ok(fa)
