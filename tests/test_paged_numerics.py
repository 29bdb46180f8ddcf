"""Paged KV cache at the edges of the types' ranges: small softmax weights, infinities among
the values, 4-bit groups and queries of the largest magnitudes; each against its definition
in 64 bits."""
import math

import pytest
import torch

from test_paged import (BF16, FP16, NAN, Cache, attend, check_paged, cu_of, fa_mod, half, held, i32, quantise, randn,
                        status_ok, turn)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("d,Hq,Hkv,lens", [(128, 8, 2, [3000, 60]), (256, 4, 1, [1500]), (512, 2, 2, [700, 33])])
def test_small_weights_beside_dominating_keys(d, Hq, Hkv, lens, dt, int4):
    """Every 16th key dominates and its value is 0: the output is what the others, 12 to 20
    nats below, weigh."""
    fa, n = fa_mod(), sum(lens)
    g = torch.Generator().manual_seed(d)
    for gap in (12.0, 15.0, 17.0, 20.0):
        c = Cache(lens, Hkv, d, 32, int4, dt)
        k, v = torch.zeros(n, Hkv, d), 20000.0 + 500.0 * torch.randn(n, Hkv, d, generator=g)
        k[..., 0] = (0.3 * torch.randn(n, Hkv, generator=g) - gap) / 4
        k[5::16] = 0.0
        v[5::16] = 0.0
        fa.fa_kv_append(None, k.to(dt).cuda(), v.to(dt).cuda(), c.k, c.v, cu_of(lens), i32(lens), c.table)
        rows = [(c.rows(c.k, b, m), c.rows(c.v, b, m)) for b, m in enumerate(lens)]
        q = torch.zeros(len(lens), Hq, d, dtype=dt, device="cuda")
        q[..., 0] = 4.0
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu_of([1] * len(lens)), i32(lens), c.table, 1, scale=1.0)
        status_ok(fa)
        for b, m in enumerate(lens):
            ro, rl, mass = attend(q[b: b + 1].double(), *rows[b], False, 1.0)
            # scores: one product each, summed with zeros (4 bits: scale * code and zero, each
            # rounded, and their sum) and scaled, four roundings of 2^-24 of at most 21 * log2 e;
            # exponentials, row sum and division 2^-21
            err = 4 * 2.0 ** -24 * 31 + 2.0 ** -21
            # a weight is held in two terms of the type: bf16 to 2^-16 of itself; fp16 to 2^-20
            # of itself or half its least step, 2^-25, where the largest weight is at least 2^14
            held_to = 2.0 ** -16 if dt == BF16 else 2.0 ** -20
            floor = 0.0 if dt == BF16 else m * 2.0 ** -39 * rows[b][1].abs().max()
            bound = half(dt) * 1.01 * ro.abs() + (err + held_to + (half(dt) * 1.01 if int4 else 0)) * mass + floor + 2.0 ** -25
            e = (o[b: b + 1].double() - ro).abs()
            assert bool((e <= bound).all()), (gap, b, (e / ro.abs()).max().item(), (bound / ro.abs()).max().item())
            assert ((lse[:, b: b + 1].double() - rl).abs() <= 1e-4).all()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("up", [2.0 ** 8, 2.0 ** 9, 2.0 ** 10, 2.0 ** 11, 2.0 ** 13])
def test_fp16_scores_further_apart_than_the_reference(up, int4):
    """Scores of 2^16 to 2^30, where 32 bits step by more than what lies between the reference
    and the greatest score: weights stay inside fp16, and the greatest score's value comes out."""
    fa, d, n, dt = fa_mod(), 128, 600, FP16
    c = Cache([n], 2, d, 32, int4, dt)
    k, v = randn(n, 2, d, seed=1, dt=dt) * up, randn(n, 2, d, seed=2, dt=dt)
    fa.fa_kv_append(None, k, v, c.k, c.v, i32([0, n]), i32([n]), c.table)
    rows = c.rows(c.k, 0, n), c.rows(c.v, 0, n)
    q = randn(1, 16, d, seed=3, dt=dt) * up
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1]), i32([n]), c.table, 1, scale=1.0)
    status_ok(fa)
    x = torch.einsum("hd,jhd->hj", q[0].double(), rows[0].repeat_interleave(8, 1))
    size = torch.einsum("hd,jhd->hj", q[0].double().abs(), rows[0].abs().repeat_interleave(8, 1)).amax(-1)
    best, order = x.sort(-1, descending=True)
    off = size * d * 2.0 ** -23                          # of a score: d products summed in fp32
    assert o.isfinite().all() and ((lse[:, 0].double() - best[:, 0]).abs() <= off + 2.0 ** -21 * best[:, 0].abs() + 1).all()
    alone = best[:, 0] - best[:, 1] > 2 * off + 40       # the others weigh nothing
    assert alone.any()
    for h in alone.nonzero()[:, 0].tolist():
        want = rows[1][order[h, 0], h // 8]
        assert ((o[0, h].double() - want).abs() <= 2.02 * half(dt) * want.abs() + 2.0 ** -24).all()


def check_infinite(dims, o, lse, c, rows, q, news, lens, causal, scale):
    """dims: {dim: what every output holds there}; the other dims and the LSE are the definition's."""
    o, rows = o.clone(), [(k, v.clone()) for k, v in rows]
    for dim, want in dims.items():
        got = o[..., dim].float()
        assert got.isnan().all() if math.isnan(want) else (got == want).all(), (dim, want, got)
        o[..., dim] = 0
        for _, v in rows:
            v[..., dim] = 0
    check_paged(c, rows, q, news, lens, causal, scale, o, lse)


@pytest.mark.parametrize("d,group,dt", [(128, 4, BF16), (128, 8, FP16), (128, 1, BF16), (192, 2, FP16), (256, 8, BF16),
                                        (384, 3, FP16), (512, 1, BF16)])
@pytest.mark.parametrize("n,m", [(1, 1), (2, 1), (70, 1), (70, 6), (3000, 1), (2000, 11)])
def test_infinite_values_stay_infinities(n, m, d, group, dt):
    """An infinity among the values that a row sees gives that infinity, in whichever token
    and whatever its weight; two of both signs give NaN, and a NaN itself."""
    fa = fa_mod()
    scale = d ** -0.5
    for at in sorted({0, 1 % n, n // 2, n - m}):
        c = Cache([n], 2, d, 16, False, dt)
        k, v = randn(n, 2, d, seed=1, dt=dt), randn(n, 2, d, seed=2, dt=dt)
        q = randn(m, 2 * group, d, seed=3, dt=dt)
        v[at, :, 5], v[at, :, d - 1] = math.inf, -math.inf
        v[at, :, 40] = math.inf
        v[(at + 1) % n, :, 40] = -math.inf if n > 1 and at + 1 <= n - m else math.inf
        v[at, :, 70] = NAN
        fa.fa_kv_append(None, k, v, c.k, c.v, i32([0, n]), i32([n]), c.table)
        rows = [(c.rows(c.k, 0, n), c.rows(c.v, 0, n))]
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, m]), i32([n]), c.table, m, causal=True, scale=scale)
        status_ok(fa)
        dims = {5: math.inf, d - 1: -math.inf, 40: NAN if n > 1 and at + 1 <= n - m else math.inf, 70: NAN}
        check_infinite(dims, o, lse, c, rows, q, [m], [n], True, scale)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("gap", [10.0, 25.0, 80.0, 200.0])
@pytest.mark.parametrize("n,at", [(200, 150), (200, 3), (5000, 20), (5000, 4000)])
def test_infinite_values_of_small_weight(n, at, gap, dt):
    """The token that holds the infinity lies far below the others' scores, before or after
    them, also where its weight is none in 32 bits."""
    fa, d = fa_mod(), 128
    c = Cache([n], 1, d, 64, False, dt)
    k, v = torch.zeros(n, 1, d), randn(n, 1, d, seed=2, dt=dt)
    k[at, 0, 0] = -gap / 4
    v[at, 0, 9] = -math.inf
    fa.fa_kv_append(None, k.to(dt).cuda(), v, c.k, c.v, i32([0, n]), i32([n]), c.table)
    rows = [(c.rows(c.k, 0, n), c.rows(c.v, 0, n))]
    q = torch.zeros(1, 4, d, dtype=dt, device="cuda")
    q[..., 0] = 4.0
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1]), i32([n]), c.table, 1, scale=1.0)
    status_ok(fa)
    check_infinite({9: -math.inf}, o, lse, c, rows, q, [1], [n], False, 1.0)


def test_infinite_values_in_some_sequences_of_a_batch():
    """Sequences with an infinity beside others, several per CTA and cut over several CTAs:
    the others come out as without them."""
    fa, d, Hq, Hkv = fa_mod(), 128, 8, 2
    lens = [(53 * b) % 300 + 1 for b in range(150)] + [4000, 2500, 4000]
    c = Cache(lens, Hkv, d, 16, False, BF16)
    k, v = randn(sum(lens), Hkv, d, seed=1), randn(sum(lens), Hkv, d, seed=2)
    cu, one, sk = cu_of(lens), cu_of([1] * len(lens)), i32(lens)
    q = randn(len(lens), Hq, d, seed=3)
    fa.fa_kv_append(None, k, v, c.k, c.v, cu, sk, c.table)
    clean = [t.clone() for t in fa.fa_fwd_paged(q, c.k, c.v, one, sk, c.table, 1)]
    hit = list(range(0, 150, 7)) + [151]
    at = torch.tensor([cu[b].item() + lens[b] // 3 for b in hit], device="cuda")
    v[at, 1, 17] = math.inf
    fa.fa_kv_append(None, k, v, c.k, c.v, cu, sk, c.table)
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, one, sk, c.table, 1)
    status_ok(fa)
    want = clean[0].clone()
    want[torch.tensor(hit, device="cuda"), 4:, 17] = math.inf
    assert torch.equal(o, want) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("d,group", [(128, 4), (192, 1), (256, 3), (512, 2)])
def test_int4_values_that_round_to_an_infinity(d, group):
    """fp16 groups whose scale and zero are finite and whose highest code stands for more
    than the type holds: infinite as the read-back has it, for the rows that see the token."""
    fa, n, m, dt = fa_mod(), 70, 4, FP16
    for at in (69, 67, 10):
        c = Cache([n], 1, d, 16, True, dt)
        k, v = randn(n, 1, d, seed=1, dt=dt), randn(n, 1, d, seed=2, dt=dt)
        v[at, 0, :32] = torch.linspace(-1, 1, 32, device="cuda") * torch.finfo(dt).max
        q = randn(m, group, d, seed=3, dt=dt)
        fa.fa_kv_append(None, k, v, c.k, c.v, i32([0, n]), i32([n]), c.table)
        rows = [(c.rows(c.k, 0, n), c.rows(c.v, 0, n))]
        assert rows[0][1].abs().max() == 65536                  # 8736 * 15 - 65504
        _, back = fa.fa_kv_gather(c.k, c.v, i32([0, n]), c.table, n, dt)
        dims = back[at, 0].isinf().nonzero()[:, 0].tolist()
        assert dims and max(dims) == 31
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, m]), i32([n]), c.table, m, causal=True)
        status_ok(fa)
        first = max(0, at - (n - m))
        if first:
            clean = [(rows[0][0][: n - m + first], rows[0][1][: n - m + first])]
            check_paged(c, clean, q[:first], [first], [n - m + first], True, d ** -0.5, o[:first], lse[:, :first])
        seen = o[first:].float()
        assert (seen[..., dims] == math.inf).all() and lse.isfinite().all()
        other = [i for i in range(d) if i not in dims]
        assert seen[..., other].isfinite().all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_int4_codes_of_the_widest_groups(dt, inter):
    """Groups whose values lie further apart than the largest number of 32 bits, as values and
    as turned keys: the codes of the definition."""
    fa, d, n = fa_mod(), 128, 12
    big = torch.finfo(dt).max
    x = torch.zeros(n, 2, d)
    x[0, 0] = big * torch.linspace(-1, 1, 32).repeat(4)
    x[0, 1] = big * torch.linspace(1, -1, 32).repeat(4)
    x[1, 0, :96] = torch.tensor([-0.9, 0.9, 0.3]).repeat(32) * big
    x[1, 1] = big * torch.cat([torch.linspace(-1, 1, 31), torch.zeros(1)]).repeat(4)
    x[2] = big * (torch.arange(d) % 2 * 2 - 1)
    g = torch.Generator().manual_seed(3)
    x[3:] = big * (2 * torch.rand(n - 3, 2, d, generator=g) - 1)
    x[9:] *= 0.7                                             # turned pairs stay within the type
    x = x.to(dt).cuda()
    assert x.isfinite().all()
    freq = (3.0 ** (-torch.arange(0, 64, 2).double() / 64)).float().cuda()
    c = Cache([n], 2, d, 16, True, dt)
    fa.fa_kv_append(None, x, x, c.k, c.v, i32([0, n]), i32([n]), c.table, inv_freq=freq, interleaved=inter)
    status_ok(fa)
    for pool, ref in ((c.v, held(x.double(), dt)), (c.k, held(turn(x, torch.arange(n, device="cuda"), freq, inter), dt))):
        assert torch.equal(c.rows(pool, 0, n).nan_to_num(nan=1e39), ref.nan_to_num(nan=1e39))
        assert ref[0].isfinite().all() and ref[9:].isfinite().all()


@pytest.mark.parametrize("group", [1, 8, 20])
@pytest.mark.parametrize("eq,ek,scale", [(118, -114, 0.088), (118, -20, 2.0 ** -103), (100, -105, 2.0), (50, -56, 16.0),
                                         (53, -62, 4.0), (44, -60, 1024.0),
                                         (0, 0, 0.088)])
def test_int4_queries_of_large_magnitude(eq, ek, scale, group):
    """bf16 queries as large as the calls over a 4-bit pool take them, beside rows of ordinary
    ones."""
    fa, d, n, dt = fa_mod(), 128, 300, BF16
    c = Cache([n], 1, d, 32, True, dt)
    k, v = randn(n, 1, d, seed=1).float() * 2.0 ** ek, randn(n, 1, d, seed=2)
    fa.fa_kv_append(None, k.to(dt), v, c.k, c.v, i32([0, n]), i32([n]), c.table)
    rows = [(c.rows(c.k, 0, n), c.rows(c.v, 0, n))]
    q = randn(1, group, d, seed=3).float().clamp(-1.9, 1.9)
    q[:, ::2] *= 2.0 ** eq
    q = q.to(dt)
    assert q.isfinite().all()
    o, lse = fa.fa_fwd_paged(q, c.k, c.v, i32([0, 1]), i32([n]), c.table, 1, scale=scale)
    status_ok(fa)
    check_paged(c, rows, q, [1], [n], False, scale, o, lse)


def test_stream_arguments():
    """stream= takes what the library's other calls take: a torch stream, anything with a
    cuda_stream, a raw handle; 0 and 1 both name the default stream."""
    fa = fa_mod()
    c = Cache([500], 2, 128, 16, False, BF16)
    rows = c.fill([500], seed=1)
    q, cu, sk = randn(1, 8, 128, seed=2), i32([0, 1]), i32([500])
    want = fa.fa_fwd_paged(q, c.k, c.v, cu, sk, c.table, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Holder:
        cuda_stream = side.cuda_stream

    for s in (side, side.cuda_stream, Holder(), 0, 1, torch.cuda.default_stream()):
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu, sk, c.table, 1, stream=s)
        k, v = fa.fa_kv_gather(c.k, c.v, i32([0, 500]), c.table, 500, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(k.double(), rows[0][0]) and torch.equal(v.double(), rows[0][1])
        # what the call allocated belongs to the stream that it ran on
        on = 0 if s in (0, 1, torch.cuda.default_stream()) else side.cuda_stream
        with fa._on(c.k.device, s):
            assert torch.cuda.current_stream().cuda_stream == on
    status_ok(fa)


@pytest.mark.parametrize("int4", [False, True])
def test_cut_sequences_are_those_of_the_varlen_forward(int4):
    """More queries than max_seqlen_q: the first ones are taken as the sequence's queries, the
    causal mask at their bottom right, as fa_fwd_varlen takes them."""
    fa, dt = fa_mod(), BF16
    news, lens, d = [5, 2, 9], [50, 60, 300], 128
    c = Cache(lens, 2, d, 16, int4, dt)
    c.fill(lens, seed=1)
    q = randn(sum(news), 4, d, seed=2, dt=dt)
    cu, ck = cu_of(news), cu_of(lens)
    k, v = fa.fa_kv_gather(c.k, c.v, ck, c.table, sum(lens), dt)
    for most in (2, 4, 9):
        o, lse = fa.fa_fwd_paged(q, c.k, c.v, cu, i32(lens), c.table, most, causal=True)
        ro, rl = fa.fa_fwd_varlen(q, k, v, cu, ck, most, max(lens), causal=True)
        status_ok(fa)
        at = 0
        for m in news:
            r = slice(at, at + min(m, most))
            # the library's forward bound, on both sides; 4-bit keys are rounded by the read-back
            assert ((o[r].double() - ro[r].double()).abs() <= 2e-2 + 2 * half(dt) * ro[r].double().abs()).all()
            assert (lse[:, r] - rl[:, r]).abs().max() <= 2e-3 + (2e-2 if int4 else 0)
            at += m
