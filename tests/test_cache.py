"""The paged key cache (sel_cache_write, sel_cache_gather, sel_cache_attention) against plain 64-bit
computations written here from the definitions.

Tolerances of the attention.  Scores are sums of d exact bf16 products in fp32: an error of at most
e_z = 2^-20 * scale * max_k sum_i |q_i K_ki| (d <= 512 additions of unit roundoff 2^-24, twice that for how the
tensor cores add).  A weight is then off by a factor of at most exp(2 e_z) and its rounding to bf16 (2^-8), an
output by the same of A = sum_k p_k |v_k|, and by its own rounding to bf16:
    |out - ref| <= 2^-8 |ref| + (2^-8 + 4 e_z + 2^-16) A
where 2^-16 covers the fp32 sums over the positions.  The log-sum has no bf16 in it: 2 e_z + 2^-16 + 2^-22 |lse|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

GROUP = 128


# ------------------------------------------------------------------------------- plain computations
def quantise64(x):
    """(values the codes stand for, scales) of rows [.., d] in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    runs = -(-d // GROUP)
    held = np.zeros_like(x)
    scales = np.zeros((*x.shape[:-1], runs))
    for g in range(runs):
        part = x[..., g * GROUP: (g + 1) * GROUP]
        amax = np.where(np.isfinite(part), np.abs(part), 0.0).max(axis=-1)
        power = np.full(amax.shape, -126.0)
        # the smallest e with 448 * 2^e >= amax, found by trying: no logarithm, no rounding
        for e in range(-126, 128):
            power = np.where((power == -126.0) & (448.0 * 2.0 ** e >= amax) & ~(448.0 * 2.0 ** -126 >= amax), e, power) \
                if e > -126 else power
        s = 2.0 ** power
        y = np.clip(part / s[..., None], -448.0, 448.0)
        mag = np.maximum(np.abs(y), 2.0 ** -6)
        step = 2.0 ** (np.frexp(mag)[1].astype(np.float64) - 4)
        held[..., g * GROUP: (g + 1) * GROUP] = np.rint(y / step) * step
        scales[..., g] = s
    return held, scales


def rows64(cache, scales):
    """Every cache row in 64 bits, rounded to bf16 as the library reads it: [pages, page_size, d]."""
    c = cache.detach().cpu()
    if scales is None:
        return c.double()
    s = scales.detach().cpu().repeat_interleave(GROUP, dim=-1)[..., : c.shape[-1]]
    return (c.float() * s).to(torch.bfloat16).double()


def attend64(q, rows, table, per, end, idx, dv, scale):
    """(out, lse, A, e_z) in 64 bits; rows: [pages, page_size, d] in 64 bits."""
    r_n, h, d = q.shape
    pages, ps, _ = rows.shape
    table = table.cpu()
    cap = table.shape[1] * ps
    out = torch.zeros((r_n, h, dv), dtype=torch.float64)
    mean = torch.zeros((r_n, h, dv), dtype=torch.float64)
    lse = torch.full((r_n, h), -math.inf, dtype=torch.float64)
    ez = torch.zeros((r_n, h), dtype=torch.float64)
    for r in range(r_n):
        e = cap if end is None else min(max(int(end[r]), 0), cap)
        if idx is None:
            pos = list(range(e))
        else:
            pos = [p for p in idx[r].tolist() if 0 <= p < e]
        where = [(int(table[r // per, p // ps]), p % ps) for p in pos]
        where = [(a, b) for a, b in where if 0 <= a < pages]
        if not where:
            continue
        a = torch.tensor([w[0] for w in where])
        b = torch.tensor([w[1] for w in where])
        keys = rows[a, b]
        qr = q[r].detach().cpu().double()
        z = scale * (qr @ keys.T)
        ez[r] = 2.0 ** -20 * abs(scale) * (qr.abs() @ keys.abs().T).amax(dim=1)
        lse[r] = torch.logsumexp(z, dim=1)
        p = torch.exp(z - lse[r][:, None])
        out[r] = p @ keys[:, :dv]
        mean[r] = p @ keys[:, :dv].abs()
    return out, lse, mean, ez


def check_attention(got, lse, ref):
    out, l64, mean, ez = ref
    got, lse = got.detach().cpu().double(), lse.detach().cpu().double()
    nan = torch.isnan(out)
    assert torch.equal(torch.isnan(got), nan)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 4 * ez[..., None] + 2.0 ** -16) * mean + 1e-37
    assert bool(((got - out).abs() <= tol)[~nan].all()), float(((got - out).abs() / tol)[~nan].max())
    empty = torch.isinf(l64)
    assert torch.equal(torch.isinf(lse), empty)
    tol = 2 * ez + 2.0 ** -16 + 2.0 ** -22 * l64.abs()
    fine = ~empty & ~torch.isnan(l64)
    assert bool(((lse - l64).abs() <= tol)[fine].all()), float(((lse - l64).abs() / tol)[fine].max())
    assert bool((got[empty] == 0).all())


def make_cache(pages, ps, d, kind, seed, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((pages, ps, d), generator=g)
    if kind == "bf16":
        return x.to(torch.bfloat16).to(dev), None
    s = 2.0 ** torch.randint(-9, -6, (pages, ps, -(-d // GROUP)), generator=g).float()
    if kind == "fp8any":  # scales that are no powers of two
        s = s * (1 + torch.rand(s.shape, generator=g))
    codes = (x * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.to(dev), s.to(dev)


def make_table(b, max_pages, pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[: b * max_pages].to(torch.int32).view(b, max_pages).cuda()


def make_q(rows, h, d, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn((rows, h, d), generator=g)).to(torch.bfloat16).cuda()


# ------------------------------------------------------------------------------- writing
WRITES = [
    # (tokens, d, source, cache, page_size, slot type)
    (1, 128, "bf16", "fp8", 16, torch.int32),
    (37, 512, "bf16", "fp8", 24, torch.int64),
    (37, 512, "f32", "fp8", 1, torch.int32),
    (130, 80, "bf16", "fp8", 7, torch.int32),    # a run of 80 only
    (65, 272, "f32", "fp8", 16, torch.int64),    # runs of 128, 128 and 16
    (300, 24, "f32", "bf16", 5, torch.int32),
    (129, 136, "bf16", "bf16", 32, torch.int64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WRITES, ids=lambda c: "-".join(map(str, c)))
def test_written_rows(case):
    import gather_radix_select_gb300 as sel
    tokens, d, src, kind, ps, itype = case
    g = torch.Generator().manual_seed(tokens + d)
    x = torch.randn((tokens, d), generator=g) * torch.exp(2 * torch.randn((tokens, 1), generator=g))
    x = x.to(torch.bfloat16) if src == "bf16" else x
    pages = -(-tokens // ps) + 2
    slots = torch.randperm(pages * ps, generator=g)[:tokens].to(itype)
    slots[1::5] = -1 - (slots[1::5] % 3)  # padding tokens
    # the cache already holds something, which the untouched rows keep
    before = torch.randint(0, 120, (pages, ps, d), generator=g, dtype=torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    live = (slots >= 0).nonzero().flatten()
    at = slots[live].long()
    if kind == "bf16":
        cache = before.to(torch.bfloat16).cuda()
        sel.cache_write(x.cuda(), cache, slots.cuda(), err_flag=err)
        want = before.to(torch.bfloat16).view(-1, d)
        want[at] = x[live].to(torch.bfloat16)
        assert torch.equal(cache.cpu().view(-1, d).view(torch.int16), want.view(torch.int16))
    else:
        runs = -(-d // GROUP)
        cache = before.cuda().view(torch.float8_e4m3fn)
        scales = torch.full((pages, ps, runs), 3.0, device="cuda")
        sel.cache_write(x.cuda(), cache, slots.cuda(), scales=scales, err_flag=err)
        held, s = quantise64(x[live].double().numpy())
        want = before.view(torch.float8_e4m3fn).double().view(-1, d)
        want[at] = torch.from_numpy(held)
        want_s = torch.full((pages * ps, runs), 3.0, dtype=torch.float64)
        want_s[at] = torch.from_numpy(s)
        assert torch.equal(cache.cpu().double().view(-1, d), want)
        assert torch.equal(scales.cpu().double().view(-1, runs), want_s)
    assert int(err.item()) == 0


@pytest.mark.gpu
def test_written_extremes():
    # zeros, the largest and smallest fp32 magnitudes, amax exactly 448 * 2^k and one step above, ties
    # between codes, infinities and NaN
    import gather_radix_select_gb300 as sel
    rows = np.zeros((10, 128), dtype=np.float32)
    rows[1, :3] = [3.4028235e38, -1.0, 1e38]
    rows[2, :3] = [1e-45, -1e-45, 1e-44]
    rows[3, :4] = [448.0, 17.0, 19.0, -21.0]     # scale 1: ties to even codes
    rows[4, :2] = [np.nextafter(np.float32(448), np.float32(1000)), 1.0]
    rows[5, :3] = [448.0 * 2.0 ** -126, 2.0 ** -126, 2.0 ** -137]
    rows[6, :3] = [np.inf, 2.0, -3.0]
    rows[7, :3] = [np.nan, 5.0, -np.inf]
    rows[8, :] = np.inf
    rows[9, :] = np.linspace(-1, 1, 128, dtype=np.float32)
    cache = torch.zeros((10, 1, 128), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros((10, 1, 1), device="cuda")
    sel.cache_write(torch.from_numpy(rows).cuda(), cache, torch.arange(10, dtype=torch.int32, device="cuda"),
                    scales=scales)
    held, s = quantise64(rows)
    got = cache.cpu().double().numpy().reshape(10, 128)
    assert np.array_equal(scales.cpu().double().numpy().reshape(10, 1), s)
    assert np.array_equal(np.isnan(got), np.isnan(rows))
    assert np.array_equal(np.where(np.isnan(got), 0, got), np.where(np.isnan(held), 0, held))


@pytest.mark.gpu
def test_slots_past_the_cache_are_reported_and_skipped():
    import gather_radix_select_gb300 as sel
    cache = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sel.cache_write(x, cache, torch.tensor([8, 3, 1 << 40], device="cuda"), err_flag=err)
    want = torch.zeros(8, 64)
    want[3] = 1
    assert torch.equal(cache.cpu().float().view(8, 64), want)
    assert int(err.item()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_strided_cache_and_rows(kind):
    # pages of several layers interleaved, rows of a fused projection, a stream of its own
    import gather_radix_select_gb300 as sel
    pages, ps, layers, d, tokens = 6, 8, 3, 192, 20
    whole = torch.zeros((pages, ps, layers, d), device="cuda").to(
        torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    s_whole = None if kind == "bf16" else torch.zeros((pages, layers, ps, 2), device="cuda")
    cache = whole[:, :, 1]
    scales = None if s_whole is None else s_whole[:, 1]
    x = torch.randn((tokens, 5, d), device="cuda").to(torch.bfloat16)[:, 2]
    slots = torch.randperm(pages * ps, device="cuda")[:tokens]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sel.cache_write(x, cache, slots, scales=scales, stream=side)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    got = sel.cache_gather(cache, table, slots.view(1, -1), scales=scales, stream=side)
    torch.cuda.synchronize()
    if kind == "bf16":
        assert torch.equal(got[0], x)
    else:
        held, s = quantise64(x.double().cpu().numpy())
        want = torch.from_numpy(held * np.repeat(s, GROUP, axis=-1)[:, :d])
        assert torch.equal(got[0].double().cpu(), want)
    other = whole.view(torch.uint8) if kind == "fp8" else whole.view(torch.int16)
    assert int(other[:, :, 0].abs().sum() if kind == "bf16" else other[:, :, 0].sum()) == 0
    assert int(other[:, :, 2].abs().sum() if kind == "bf16" else other[:, :, 2].sum()) == 0


# ------------------------------------------------------------------------------- reading back
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8any"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 1, 3), (6, 3, 130, 80, 7, 9), (4, 1, 513, 512, 24, 5),
                                   (10, 2, 40, 272, 1, 50)], ids=str)
@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_gathered_rows(kind, shape, itype):
    import gather_radix_select_gb300 as sel
    rows, b, n, d, ps, mp = shape
    pages = b * mp + 2
    cache, scales = make_cache(pages, ps, d, kind, 1)
    table = make_table(b, mp, pages, 2)
    g = torch.Generator().manual_seed(3)
    idx = torch.randint(-1, mp * ps, (rows, n), generator=g).to(itype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sel.cache_gather(cache, table, idx.cuda(), scales=scales, err_flag=err)
    p = idx.long().clamp(min=0)
    seq = (torch.arange(rows) // (rows // b))[:, None]
    page = table.cpu().long()[seq, p // ps]
    assert torch.equal(got.cpu().double(), rows64(cache, scales)[page, p % ps])
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("b,per,n", [(7, 300, 3), (3, 1, 129), (1, 5000, 1), (2, 61, 67)])
def test_gathered_runs_cross_rows(kind, b, per, n):
    import gather_radix_select_gb300 as sel
    cache, scales = make_cache(40, 12, 48, kind, 37)
    table = make_table(b, 5, 40, 38)
    g = torch.Generator().manual_seed(39)
    wide = torch.randint(0, 60, (b * per, n + 3), generator=g, dtype=torch.int32)
    out = sel.cache_gather(cache, table, wide.cuda()[:, :n], scales=scales)
    idx = wide[:, :n].long()
    seq = (torch.arange(b * per) // per)[:, None].expand(-1, n)
    want = rows64(cache, scales)[table.cpu().long()[seq, idx // 12], idx % 12]
    assert torch.equal(out.cpu().double(), want)


@pytest.mark.gpu
def test_gathered_positions_outside_give_zero_rows_and_the_flag():
    import gather_radix_select_gb300 as sel
    cache, _ = make_cache(3, 4, 16, "bf16", 1)
    for bad_idx, bad_page in ((8, 1), (1 << 40, 1), (5, -1), (5, 3)):
        table = torch.tensor([[0, bad_page]], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = sel.cache_gather(cache, table, torch.tensor([[2, bad_idx]], device="cuda"), err_flag=err)
        assert torch.equal(got[0, 0], cache[0, 2]) and int(got[0, 1].abs().sum()) == 0
        assert int(err.item()) == 1


# ------------------------------------------------------------------------------- attention
ATTENDS = [
    # (b, rows a sequence, h, d, dv, page_size, max_pages)
    (1, 1, 1, 16, 8, 1, 1),         # one position
    (1, 1, 64, 128, 128, 16, 9),    # one token, a page that ends inside a tile
    (3, 1, 5, 80, 40, 7, 20),
    (2, 1, 128, 512, 512, 32, 17),  # more heads than one tile takes
    (2, 1, 96, 64, 64, 16, 40),
    (2, 3, 64, 512, 512, 24, 12),
    (1, 150, 16, 128, 128, 16, 11), # a chunk whose last tile of rows is partial
    (3, 33, 24, 192, 128, 100, 3),
    (2, 70, 8, 272, 272, 1, 200),
    (2, 9, 32, 384, 256, 48, 6),
    (1, 40, 1, 320, 320, 16, 20),
    (1, 20, 48, 256, 256, 8, 70),
    (1, 2, 200, 96, 96, 16, 10),
]


def causal_ends(b, per, cap, seed):
    g = torch.Generator().manual_seed(seed)
    ends = []
    for s in range(b):
        ctx = max(per, cap - int(torch.randint(0, max(1, cap // 3), (1,), generator=g)))
        ends += [min(cap, ctx - per + i + 1) for i in range(per)]
    return torch.tensor(ends, dtype=torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8any"])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c)))
def test_attention_over_every_position(case, kind):
    import gather_radix_select_gb300 as sel
    b, per, h, d, dv, ps, mp = case
    pages = b * mp + 1
    cache, scales = make_cache(pages, ps, d, kind, 11)
    table = make_table(b, mp, pages, 12)
    q = make_q(b * per, h, d, 13)
    end = causal_ends(b, per, mp * ps, 14)
    if b * per > 2:
        end[b * per // 2] = 0  # a row that has no position
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv, return_lse=True)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, end, None, dv, 1 / math.sqrt(d)))
    again, _ = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [0, 1, 127, 128, 300])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_attention_at_selected_positions(kind, n, itype):
    import gather_radix_select_gb300 as sel
    b, per, h, d, ps, mp = 2, 5, 40, 512 if n != 300 else 144, 16, 30
    pages = b * mp
    cache, scales = make_cache(pages, ps, d, kind, 21)
    table = make_table(b, mp, pages, 22)
    q = make_q(b * per, h, d, 23)
    g = torch.Generator().manual_seed(24)
    idx = torch.randint(0, mp * ps, (b * per, n), generator=g).to(itype)
    idx[torch.rand(idx.shape, generator=g) < 0.2] = -1
    if n:
        idx[1, n // 2:] = -1
        idx[2] = -1          # nothing selected
        idx[3] = idx[3, 0]   # one position many times
    out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx.cuda(), return_lse=True, scale=0.07)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, None, idx, d, 0.07))
    end = torch.randint(-3, mp * ps + 9, (b * per,), generator=g, dtype=torch.int32)
    out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx.cuda(), end=end.cuda(), return_lse=True,
                                   scale=0.07)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, end, idx, d, 0.07))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 512])
@pytest.mark.parametrize("b,per", [(1, 1), (3, 1), (1, 7)])
def test_attention_over_long_contexts(b, per, d):
    # few rows over many positions: the positions are shared out over CTAs and joined
    import gather_radix_select_gb300 as sel
    h, ps, mp = 16, 64, 150
    pages = b * mp
    cache, scales = make_cache(pages, ps, d, "bf16", 31)
    table = make_table(b, mp, pages, 32)
    q = make_q(b * per, h, d, 33)
    for top in (mp * ps, 5000, 129, 1, 0):
        end = torch.full((b * per,), top, dtype=torch.int32)
        end[0] = max(0, top - 3)
        out, lse = sel.cache_attention(q, cache, table, end=end.cuda(), return_lse=True)
        check_attention(out, lse, attend64(q, rows64(cache, None), table, per, end, None, d, 1 / math.sqrt(d)))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("h,d,ends", [
    (64, 128, [0, 1, 130, 7000, 3]),          # most have next to nothing
    (96, 64, [6000, 0, 0, 5999]),             # two blocks of heads a row
    (8, 512, [5, 2000]),
    (40, 256, [0, 0, 0]),                     # nothing at all
    (16, 192, [128 * i for i in range(40)]),  # more rows than can have many parts
])
def test_unequal_contexts(h, d, ends, kind):
    import gather_radix_select_gb300 as sel
    b, ps = len(ends), 64
    mp = -(-max(max(ends), 1) // ps) + 9
    cache, scales = make_cache(300, ps, d, kind, 45)
    g = torch.Generator().manual_seed(46)
    table = torch.randint(0, 300, (b, mp), generator=g, dtype=torch.int32).cuda()  # (sequences may share pages)
    q = make_q(b, h, d, 47)
    end = torch.tensor(ends, dtype=torch.int32)
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), return_lse=True)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, 1, end, None, d, 1 / math.sqrt(d)))
    again, _ = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda())
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0.0, 30.0, -30.0])
def test_attention_when_the_maximum_moves(spread):
    # scores that climb (or fall) along the positions: the running maximum moves at every tile, or never
    import gather_radix_select_gb300 as sel
    h, d, ps, mp = 24, 128, 32, 24
    cache, _ = make_cache(mp, ps, d, "bf16", 41)
    q = make_q(2, h, d, 42)
    rise = torch.linspace(0, spread, mp * ps).view(mp, ps, 1)
    q[:, :, 0] = 4.0
    cache = cache.float().cpu()
    cache[:, :, :1] = rise
    cache = cache.to(torch.bfloat16).cuda()
    table = torch.arange(mp, dtype=torch.int32, device="cuda").view(1, mp)
    out, lse = sel.cache_attention(q, cache, table, return_lse=True, scale=0.25)
    check_attention(out, lse, attend64(q, rows64(cache, None), table, 2, None, None, d, 0.25))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 8.0])
def test_attention_scales(scale):
    import gather_radix_select_gb300 as sel
    cache, scales = make_cache(5, 50, 96, "fp8", 51)
    table = make_table(1, 5, 5, 52)
    q = make_q(3, 7, 96, 53)
    out, lse = sel.cache_attention(q, cache, table, scales=scales, return_lse=True, scale=scale)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, 3, None, None, 96, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_outside_the_mask_have_no_influence(kind, bad):
    # rows at or past a row's end, unselected rows and unused pages hold NaN or infinities; rows that do
    # attend to a NaN give NaN, the others of the same chunk do not notice
    import gather_radix_select_gb300 as sel
    if kind == "fp8" and not math.isnan(bad):
        pytest.skip("e4m3 has no infinity")
    b, per, h, d, ps, mp = 2, 12, 16, 256, 16, 20
    pages = b * mp + 3
    cache, scales = make_cache(pages, ps, d, kind, 61)
    table = make_table(b, mp, pages, 62)
    q = make_q(b * per, h, d, 63)
    end = torch.tensor([250 + i for i in range(per)] + [130 + i for i in range(per)], dtype=torch.int32)
    clean = attend64(q, rows64(cache, scales), table, per, end, None, d, 1 / 16)
    poisoned = cache.float()
    poisoned[int(table[0, 257 // ps]), 257 % ps, 200:] = bad  # rows 8.. of the first sequence see position 257
    used = table[0].tolist()[: -(-(250 + per) // ps)] + table[1].tolist()[: -(-(130 + per) // ps)]
    poisoned[[p for p in range(pages) if p not in used]] = bad
    poisoned[used[-1], (130 + per) % ps:] = bad
    poisoned = poisoned.to(cache.dtype)
    out, lse = sel.cache_attention(q, poisoned, table, scales=scales, end=end.cuda(), return_lse=True)
    seen = torch.tensor([e > 257 and r < per for r, e in enumerate(end.tolist())])
    check_attention(out[~seen], lse[~seen], tuple(t[~seen] for t in clean))
    assert not bool(torch.isfinite(out[seen].float()).all())
    # at selected positions: position 257 is not in the list
    g = torch.Generator().manual_seed(64)
    idx = torch.randint(0, 120, (b * per, 130), generator=g, dtype=torch.int32)
    out, lse = sel.cache_attention(q, poisoned, table, scales=scales, idx=idx.cuda(), return_lse=True)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, None, idx, d, 1 / 16))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("h,d,dv", [(24, 192, 128), (24, 192, 192), (16, 128, 128), (16, 320, 128), (40, 384, 384),
                                    (16, 512, 256), (64, 512, 512)])
def test_a_row_that_is_not_finite_stays_with_the_rows_that_see_it(h, d, dv, kind):
    # every layout of the kernel: the NaN lies in the third tile, in the value and past it
    import gather_radix_select_gb300 as sel
    per, ps, mp, at = 12, 16, 20, 295
    cache, scales = make_cache(mp, ps, d, kind, 65)
    table = make_table(1, mp, mp, 66)
    q = make_q(per, h, d, 67)
    end = torch.tensor([290 + i for i in range(per)], dtype=torch.int32)
    clean = attend64(q, rows64(cache, scales), table, per, end, None, dv, 1 / 16)
    for first in (dv - 8, 0, d - 1):
        poisoned = cache.float()
        poisoned[int(table[0, at // ps]), at % ps, first:] = math.nan
        out, lse = sel.cache_attention(q, poisoned.to(cache.dtype), table, scales=scales, end=end.cuda(), dv=dv,
                                       scale=1 / 16, return_lse=True)
        seen = end > at
        check_attention(out[~seen], lse[~seen], tuple(t[~seen] for t in clean))
        assert bool(torch.isnan(out[seen].float()).all()) and bool(torch.isnan(lse[seen]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,where", [(1, 0), (300, 299), (300, 0), (129, 128)])
def test_an_entry_outside_the_cache_is_flagged_wherever_it_is_in_the_list(n, where):
    import gather_radix_select_gb300 as sel
    cache, _ = make_cache(20, 16, 64, "bf16", 73)
    table = make_table(1, 20, 20, 74)
    q = make_q(2, 4, 64, 75)
    g = torch.Generator().manual_seed(76)
    idx = torch.randint(0, 320, (2, n), generator=g)
    for entry, flag in ((320, 1), (-7, 0), (2 ** 31, 1), (2 ** 62, 1), (-2 ** 62, 0)):
        idx[1, where] = entry
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, idx=idx.cuda(), return_lse=True, err_flag=err)
        check_attention(out, lse, attend64(q, rows64(cache, None), table, 2, None, idx, 64, 1 / 8))
        assert int(err.item()) == flag


@pytest.mark.gpu
def test_positions_outside_the_cache_are_left_out_and_flagged():
    import gather_radix_select_gb300 as sel
    cache, _ = make_cache(4, 8, 64, "bf16", 71)
    q = make_q(2, 4, 64, 72)
    for entry in (-1, 4, 1 << 30):
        table = torch.tensor([[0, entry, 2]], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, return_lse=True, err_flag=err)
        check_attention(out, lse, attend64(q, rows64(cache, None), table, 2, None, None, 64, 1 / 8))
        assert int(err.item()) == 1
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    idx = torch.tensor([[3, 24, 1 << 40, 7], [-5, 23, 1, -1]], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sel.cache_attention(q, cache, table, idx=idx, return_lse=True, err_flag=err)
    check_attention(out, lse, attend64(q, rows64(cache, None), table, 2, None, idx, 64, 1 / 8))
    assert int(err.item()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_offsets_past_32_bits_strides_and_a_side_stream(kind):
    # the last page starts past 2^32 elements; queries are a slice of a fused projection
    import gather_radix_select_gb300 as sel
    d, ps, pages, h = 128, 16, 3, 8
    stride = (1 << 31) + 4096
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    whole = torch.empty(2 * stride + ps * d, dtype=torch.uint8 if kind == "fp8" else torch.bfloat16, device="cuda")
    cache = whole.view(dtype).as_strided((pages, ps, d), (stride, d, 1))
    small, scales = make_cache(pages, ps, d, kind, 81)
    for p in range(pages):
        whole[p * stride: p * stride + ps * d] = small[p].flatten().view(whole.dtype)
    fused = make_q(4, 3 * h, d, 82)
    q = fused[:, h: 2 * h]
    table = torch.tensor([[2, 0, 1], [1, 2, 0]], dtype=torch.int32, device="cuda")
    end = torch.tensor([40, 48, 17, 0], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end, return_lse=True, stream=side)
    got = sel.cache_gather(cache, table, torch.tensor([[0, 47], [16, 3]], device="cuda"), scales=scales, stream=side)
    torch.cuda.synchronize()
    check_attention(out, lse, attend64(q, rows64(small, scales), table, 2, end.cpu(), None, d, 1 / math.sqrt(d)))
    r = rows64(small, scales)
    assert torch.equal(got.cpu().double(), torch.stack([torch.stack([r[2, 0], r[1, 15]]),
                                                        torch.stack([r[2, 0], r[1, 3]])]))


@pytest.mark.gpu
@pytest.mark.parametrize("per", [1, 6])
def test_captured_in_a_graph(per):
    import gather_radix_select_gb300 as sel
    b, h, d, ps, mp = 2, 64, 128, 16, 60
    pages = b * mp
    cache, scales = make_cache(pages, ps, d, "fp8", 91)
    table = make_table(b, mp, pages, 92)
    q = make_q(b * per, h, d, 93)
    x = torch.randn((b * per, d), device="cuda").to(torch.bfloat16)
    end = torch.full((b * per,), mp * ps, dtype=torch.int32, device="cuda")
    slots = (table[:, 3].long() * ps).repeat_interleave(per) + torch.arange(per, device="cuda").repeat(b)

    def step():
        sel.cache_write(x, cache, slots, scales=scales)
        return sel.cache_attention(q, cache, table, scales=scales, end=end, return_lse=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for k in range(2):
        x.copy_(torch.randn((b * per, d), device="cuda") * (k + 1))
        end.fill_(700 - 100 * k)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, end.cpu(), None, d,
                                           1 / math.sqrt(d)))


@pytest.mark.gpu
def test_rows_are_written_selected_and_attended_to():
    # the chain of a step: new rows into the cache, positions chosen by score, attention there; equal to
    # gathering the selected rows and attending to them
    import gather_radix_select_gb300 as sel
    rows, h, d, ps, mp, k = 24, 16, 128, 16, 40, 96
    ctx = mp * ps
    g = torch.Generator().manual_seed(7)
    x = torch.randn((ctx, d), generator=g).to(torch.bfloat16).cuda()
    cache = torch.zeros((mp, ps, d), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros((mp, ps, 1), device="cuda")
    table = make_table(1, mp, mp, 8)
    pos = torch.arange(ctx, device="cuda")
    sel.cache_write(x, cache, table[0, pos // ps].long() * ps + pos % ps, scales=scales)
    score = torch.randn((rows, ctx), generator=g).to(torch.bfloat16).cuda()
    end = torch.arange(60, 60 + 20 * rows, 20, dtype=torch.int32, device="cuda")
    _, idx = sel.topk(score, k, end=end, sorted_index=True, return_value=False)
    q = make_q(rows, h, d, 9)
    out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx, end=end, return_lse=True)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, rows, end.cpu(), idx.cpu(), d,
                                       1 / math.sqrt(d)))
    held, s = quantise64(x.double().cpu().numpy())
    back = sel.cache_gather(cache, table, idx, scales=scales)
    want = torch.from_numpy(held * s)[idx.cpu().long().clamp(min=0)]
    assert torch.equal(back.double().cpu(), want)


# ------------------------------------------------------------------------------- refusals (no GPU needed)
FAKE = 0x10000  # never dereferenced: every call below is rejected on the host
EINVAL, EALIGN, EUNSUP = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from gather_radix_select_gb300 import _native
    return _native.load(build_if_missing=True)


def struct(**kw):
    from gather_radix_select_gb300 import _native
    c = _native.SelCache()
    base = dict(data=FAKE, scales=FAKE, dtype=2, pages=4, page_size=16, d=128, page_stride=16 * 128, row_stride=128,
                scale_page_stride=16, scale_row_stride=1)
    base.update(kw)
    for name, v in base.items():
        setattr(c, name, v)
    return c


BAD_CACHES = [
    (dict(dtype=0), EINVAL), (dict(pages=-1), EINVAL), (dict(page_size=0), EINVAL), (dict(d=0), EINVAL),
    (dict(data=None), EINVAL), (dict(row_stride=112), EINVAL), (dict(scales=None), EINVAL),
    (dict(scale_row_stride=0), EINVAL), (dict(dtype=1), EINVAL),  # bf16 with scales
    (dict(dtype=1, scales=None, d=12, row_stride=16), EALIGN), (dict(d=8), EALIGN), (dict(data=FAKE + 8), EALIGN),
    (dict(row_stride=136), EALIGN), (dict(page_stride=16 * 128 + 8), EALIGN), (dict(scales=FAKE + 2), EALIGN),
    (dict(pages=1 << 40, page_size=1 << 30), EUNSUP),
]


def call(lib, what, c, **kw):
    if what == "write":
        a = dict(x=FAKE, x_dtype=1, tokens=4, x_stride=128, slots=FAKE, slot_dtype=0)
        a.update(kw)
        return lib.sel_cache_write(a["x"], a["x_dtype"], a["tokens"], a["x_stride"], a["slots"], a["slot_dtype"],
                                   ctypes.byref(c) if c else None, None, None)
    if what == "gather":
        a = dict(table=FAKE, b=2, mp=8, ts=8, idx=FAKE, idx_dtype=0, rows=4, n=3, irs=3, out=FAKE)
        a.update(kw)
        return lib.sel_cache_gather(ctypes.byref(c) if c else None, a["table"], a["b"], a["mp"], a["ts"], a["idx"],
                                    a["idx_dtype"], a["rows"], a["n"], a["irs"], a["out"], None, None)
    a = dict(q=FAKE, rows=4, h=8, qrs=1024, qhs=128, table=FAKE, b=2, mp=8, ts=8, end=None, idx=None, idx_dtype=0,
             n=0, irs=0, dv=128, scale=0.1, out=FAKE, lse=None, ws=None, wsb=0)
    a.update(kw)
    return lib.sel_cache_attention(a["q"], a["rows"], a["h"], a["qrs"], a["qhs"], ctypes.byref(c) if c else None,
                                   a["table"], a["b"], a["mp"], a["ts"], a["end"], a["idx"], a["idx_dtype"], a["n"],
                                   a["irs"], a["dv"], a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("what", ["write", "gather", "attend"])
def test_bad_caches_are_refused(lib, what):
    for kw, want in BAD_CACHES:
        assert call(lib, what, struct(**kw)) == want, kw
    assert call(lib, what, None) == EINVAL


def test_write_refusals(lib):
    c = struct()
    assert call(lib, "write", c, tokens=0) == 0
    assert call(lib, "write", c, tokens=-1) == EINVAL
    assert call(lib, "write", c, x_dtype=2) == EINVAL
    assert call(lib, "write", c, slot_dtype=2) == EINVAL
    assert call(lib, "write", c, x=None) == EINVAL
    assert call(lib, "write", c, slots=None) == EINVAL
    assert call(lib, "write", c, x_stride=64) == EINVAL
    assert call(lib, "write", c, x=FAKE + 4) == EALIGN
    assert call(lib, "write", c, x_stride=132) == EALIGN
    assert call(lib, "write", c, slots=FAKE + 2) == EALIGN
    assert call(lib, "write", struct(page_stride=0)) == EINVAL  # pages on top of one another
    assert call(lib, "write", c, tokens=1 << 40) == EUNSUP


def test_gather_refusals(lib):
    c = struct()
    assert call(lib, "gather", c, rows=0) == 0 and call(lib, "gather", c, n=0) == 0
    assert call(lib, "gather", c, rows=5) == EINVAL
    assert call(lib, "gather", c, b=0) == EINVAL
    assert call(lib, "gather", c, n=-1) == EINVAL
    assert call(lib, "gather", c, idx_dtype=3) == EINVAL
    assert call(lib, "gather", c, idx=None) == EINVAL
    assert call(lib, "gather", c, out=None) == EINVAL
    assert call(lib, "gather", c, table=None) == EINVAL
    assert call(lib, "gather", c, ts=4) == EINVAL
    assert call(lib, "gather", c, irs=2) == EINVAL
    assert call(lib, "gather", c, out=FAKE + 8) == EALIGN
    assert call(lib, "gather", c, idx=FAKE + 2) == EALIGN
    assert call(lib, "gather", c, table=FAKE + 2) == EALIGN


def test_attention_refusals(lib):
    c = struct()
    assert call(lib, "attend", c, rows=0) == 0
    assert call(lib, "attend", c, rows=3) == EINVAL
    assert call(lib, "attend", c, rows=-2) == EINVAL
    assert call(lib, "attend", c, h=0) == EINVAL
    assert call(lib, "attend", c, dv=0) == EINVAL
    assert call(lib, "attend", c, dv=136) == EINVAL
    assert call(lib, "attend", c, scale=float("nan")) == EINVAL
    assert call(lib, "attend", c, scale=float("inf")) == EINVAL
    assert call(lib, "attend", c, q=None) == EINVAL
    assert call(lib, "attend", c, out=None) == EINVAL
    assert call(lib, "attend", c, table=None) == EINVAL
    assert call(lib, "attend", c, idx=FAKE, idx_dtype=5) == EINVAL
    assert call(lib, "attend", c, idx=FAKE, n=9, irs=8) == EINVAL
    assert call(lib, "attend", c, idx=FAKE, n=-1) == EINVAL
    assert call(lib, "attend", c, dv=12) == EALIGN
    assert call(lib, "attend", c, q=FAKE + 2) == EALIGN
    assert call(lib, "attend", c, qrs=1028) == EALIGN
    assert call(lib, "attend", c, qhs=132) == EALIGN
    assert call(lib, "attend", c, lse=FAKE + 1) == EALIGN
    assert call(lib, "attend", struct(d=528, row_stride=528, scale_row_stride=5, page_stride=528 * 16)) == EUNSUP
    assert call(lib, "attend", c, mp=1 << 29, ts=1 << 29) == EUNSUP
    assert call(lib, "attend", c, rows=1 << 30, h=4) == EUNSUP


def test_workspace_size_refuses_bad_arguments(lib):
    size = lib.sel_cache_attention_workspace_size
    assert size(0, 8, 128, 128, 1, 8, 16, 0, 0) == 0
    assert size(4, 8, 1024, 128, 1, 8, 16, 0, 0) == 0
    assert size(4, 8, 128, 136, 1, 8, 16, 0, 0) == 0
    assert size(4, 8, 128, 128, 3, 8, 16, 0, 0) == 0


def test_binding_refuses_before_the_library():
    # the Python checks that need no GPU
    import gather_radix_select_gb300 as sel
    with pytest.raises(ValueError):
        sel.cache_gather(torch.zeros((2, 4, 16), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32),
                         torch.zeros((1, 3), dtype=torch.int32))       # not on a GPU
    with pytest.raises(ValueError):
        sel.cache_write(torch.zeros((2, 16)), torch.zeros((2, 4, 16)), torch.zeros(2, dtype=torch.int32))  # fp32 cache


@pytest.mark.gpu
def test_binding_refusals():
    import gather_radix_select_gb300 as sel
    cache, scales = make_cache(4, 8, 64, "fp8", 1)
    plain, _ = make_cache(4, 8, 64, "bf16", 1)
    table = make_table(2, 2, 4, 2)
    q = make_q(4, 2, 64, 3)
    idx = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 64), device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: sel.cache_gather(cache, table, idx),                              # codes without scales
                lambda: sel.cache_gather(plain, table, idx, scales=scales),
                lambda: sel.cache_gather(cache, table, idx, scales=scales[:, :4]),
                lambda: sel.cache_gather(plain, table.long(), idx),
                lambda: sel.cache_gather(plain, table, idx.float()),
                lambda: sel.cache_gather(plain, table, idx, out=torch.empty((4, 3, 64), device="cuda")),
                lambda: sel.cache_gather(plain.transpose(1, 2), table, idx),
                lambda: sel.cache_write(x.half(), plain, slots),
                lambda: sel.cache_write(x[:, :32], plain, slots),
                lambda: sel.cache_write(x, plain, slots[:1]),
                lambda: sel.cache_attention(q.float(), plain, table),
                lambda: sel.cache_attention(q[:, :, :32], plain, table),
                lambda: sel.cache_attention(q, plain, table, idx=idx[:3]),
                lambda: sel.cache_attention(q, plain, table, end=torch.zeros(4, device="cuda")),
                lambda: sel.cache_attention(q, plain, table, out=torch.empty_like(q.float())),
                lambda: sel.cache_attention(q, plain, table, err_flag=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for status, bad in ((EINVAL, lambda: sel.cache_attention(q[:3], plain, table)),
                        (EALIGN, lambda: sel.cache_attention(q, plain, table, dv=20)),
                        (EINVAL, lambda: sel.cache_attention(q, plain, table, dv=72)),
                        (EINVAL, lambda: sel.cache_gather(plain, table, idx[:3]))):
        with pytest.raises(sel.SelError) as e:
            bad()
        assert e.value.status == status


def test_plain_quantiser_is_pinned():
    # hand-computed rows: scale 1 with ties to even, a subnormal code, the step above 448
    x = np.zeros((3, 128))
    x[0, :5] = [448, 17, 19, 2.0 ** -9, 2.0 ** -10]
    x[1, :2] = [449, 3]
    x[2, :1] = [0]
    held, s = quantise64(x)
    assert s[:, 0].tolist() == [1.0, 2.0, 2.0 ** -126]
    assert held[0, :5].tolist() == [448, 16, 20, 2.0 ** -9, 0]
    assert held[1, :2].tolist() == [224, 1.5]
