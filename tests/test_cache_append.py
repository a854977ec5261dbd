"""sel_cache_append: rows and queries rotated and put into the cache.

What is expected is formed in numpy from the definition, twice.  In 32 bits with each product and sum rounded once: the
cache and the queries have to have those bits.  In 64 bits: the fp32 value is off by 2^-24 of each product and of the sum
at most, 2^-23 (|u cos| + |v sin|) in all; its rounding to bf16 is off by 2^-8 of the value.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_cache import EALIGN, EINVAL, EUNSUP, FAKE, GROUP, lib, quantise64, struct  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32


def turned(x, at, table, first, interleaved, dtype):
    """Rows x [tokens, .., d] (numpy) rotated in `dtype`; at: positions, negative for those that stay."""
    x = np.array(x, dtype=dtype)
    rot = table.shape[1]
    half = rot // 2
    j = np.arange(half)
    u_at, v_at = (first + 2 * j, first + 2 * j + 1) if interleaved else (first + j, first + half + j)
    for t, p in enumerate(at):
        if p < 0 or p >= table.shape[0]:
            continue
        c, s = table[p, :half].astype(dtype), table[p, half:].astype(dtype)
        u, v = x[t][..., u_at].copy(), x[t][..., v_at].copy()
        x[t][..., u_at] = u * c - v * s
        x[t][..., v_at] = v * c + u * s
    return x


def rotation(n, rot, seed=0):
    g = np.random.default_rng(seed)
    angle = np.arange(n)[:, None] * (10000.0 ** (-np.arange(rot // 2) * 2.0 / rot))[None] + g.random()
    return np.concatenate((np.cos(angle), np.sin(angle)), axis=1).astype(np.float32)


CASES = [
    # tokens, b, d, rot, first, h, x, q, cache, page size, index type
    (1, 1, 128, 128, 0, 0, BF16, None, "bf16", 16, torch.int32),
    (1, 1, 16, 16, 0, 1, BF16, BF16, "fp8", 1, torch.int64),
    (37, 1, 512, 64, 448, 3, BF16, BF16, "fp8", 24, torch.int64),
    (36, 4, 512, 64, 448, 64, F32, BF16, "bf16", 7, torch.int32),
    (130, 2, 80, 32, 8, 5, BF16, F32, "fp8", 7, torch.int32),      # a run of 80 only, rotated in its middle
    (66, 3, 272, 160, 64, 2, F32, F32, "fp8", 16, torch.int64),    # a rotated run across three runs of 128
    (300, 1, 192, 192, 0, 24, F32, F32, "bf16", 5, torch.int32),
    (129, 3, 136, 48, 88, 7, BF16, BF16, "bf16", 32, torch.int64),
    (20, 20, 576, 64, 512, 16, BF16, BF16, "fp8", 16, torch.int32),  # wider than the attention takes
    (513, 1, 64, 32, 0, 0, BF16, None, "fp8", 16, torch.int32),
]


def check_queries(got, q, at, table, first, interleaved):
    want32 = torch.from_numpy(turned(q.float().cpu().numpy(), at, table, first, interleaved, np.float32)).to(BF16)
    assert torch.equal(got.cpu().view(torch.int16), want32.view(torch.int16))
    q64 = q.double().cpu().numpy()
    ref = turned(q64, at, table, first, interleaved, np.float64)
    size = turned(np.abs(q64), at, np.abs(table) * np.r_[np.ones(table.shape[1] // 2), -np.ones(table.shape[1] // 2)],
                  first, interleaved, np.float64)  # |u c| + |v s| of the first of a pair
    other = turned(np.abs(q64), at, np.abs(table), first, interleaved, np.float64)  # |v c| + |u s| of the second
    tol = 2.0 ** -23 * (np.maximum(np.abs(size), np.abs(other))) + 2.0 ** -8 * np.abs(ref) + 1e-37
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol * (1 + 2.0 ** -7)).all()  # (bf16 of the rounded value)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_appended_rows(case, interleaved):
    import gather_radix_select_gb300 as sel
    tokens, b, d, rot, first, h, xt, qt, kind, ps, itype = case
    g = torch.Generator().manual_seed(tokens + d)
    per, known = tokens // b, 4 * (tokens // b) + 9
    mp = -(-known // ps)
    pages = b * mp + 2
    table = torch.randperm(pages, generator=g)[: b * mp].to(torch.int32).view(b, mp)
    positions = torch.stack([torch.randperm(known, generator=g)[:per] for _ in range(b)]).to(itype)
    if per > 4:
        positions[:, 1::5] = -1 - (positions[:, 1::5] % 3)  # padding
    x = (torch.randn((tokens, d), generator=g) * torch.exp(2 * torch.randn((tokens, 1), generator=g))).to(xt)
    q = None if qt is None else torch.randn((tokens, h, d), generator=g).to(qt)
    angles = rotation(known, rot)
    before = torch.randint(0, 120, (pages, ps, d), generator=g, dtype=torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = before.to(BF16).cuda() if kind == "bf16" else before.cuda().view(torch.float8_e4m3fn)
    runs = -(-d // GROUP)
    scales = None if kind == "bf16" else torch.full((pages, ps, runs), 3.0, device="cuda")
    got = sel.cache_append(x.cuda(), cache, table.cuda(), positions.flatten().cuda(), torch.from_numpy(angles).cuda(),
                           scales=scales, first=first, interleaved=interleaved, q=None if q is None else q.cuda(),
                           err_flag=err)
    at = positions.flatten().tolist()
    rows = turned(x.float().numpy(), at, angles, first, interleaved, np.float32)
    live = [t for t in range(tokens) if at[t] >= 0]
    to = torch.tensor([int(table[t // per, at[t] // ps]) * ps + at[t] % ps for t in live], dtype=torch.long)
    if kind == "bf16":
        want = before.to(BF16).view(-1, d)
        want[to] = torch.from_numpy(rows[live]).to(BF16)
        assert torch.equal(cache.cpu().view(-1, d).view(torch.int16), want.view(torch.int16))
    else:
        held, s = quantise64(rows[live].astype(np.float64))
        want = before.view(torch.float8_e4m3fn).double().view(-1, d)
        want[to] = torch.from_numpy(held)
        want_s = torch.full((pages * ps, runs), 3.0, dtype=torch.float64)
        want_s[to] = torch.from_numpy(s)
        assert torch.equal(cache.cpu().double().view(-1, d), want)
        assert torch.equal(scales.cpu().double().view(-1, runs), want_s)
    if q is None:
        assert got is None
    else:
        check_queries(got, q, at, angles, first, interleaved)
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
def test_queries_rotated_where_they_are(interleaved):
    import gather_radix_select_gb300 as sel
    tokens, h, d, rot = 70, 9, 144, 48
    g = torch.Generator().manual_seed(3)
    q = torch.randn((tokens, h, d), generator=g).to(BF16).cuda()
    was = q.clone()
    cache = torch.zeros((10, 8, d), dtype=BF16, device="cuda")
    at = torch.arange(tokens, dtype=torch.int32)
    at[5] = -1
    angles = rotation(80, rot)
    got = sel.cache_append(torch.zeros((tokens, d), device="cuda"), cache,
                           torch.arange(10, dtype=torch.int32, device="cuda")[None], at.cuda(),
                           torch.from_numpy(angles).cuda(), first=40, interleaved=interleaved, q=q, q_out=q)
    assert got is q
    check_queries(q, was, at.tolist(), angles, 40, interleaved)


@pytest.mark.gpu
def test_strided_tensors_and_another_stream():
    # a fused projection's output holds queries and the key, pages of several layers interleave, the rotation is a slice
    import gather_radix_select_gb300 as sel
    tokens, h, d, rot, pages, ps = 24, 4, 192, 64, 6, 8
    g = torch.Generator().manual_seed(5)
    fused = torch.randn((tokens, h + 2, d), generator=g).to(BF16).cuda()
    whole = torch.zeros((pages, ps, 3, d), dtype=BF16, device="cuda")
    angles = rotation(60, rot)
    wide = torch.full((60, rot + 12), 9.0, device="cuda")
    wide[:, 4: 4 + rot] = torch.from_numpy(angles).cuda()
    table = torch.tensor([[5, 0, 3], [1, 4, 2]], dtype=torch.int32, device="cuda")
    at = torch.stack([torch.randperm(24, generator=g)[:12], torch.randperm(24, generator=g)[:12]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sel.cache_append(fused[:, h], whole[:, :, 1], table, at.flatten().cuda(), wide[:, 4: 4 + rot], q=fused[:, :h],
                           stream=side)
    torch.cuda.synchronize()
    check_queries(got, fused[:, :h], at.flatten().tolist(), angles, d - rot, False)
    rows = turned(fused[:, h].float().cpu().numpy(), at.flatten().tolist(), angles, d - rot, False, np.float32)
    want = torch.zeros((pages, ps, 3, d), dtype=BF16)
    for t in range(tokens):
        p = int(at.flatten()[t])
        want[int(table[t // 12, p // ps]), p % ps, 1] = torch.from_numpy(rows[t]).to(BF16)
    assert torch.equal(whole.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_positions_outside_are_reported_and_skipped(kind):
    import gather_radix_select_gb300 as sel
    d, rot, ps = 64, 32, 4
    x = torch.ones((5, d), device="cuda")
    q = torch.randn((5, 2, d), device="cuda").to(BF16)
    angles = rotation(12, rot)
    for bad, page, col in ((16, 1, 3), (1 << 40, 1, 3), (12, 1, 3), (5, -1, 1), (5, 4, 1), (5, -(1 << 31), 1)):
        table = torch.tensor([[0, 2, 3, 1]], dtype=torch.int32, device="cuda")
        table[0, col] = page
        cache = torch.zeros((4, ps, d), device="cuda").to(BF16 if kind == "bf16" else torch.float8_e4m3fn)
        scales = None if kind == "bf16" else torch.ones((4, ps, 1), device="cuda")
        at = torch.tensor([0, bad, -7, 1, 2], device="cuda")
        for table_rows in (12, 0):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            cache.view(torch.uint8).zero_()
            got = sel.cache_append(x, cache, table, at, torch.from_numpy(angles[:table_rows]).cuda(), scales=scales,
                                   q=q, err_flag=err)
            assert int(err.item()) == 1
            rows = cache.float().cpu().view(-1, d)
            assert rows[:3].abs().sum(dim=1).gt(0).tolist() == [table_rows > 0] * 3 and int((rows[3:] != 0).sum()) == 0
            check_queries(got, q, at.tolist(), angles[:table_rows], d - rot, False)


@pytest.mark.gpu
def test_infinities_and_nan():
    # what a rotation makes of them goes the way of what cache_write makes of them; other tokens are untouched
    import gather_radix_select_gb300 as sel
    d, rot = 128, 64
    x = torch.randn((4, d))
    x[1, 70] = float("inf")
    x[2, 100] = float("nan")
    x[3, 64:128] = 3.4e38                      # the sum of two products passes fp32's range
    angles = np.full((4, rot), np.sqrt(0.5), dtype=np.float32)
    cache = torch.zeros((1, 4, d), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros((1, 4, 1), device="cuda")
    sel.cache_append(x.cuda(), cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.arange(4, device="cuda"),
                     torch.from_numpy(angles).cuda(), scales=scales)
    with np.errstate(all="ignore"):
        held, s = quantise64(turned(x.numpy(), range(4), angles, d - rot, False, np.float32))
    got = cache.cpu().double().numpy().reshape(4, d)
    assert np.array_equal(scales.cpu().double().numpy().reshape(4, 1), s)
    assert np.array_equal(np.isnan(got), np.isnan(held))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(held))


@pytest.mark.gpu
def test_captured_and_replayed():
    import gather_radix_select_gb300 as sel
    tokens, h, d, rot, ps = 6, 3, 128, 64, 4
    cache = torch.zeros((8, ps, d), dtype=BF16, device="cuda")
    table = torch.randperm(8, device="cuda").to(torch.int32).view(2, 4)
    angles = rotation(16, rot)
    on = torch.from_numpy(angles).cuda()
    x, q = torch.randn((tokens, d), device="cuda"), torch.randn((tokens, h, d), device="cuda")
    at = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32, device="cuda")

    def step():
        return sel.cache_append(x, cache, table, at, on, q=q)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in (3, 6, 9):
        x.normal_(), q.normal_(), at.add_(3)
        cache.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_queries(got, q, at.tolist(), angles, d - rot, False)
        rows = turned(x.cpu().numpy(), at.tolist(), angles, d - rot, False, np.float32)
        back = sel.cache_gather(cache, table, at.view(2, 3)).view(tokens, d)
        assert torch.equal(back.cpu(), torch.from_numpy(rows).to(BF16))
        assert int((cache.flatten(0, 1) != 0).any(dim=1).sum()) == tokens


# ------------------------------------------------------------------------------- refusals, without a GPU
def append(lib, c, **kw):  # noqa: F811
    from gather_radix_select_gb300 import _native
    a = dict(x=FAKE, x_dtype=1, tokens=4, x_stride=128, table=FAKE, b=2, mp=8, ts=8, pos=FAKE, pos_dtype=0, turn=True,
             angles=FAKE, known=16, stride=64, first=64, rot=64, neighbours=0, q=None, q_dtype=1, h=2, qrs=256, qhs=128,
             q_out=None)
    a.update(kw)
    turn = _native.SelRotation(a["angles"], a["known"], a["stride"], a["first"], a["rot"], a["neighbours"])
    return lib.sel_cache_append(a["x"], a["x_dtype"], a["tokens"], a["x_stride"], ctypes.byref(c) if c else None,
                                a["table"], a["b"], a["mp"], a["ts"], a["pos"], a["pos_dtype"],
                                ctypes.byref(turn) if a["turn"] else None, a["q"], a["q_dtype"], a["h"], a["qrs"],
                                a["qhs"], a["q_out"], None, None)


def test_append_refusals(lib):  # noqa: F811
    c = struct()
    assert append(lib, c, tokens=0) == 0
    assert append(lib, None) == EINVAL
    assert append(lib, struct(page_stride=0)) == EINVAL  # pages on top of one another
    for kw in (dict(tokens=-1), dict(tokens=3), dict(x_dtype=2), dict(pos_dtype=2), dict(x=None), dict(pos=None),
               dict(x_stride=64), dict(b=0), dict(mp=-1), dict(table=None), dict(ts=7), dict(turn=False),
               dict(angles=None), dict(known=-1), dict(stride=48), dict(first=-8), dict(first=72), dict(rot=0),
               dict(rot=144), dict(rot=-16), dict(first=1 << 62)):
        assert append(lib, c, **kw) == EINVAL, kw
    for kw in (dict(x=FAKE + 4), dict(x_stride=132), dict(pos=FAKE + 2), dict(table=FAKE + 2), dict(rot=40, stride=40),
               dict(first=4), dict(angles=FAKE + 4), dict(stride=66)):
        assert append(lib, c, **kw) == EALIGN, kw
    assert append(lib, c, tokens=1 << 40) == EUNSUP
    far = FAKE + (1 << 30)
    with_q = dict(q=FAKE, q_out=far)
    for kw in (dict(q_dtype=2), dict(h=0), dict(qrs=-8), dict(qhs=-8), dict(q_out=None)):
        assert append(lib, c, **(with_q | kw)) == EINVAL, kw
    for kw in (dict(q=FAKE + 2), dict(q_out=far + 8), dict(qrs=260), dict(qhs=132), dict(q_dtype=0, qhs=130)):
        assert append(lib, c, **(with_q | kw)) == EALIGN, kw
    for kw in (dict(h=1 << 40), dict(h=1 << 24, tokens=1 << 20), dict(qrs=1 << 60), dict(qhs=1 << 62)):
        assert append(lib, c, **(with_q | kw)) == EUNSUP, kw
    # queries over one another: elsewhere in one another's memory, or in place with other strides or another type
    for kw in (dict(q_out=FAKE + 16), dict(q=FAKE + 16, q_out=FAKE), dict(q_out=FAKE, qrs=264), dict(q_out=FAKE, qhs=136),
               dict(q_out=FAKE, q_dtype=0), dict(q_out=FAKE + 2 * (3 * 256 + 128 + 120))):
        assert append(lib, c, **(with_q | kw)) == EINVAL, kw


@pytest.mark.gpu
def test_binding_refusals():
    import gather_radix_select_gb300 as sel
    cache = torch.zeros((4, 8, 64), dtype=BF16, device="cuda")
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    x, at = torch.zeros((4, 64), device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    turn, q = torch.zeros((8, 32), device="cuda"), torch.zeros((4, 2, 64), dtype=BF16, device="cuda")
    for bad in (lambda: sel.cache_append(x.half(), cache, table, at, turn),
                lambda: sel.cache_append(x[:, :32], cache, table, at, turn),
                lambda: sel.cache_append(x, cache, table.long(), at, turn),
                lambda: sel.cache_append(x, cache, table, at[:3], turn),
                lambda: sel.cache_append(x, cache, table, at.float(), turn),
                lambda: sel.cache_append(x, cache, table, at, turn.double()),
                lambda: sel.cache_append(x, cache, table, at, turn.T),
                lambda: sel.cache_append(x, cache, table, at, turn.cpu()),
                lambda: sel.cache_append(x, cache, table, at, turn, q=q[:3]),
                lambda: sel.cache_append(x, cache, table, at, turn, q=q.half()),
                lambda: sel.cache_append(x, cache, table, at, turn, q_out=q),
                lambda: sel.cache_append(x, cache, table, at, turn, q=q, q_out=q[:, :1]),
                lambda: sel.cache_append(x, cache, table, at, turn, q=q, q_out=q.float())):
        with pytest.raises(ValueError):
            bad()
    for status, bad in ((EINVAL, lambda: sel.cache_append(x[:3], cache, table, at[:3], turn)),
                        (EINVAL, lambda: sel.cache_append(x, cache, table, at, turn, first=40)),
                        (EALIGN, lambda: sel.cache_append(x, cache, table, at, turn, first=4)),
                        (EALIGN, lambda: sel.cache_append(x, cache, table, at, turn[:, :24].contiguous()))):
        with pytest.raises(sel.SelError) as e:
            bad()
        assert e.value.status == status
    assert sel.cache_append(x[:0], cache, table, at[:0], turn) is None
    assert sel.cache_append(x[:0], cache, table, at[:0], turn, q=q[:0]).shape == (0, 2, 64)
