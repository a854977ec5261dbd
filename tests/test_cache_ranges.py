"""The attention whose positions are ranges: under a window with first tokens that stay visible (sel_cache_attention_window),
and behind a prefix that all sequences share (sel_cache_attention_shared), against 64 bits (tests/test_cache.py has the
computation and where its tolerances come from; here each row's positions are listed for it)."""
import ctypes
import math

import pytest
import torch

from tests.test_cache import (EALIGN, EINVAL, EUNSUP, FAKE, attend64, causal_ends, check_attention, lib,  # noqa: F401
                              make_cache, make_q, make_table, rows64, struct)


def seen_by_window(ends, cap, window, sinks):
    """The positions that each row sees."""
    out = []
    for e in ends.tolist():
        e = min(max(e, 0), cap)
        p = torch.arange(e)
        out.append(p[(p >= e - window) | (p < sinks)])
    return out


def check_window(case, kind, window, sinks, ends=None, seed=50, edit=None):
    import gather_radix_select_gb300 as sel
    b, per, h, d, dv, ps, mp = case
    pages = b * mp + 1
    cache, scales = make_cache(pages, ps, d, kind, seed)
    table = make_table(b, mp, pages, seed + 1)
    q = make_q(b * per, h, d, seed + 2)
    if ends is None:
        ends = causal_ends(b, per, mp * ps, seed + 3)
        if b * per > 2:
            ends[b * per // 2] = 0  # a row that has no position
    if edit:
        edit(cache, table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=ends.cuda(), dv=dv, return_lse=True, window=window,
                                   sinks=sinks, err_flag=err)
    seen = seen_by_window(ends, mp * ps, window, sinks)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, None, seen, dv, 1 / math.sqrt(d)))
    again, _ = sel.cache_attention(q, cache, table, scales=scales, end=ends.cuda(), dv=dv, window=window, sinks=sinks)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    return int(err.item())


# every layout of the kernel: chunks of 128 elements by 64 and by 128 columns, several rows a tile and heads of one row
# over several
WINDOWS = [
    (1, 1, 1, 16, 8, 1, 300),
    (1, 1, 64, 128, 128, 16, 40),
    (3, 1, 5, 80, 40, 7, 70),
    (2, 1, 128, 512, 512, 32, 17),
    (2, 3, 64, 512, 512, 24, 22),
    (1, 150, 16, 128, 128, 16, 31),
    (3, 33, 24, 192, 128, 100, 5),
    (2, 70, 8, 272, 272, 1, 400),
    (2, 9, 32, 384, 256, 48, 9),
    (1, 20, 48, 256, 256, 8, 70),
    (1, 40, 200, 96, 96, 16, 30),
]
WIDTHS = [(1, 0), (1, 3), (5, 130), (100, 1), (128, 4), (129, 0), (300, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8any"])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_windows(case, kind):
    for window, sinks in WIDTHS:
        assert check_window(case, kind, window, sinks) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("h,d", [(16, 128), (8, 512), (24, 192)])
def test_windows_of_unequal_rows(h, d, kind):
    # rows of a tile whose ends lie far apart: positions between their windows that no row sees, and rows that see only
    # first tokens, everything, or nothing
    case = (2, 12, h, d, d, 16, 60)
    g = torch.Generator().manual_seed(60)
    for window, sinks in ((1, 0), (7, 3), (64, 200), (200, 5), (900, 0), (4, 129)):
        ends = torch.randint(-5, 1000, (24,), generator=g, dtype=torch.int32)
        ends[3:6] = torch.tensor([0, 960, 1], dtype=torch.int32)
        ends[12:] = 0 if window == 64 else ends[12:]  # a sequence of padding alone
        assert check_window(case, kind, window, sinks, ends=ends) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h,d", [(64, 128), (16, 512), (96, 64)])
def test_long_contexts_under_a_window(h, d):
    # few rows: the window's tiles are shared out and joined
    for ends in ([9000, 3], [9600], [129] * 5, [1, 0, 5000, 9599]):
        for window, sinks in ((4096, 16), (1000, 0), (9500, 150)):
            assert check_window((len(ends), 1, h, d, d, 64, 150), "bf16", window, sinks,
                                ends=torch.tensor(ends, dtype=torch.int32)) == 0


# layouts as above; few rows over few tiles, some of them none
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("h,d,dv", [(7, 64, 64), (64, 128, 128), (100, 128, 96), (128, 192, 192), (33, 256, 256),
                                    (64, 320, 200), (64, 512, 512)])
def test_few_short_rows(h, d, dv, kind):
    ps, mp, window, sinks = 16, 80, 600, 10
    for b in (1, 2, 15, 16, 30, 60):
        ends = torch.tensor([(1280, 0, 1, 611, 130, 128, 257, 1000)[i % 8] - i // 8 for i in range(b)], dtype=torch.int32)
        assert check_window((b, 1, h, d, dv, ps, mp), kind, window, sinks, ends=ends) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rows_outside_a_window_have_no_influence(kind):
    # NaN and infinities in cache rows that some of a tile's rows see and others do not, and that none sees
    def spoil(cache, table):
        rows = cache.view(torch.int16 if kind == "bf16" else torch.uint8)
        bad = 0x7FC0 if kind == "bf16" else 0x7F
        for p in (2, 30, 31, 200, 400, 401, 500, 520):
            rows[int(table[0, p // 16]), p % 16, ::3] = bad

    case = (1, 8, 8, 192, 128, 16, 40)
    ends = torch.tensor([100, 233, 202, 232, 500, 520, 521, 640], dtype=torch.int32)
    for window, sinks in ((32, 0), (32, 2), (119, 3), (20, 31)):
        assert check_window(case, kind, window, sinks, ends=ends, edit=spoil) == 0


@pytest.mark.gpu
def test_pages_outside_the_window_are_not_looked_at():
    # freed pages of a sequence whose window has moved on; one inside it is left out and reported
    def freed(cache, table):
        table[0, 1:6] = -1

    case, end = (1, 1, 16, 128, 128, 16, 40), torch.tensor([500], dtype=torch.int32)
    assert check_window(case, "bf16", 300, 16, ends=end, edit=freed) == 0
    assert check_window(case, "bf16", 300, 17, ends=end, edit=freed) == 1
    assert check_window(case, "bf16", 404, 16, ends=end, edit=freed) == 0
    assert check_window(case, "bf16", 405, 16, ends=end, edit=freed) == 1


@pytest.mark.gpu
def test_a_window_that_holds_everything_is_plain_attention():
    import gather_radix_select_gb300 as sel
    cache, _ = make_cache(30, 16, 128, "bf16", 70)
    table = make_table(2, 10, 30, 71)
    q = make_q(6, 16, 128, 72)
    end = torch.tensor([160, 3, 0, 128, 129, 40], dtype=torch.int32, device="cuda")
    plain, lse = sel.cache_attention(q, cache, table, end=end, return_lse=True)
    for window, sinks in ((160, 0), (150, 10), (1, 159), (1 << 40, 0), (1, 1 << 40), ((1 << 63) - 1, (1 << 63) - 1)):
        got, l2 = sel.cache_attention(q, cache, table, end=end, return_lse=True, window=window, sinks=sinks)
        assert torch.equal(got.view(torch.int16), plain.view(torch.int16)) and torch.equal(l2, lse)
    got, _ = sel.cache_attention(q, cache, table, window=159)  # (without ends: the whole page table)
    seen = seen_by_window(torch.full((6,), 160), 160, 159, 0)
    ref = attend64(q, rows64(cache, None), table, 3, None, seen, 128, 1 / math.sqrt(128))
    check_attention(got, ref[1].float(), ref)


# ------------------------------------------------------------------------------- a shared prefix
def shared_tables(b, mp, common, pages, seed):
    """Page tables whose first `common` pages are the same."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    rest = ids[common: common + b * (mp - common)].view(b, mp - common)
    return torch.cat((ids[:common].expand(b, -1), rest), dim=1).contiguous().cuda()


def groups(rows, h, d, dv, b, mp, ps, shared):
    """Whether a call attends to the prefix once for all: it has scratch, and other scratch than a plain call."""
    from gather_radix_select_gb300 import _native
    lib = _native.load()  # noqa: F811
    return lib.sel_cache_attention_shared_workspace_size(rows, h, d, dv, b, mp, ps, shared) not in \
        (0, lib.sel_cache_attention_workspace_size(rows, h, d, dv, b, mp, ps, 0, 0))


def check_shared(case, kind, shared, ends, seed=80, edit=None, grouped=None):
    import gather_radix_select_gb300 as sel
    b, per, h, d, dv, ps, mp = case
    common = shared // ps
    pages = common + b * (mp - common) + 2
    cache, scales = make_cache(pages, ps, d, kind, seed)
    table = shared_tables(b, mp, common, pages, seed + 1)
    if shared % ps and common < mp:  # the page that ends within the prefix: every sequence's holds the same rows there
        whole = cache.view(torch.uint8 if kind != "bf16" else torch.int16)
        for s in range(1, b):
            whole[int(table[s, common]), : shared % ps] = whole[int(table[0, common]), : shared % ps]
            if scales is not None:
                scales[int(table[s, common]), : shared % ps] = scales[int(table[0, common]), : shared % ps]
    q = make_q(b * per, h, d, seed + 2)
    if edit:
        edit(cache, table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=ends.cuda(), dv=dv, return_lse=True, shared=shared,
                                   err_flag=err)
    if grouped is not None:
        assert groups(b * per, h, d, dv, b, mp, ps, shared) == grouped
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, ends, None, dv, 1 / math.sqrt(d)))
    again, _ = sel.cache_attention(q, cache, table, scales=scales, end=ends.cuda(), dv=dv, shared=shared)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    return int(err.item())


def shared_ends(b, per, shared, cap, seed):
    """Causal ends behind the prefix; among them a padding row and rows that end within or at the prefix."""
    g = torch.Generator().manual_seed(seed)
    ends = []
    for _ in range(b):
        most = int(torch.randint(shared + per, cap + 1, (1,), generator=g))
        ends += [most - per + i + 1 for i in range(per)]
    ends = torch.tensor(ends, dtype=torch.int32)
    ends[b * per // 2] = 0
    ends[b * per // 3] = max(1, shared // 2)
    ends[b * per // 4] = shared
    return ends


# (b, rows a sequence, h, d, dv, page size, pages), shared positions: both layouts of 128 elements and of 129 .. 192, the
# others by 64 columns; rows whose tiles are whole, or cut; more items than can be cut
SHARED = [
    ((40, 1, 8, 128, 128, 16, 50), 700),
    ((33, 1, 24, 64, 32, 16, 64), 960),
    ((40, 2, 12, 192, 128, 24, 40), 888),
    ((30, 1, 16, 512, 512, 32, 36), 1088),
    ((40, 3, 5, 320, 256, 7, 130), 850),
    ((50, 1, 1, 256, 136, 16, 70), 1000),
    ((60, 1, 20, 384, 384, 64, 14), 800),
    ((600, 1, 1, 128, 128, 16, 40), 600),
    ((560, 1, 2, 272, 272, 16, 40), 576),
    ((45, 1, 63, 80, 80, 1, 800), 780),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8any"])
@pytest.mark.parametrize("case,shared", SHARED, ids=str)
def test_a_shared_prefix(case, shared, kind):
    ends = shared_ends(case[0], case[1], shared, case[5] * case[6], 90)
    assert check_shared(case, kind, shared, ends, grouped=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_prefixes_that_are_read_by_every_sequence(kind):
    # one sequence, rows that fill a tile by themselves, prefixes too short to pay, prefixes of everything
    for case, shared in (((1, 4, 16, 128, 128, 16, 20), 200), ((3, 2, 64, 192, 128, 16, 20), 300),
                         ((4, 1, 16, 512, 512, 16, 3), 16), ((40, 1, 8, 128, 64, 16, 50), 1),
                         ((37, 1, 20, 384, 384, 64, 14), 800)):
        ends = shared_ends(case[0], case[1], shared, case[5] * case[6], 91)
        assert check_shared(case, kind, shared, ends, grouped=False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_nothing_behind_the_prefix(kind):
    case, cap = (40, 1, 8, 128, 128, 16, 50), 800
    for shared in (800, 5000, 1 << 40):
        ends = torch.arange(40, dtype=torch.int32) * 21 - 3  # (below 0 .. past the page table)
        import gather_radix_select_gb300 as sel
        b, per, h, d, dv, ps, mp = case
        cache, scales = make_cache(mp + 1, ps, d, kind, 100)
        table = make_table(1, mp, mp + 1, 101).expand(b, -1).contiguous()
        q = make_q(b, h, d, 102)
        out, lse = sel.cache_attention(q, cache, table, scales=scales, end=ends.cuda(), return_lse=True, shared=shared)
        ref = attend64(q, rows64(cache, scales), table, 1, ends.clamp(0, cap), None, dv, 1 / math.sqrt(d))
        check_attention(out, lse, ref)
        zeros = torch.zeros(b, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, scales=scales, end=zeros, return_lse=True, shared=shared)
        assert int((out != 0).sum()) == 0 and bool((lse == -math.inf).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rows_behind_the_prefix_are_their_sequences_own(kind):
    # NaN in one sequence's own rows, in rows of the prefix past some rows' ends, and past everyone's end
    ps, shared = 16, 704

    def spoil(cache, table):
        rows = cache.view(torch.int16 if kind == "bf16" else torch.uint8)
        bad = 0x7FC0 if kind == "bf16" else 0x7F
        for s, p in ((7, shared + 3), (7, shared + 20), (0, 350), (0, 690), (9, 799)):
            rows[int(table[s, p // ps]), p % ps, ::5] = bad

    ends = torch.full((40,), 760, dtype=torch.int32)
    ends[::3] = 340  # (they see none of the prefix's NaN)
    ends[7] = 710
    ends[9] = 351
    assert check_shared((40, 1, 8, 128, 128, ps, 50), kind, shared, ends, edit=spoil, grouped=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_page_tables_of_padding_sequences_are_not_read(kind):
    # sequences without a row that sees anything, the first of a tile's among them, whose page tables hold nothing; and
    # one whose row ends within the prefix, with pages for no more than that
    def lose(cache, table):
        table[[0, 1, 16, 32, 39]] = -1
        table[17, 10:] = -1

    ends = torch.full((40,), 780, dtype=torch.int32) - torch.arange(40, dtype=torch.int32)
    ends[[0, 1, 16, 32, 39]] = 0
    ends[17] = 160
    assert check_shared((40, 1, 8, 128, 128, 16, 50), kind, 704, ends, edit=lose, grouped=True) == 0


@pytest.mark.gpu
def test_a_page_outside_the_cache_in_the_prefix_is_reported():
    def lose(cache, table):
        table[:, 5] = 1 << 30

    ends = torch.full((40,), 780, dtype=torch.int32)
    assert check_shared((40, 1, 8, 128, 128, 16, 50), "bf16", 704, ends, edit=lose, grouped=True) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [40.0, -40.0])
def test_parts_of_very_different_size(spread):
    # a prefix whose scores lie far above, or below, those behind it: each part keeps its own reference
    import gather_radix_select_gb300 as sel
    b, h, d, ps, mp, shared = 40, 8, 128, 16, 50, 640
    cache, _ = make_cache(40 + b * 10 + 2, ps, d, "bf16", 110)
    table = shared_tables(b, mp, 40, cache.shape[0], 111)
    q = make_q(b, h, d, 112)
    q[:, :, 0] = 16.0
    cache[table[0, :40].long(), :, 0] = spread
    cache[table[:, 40:].long().flatten(), :, 0] = 0.0
    out, lse = sel.cache_attention(q, cache, table, return_lse=True, shared=shared)
    assert groups(b, h, d, d, b, mp, ps, shared)
    check_attention(out, lse, attend64(q, rows64(cache, None), table, 1, None, None, d, 1 / math.sqrt(d)))


# ------------------------------------------------------------------------------- both
@pytest.mark.gpu
@pytest.mark.parametrize("form", [{"window": 200, "sinks": 5}, {"shared": 640}], ids=["window", "shared"])
def test_captured_replayed_and_on_another_stream(form):
    import gather_radix_select_gb300 as sel
    b, h, d, ps, mp = 40, 8, 128, 16, 50
    cache, _ = make_cache(40 + b * 10 + 2, ps, d, "bf16", 120)
    table = shared_tables(b, mp, 40, cache.shape[0], 121)
    q = make_q(b, h, d, 122)
    end = torch.full((b,), 700, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = sel.cache_attention(q, cache, table, end=end, return_lse=True, stream=side, **form)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs whose scratch lies in one pool, replayed one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0][0].pool() if graphs else None):
            graphs.append((graph, *sel.cache_attention(q, cache, table, end=end, return_lse=True, **form)))
    for n in (700, 655, 799):
        end.fill_(n)
        want, l64 = sel.cache_attention(q, cache, table, end=end, return_lse=True, **form)
        for graph, got, l2 in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(l2, l64)
        if n == 700:
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, l64)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.03, -0.07, 0.0])
@pytest.mark.parametrize("form", [{"window": 150, "sinks": 20}, {"shared": 640}], ids=["window", "shared"])
def test_strided_queries_an_output_given_and_scales(form, scale):
    import gather_radix_select_gb300 as sel
    b, per, h, d, dv, ps, mp = 40, 2, 6, 144, 96, 16, 50
    cache, scales = make_cache(40 + b * 10 + 2, ps, d, "fp8", 150)
    table = shared_tables(b, mp + 3, 40, cache.shape[0] + 2000, 151) % cache.shape[0]
    table = table[:, :mp]  # (rows of the page table are strided too)
    fused = make_q(b * per, h + 3, d, 152)
    q = fused[:, 2: 2 + h]
    end = torch.tensor([mp * ps - 5 * i for i in range(b * per)], dtype=torch.int32)
    out = torch.full((b * per, h, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv, scale=scale, return_lse=True,
                                   out=out, **form)
    assert got is out
    seen = seen_by_window(end, mp * ps, form["window"], form["sinks"]) if "window" in form else None
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, per, None if seen else end, seen, dv, scale))


@pytest.mark.gpu
def test_rows_past_2_to_the_32_elements():
    # a cache of 8.6 GB: rows appended to its last pages and attended to there
    import gather_radix_select_gb300 as sel
    from tests.test_cache_append import rotation, turned
    d, pages, n = 512, (1 << 23) + 40, 40
    cache = torch.empty((pages, 1, d), dtype=torch.bfloat16, device="cuda")
    last = torch.arange(pages - n, pages, dtype=torch.int32, device="cuda")
    cache[last.long()] = 0
    table = last[None]
    angles = rotation(n, 64)
    x = torch.randn((n, d), device="cuda")
    sel.cache_append(x, cache, table, torch.arange(n, device="cuda"), torch.from_numpy(angles).cuda())
    want = torch.from_numpy(turned(x.cpu().numpy(), range(n), angles, d - 64, False, "float32")).to(torch.bfloat16)
    assert torch.equal(cache[last.long(), 0].cpu().view(torch.int16), want.view(torch.int16))
    q = make_q(1, 16, d, 160)
    out, lse = sel.cache_attention(q, cache, table, return_lse=True, window=30, sinks=3)
    rows = want.double()[:, None]
    here = torch.arange(n, dtype=torch.int32)[None]
    seen = seen_by_window(torch.tensor([n]), n, 30, 3)
    check_attention(out, lse, attend64(q, rows, here, 1, None, seen, d, 1 / math.sqrt(d)))


@pytest.fixture
def limit():
    from gather_radix_select_gb300 import _native
    yield _native.load().sel_cache_set_wait_limit
    _native.load().sel_cache_set_wait_limit(-1)


@pytest.mark.gpu
@pytest.mark.parametrize("h,d,dv", [(16, 128, 128), (40, 512, 512), (50, 192, 128), (24, 384, 256)])
@pytest.mark.parametrize("form", [{"window": 300, "sinks": 5}, {"shared": 512}], ids=["window", "shared"])
@pytest.mark.parametrize("b,kind", [(3, "bf16"), (40, "fp8"), (40, "bf16"), (530, "fp8")])
def test_ranges_under_short_limits(limit, h, d, dv, form, b, kind):
    # waits that give up anywhere, or nowhere: rows are right or NaN, and the next call is right
    import gather_radix_select_gb300 as sel
    from tests.test_cache_waits import ETIMEOUT, check_lost
    ps, mp = 16, 37
    h = 1 if b > 500 else h  # (more items than can be cut, and a prefix that pays)
    cache, scales = make_cache(32 + 5 * min(b, 40) + 2, ps, d, kind, 131)
    table = shared_tables(min(b, 40), mp, 32, cache.shape[0], 132).repeat(-(-b // 40), 1)[:b].contiguous()
    q = make_q(b, h, d, 133)
    end = torch.tensor([mp * ps - 3 * i % 80 for i in range(b)], dtype=torch.int32)
    seen = seen_by_window(end, mp * ps, form["window"], form["sinks"]) if "window" in form else None
    ref = attend64(q, rows64(cache, scales), table, 1, None if seen else end, seen, dv, 1 / math.sqrt(d))
    for cycles in (0, 500, 3000, 10000, -1):
        limit(cycles)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv, return_lse=True, err_flag=err,
                                       **form)
        torch.cuda.synchronize()
        lost = check_lost(out, lse, ref)
        assert int(err.item()) in ((0,) if cycles == -1 else (0, ETIMEOUT))
        assert lost == 0 or int(err.item()) == ETIMEOUT


@pytest.mark.gpu
def test_a_step_of_serving():
    # prompts behind a common document appended, a token appended to each sequence with its queries rotated, attended to
    # behind the prefix and, in another layer, under a window
    import gather_radix_select_gb300 as sel
    from tests.test_cache_append import rotation, turned
    import numpy as np
    b, h, d, rot, ps, common, own = 20, 4, 128, 64, 16, 40, 4
    pages = common + b * own
    cache = torch.zeros((pages, ps, d), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.ones((pages, ps, 1), device="cuda")
    table = shared_tables(b, common + own, common, pages, 141)
    known = (common + own) * ps
    angles = rotation(known, rot)
    on = torch.from_numpy(angles).cuda()
    g = torch.Generator().manual_seed(142)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    doc = torch.randn((common * ps, d), generator=g).to(torch.bfloat16)
    sel.cache_append(doc.cuda(), cache, table[:1], torch.arange(common * ps, device="cuda"), on, scales=scales, err_flag=err)
    per = 30
    prompt = torch.randn((b * per, d), generator=g).to(torch.bfloat16)
    at = common * ps + torch.arange(per).repeat(b)
    sel.cache_append(prompt.cuda(), cache, table, at.cuda(), on, scales=scales, err_flag=err)
    q = torch.randn((b, h, d), generator=g).to(torch.bfloat16)
    x = torch.randn((b, d), generator=g).to(torch.bfloat16)
    now = torch.full((b,), common * ps + per, dtype=torch.int32, device="cuda")
    q_now = sel.cache_append(x.cuda(), cache, table, now, on, scales=scales, q=q.cuda(), err_flag=err)
    want_q = turned(q.float().numpy(), now.tolist(), angles, d - rot, False, np.float32)
    assert torch.equal(q_now.cpu(), torch.from_numpy(want_q).to(torch.bfloat16))
    end = now + 1
    held = rows64(cache, scales)
    out, lse = sel.cache_attention(q_now, cache, table, scales=scales, end=end, return_lse=True, shared=common * ps,
                                   err_flag=err)
    check_attention(out, lse, attend64(q_now, held, table, 1, end.cpu(), None, d, 1 / math.sqrt(d)))
    out, lse = sel.cache_attention(q_now, cache, table, scales=scales, end=end, return_lse=True, window=100, sinks=4,
                                   err_flag=err)
    seen = seen_by_window(end.cpu(), known, 100, 4)
    check_attention(out, lse, attend64(q_now, held, table, 1, None, seen, d, 1 / math.sqrt(d)))
    assert int(err.item()) == 0


# ------------------------------------------------------------------------------- refusals, without a GPU
def call(lib, c, form, **kw):  # noqa: F811
    a = dict(q=FAKE, rows=4, h=8, qrs=1024, qhs=128, table=FAKE, b=2, mp=8, ts=8, end=None, window=100, sinks=4,
             shared=64, dv=128, scale=0.1, out=FAKE, lse=None, ws=None, wsb=0)
    a.update(kw)
    seen = (a["window"], a["sinks"]) if form == "window" else (a["shared"],)
    entry = lib.sel_cache_attention_window if form == "window" else lib.sel_cache_attention_shared
    return entry(a["q"], a["rows"], a["h"], a["qrs"], a["qhs"], ctypes.byref(c) if c else None, a["table"], a["b"],
                 a["mp"], a["ts"], a["end"], *seen, a["dv"], a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("form", ["window", "shared"])
def test_range_refusals(lib, form):  # noqa: F811
    c = struct()
    assert call(lib, c, form, rows=0) == 0
    assert call(lib, None, form) == EINVAL
    for kw in (dict(rows=3), dict(rows=-2), dict(h=0), dict(dv=0), dict(dv=136), dict(scale=float("nan")), dict(q=None),
               dict(out=None), dict(table=None), dict(b=0), dict(ts=7), dict(qrs=-8)):
        assert call(lib, c, form, **kw) == EINVAL, kw
    for kw in (dict(dv=12), dict(q=FAKE + 2), dict(qrs=1028), dict(qhs=132), dict(lse=FAKE + 1), dict(end=FAKE + 2)):
        assert call(lib, c, form, **kw) == EALIGN, kw
    wide = struct(d=528, row_stride=528, scale_row_stride=5, page_stride=528 * 16)
    assert call(lib, wide, form) == EUNSUP
    assert call(lib, c, form, mp=1 << 29, ts=1 << 29) == EUNSUP
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1)) if form == "window" else (dict(shared=-1),):
        assert call(lib, c, form, **kw) == EINVAL, kw


def test_workspace_sizes_refuse_bad_arguments(lib):  # noqa: F811
    window, shared = lib.sel_cache_attention_window_workspace_size, lib.sel_cache_attention_shared_workspace_size
    assert window(4, 8, 128, 128, 1, 8, 16, 0, 0) == 0 and window(4, 8, 128, 128, 1, 8, 16, 5, -1) == 0
    assert window(4, 8, 1024, 128, 1, 8, 16, 5, 0) == 0 and window(4, 8, 128, 128, 3, 8, 16, 5, 0) == 0
    assert shared(4, 8, 128, 128, 1, 8, 16, -1) == 0 and shared(0, 8, 128, 128, 1, 8, 16, 4) == 0
    assert shared(4, 8, 128, 136, 1, 8, 16, 4) == 0 and shared(4, 8, 128, 128, 1, 1 << 40, 1 << 40, 4) == 0


@pytest.mark.gpu
def test_binding_refuses():
    import gather_radix_select_gb300 as sel
    cache, _ = make_cache(4, 8, 64, "bf16", 1)
    table = make_table(2, 2, 4, 2)
    q = make_q(4, 2, 64, 3)
    idx = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    for kw in (dict(window=0), dict(window=-3), dict(window=4, sinks=-1), dict(sinks=4), dict(shared=-1),
               dict(window=4, shared=8), dict(window=4, idx=idx), dict(shared=8, idx=idx), dict(shared=8, sinks=2)):
        with pytest.raises(ValueError):
            sel.cache_attention(q, cache, table, **kw)
