"""The attention's bounded waits: with a limit of no cycles at all they give up wherever they would really wait, without
anything being broken for it.  The kernel then ends, says SEL_ETIMEOUT, leaves NaN instead of the results it lost, and
the next call with the usual limit is right."""
import math

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_cache, make_q, make_table, rows64

pytestmark = pytest.mark.gpu

ETIMEOUT = 5


@pytest.fixture
def limit():
    from gather_radix_select_gb300 import _native
    lib = _native.load()
    yield lib.sel_cache_set_wait_limit
    lib.sel_cache_set_wait_limit(-1)


def check_lost(out, lse, ref):
    """Each row is NaN throughout, or right; returns how many are NaN."""
    gone = torch.isnan(out).any(dim=2) | torch.isnan(lse)
    assert bool(torch.isnan(out[gone]).all()) and bool(torch.isnan(lse[gone]).all())
    kept = ~gone.any(dim=1).cpu()
    check_attention(out[kept], lse[kept], tuple(t[kept] for t in ref))
    return int((~kept).sum())


# chunks of 128 elements by 64 or 128 columns, each with its own rows in flight
@pytest.mark.parametrize("h,d,dv", [(16, 128, 128), (40, 512, 512), (80, 192, 128), (24, 384, 256)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_lists_whose_units_come_late(limit, h, d, dv, kind):
    # the search for a list's last entry takes far longer than the limit: the units come too late for every row
    import gather_radix_select_gb300 as sel
    n, ps, mp = 5000, 16, 40
    cache, scales = make_cache(mp, ps, d, kind, 301)
    table = make_table(1, mp, mp, 302)
    for rows in (1, 3, 2 * torch.cuda.get_device_properties(0).multi_processor_count + 16):
        q = make_q(rows, h, d, 303)
        g = torch.Generator().manual_seed(304)
        idx = torch.full((rows, n), -1, dtype=torch.int32)
        idx[:, :200] = torch.randint(0, mp * ps, (rows, 200), generator=g, dtype=torch.int32)
        ref = attend64(q, rows64(cache, scales), table, rows, None, idx, dv, 1 / math.sqrt(d))
        idx = idx.cuda()

        def call(err):
            got = sel.cache_attention(q, cache, table, scales=scales, idx=idx, dv=dv, return_lse=True, err_flag=err)
            torch.cuda.synchronize()
            return got

        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        limit(0)
        out, lse = call(err)
        assert int(err.item()) == ETIMEOUT
        assert check_lost(out, lse, ref) > 0
        out, lse = call(None)  # (no flag to write to: the results say it)
        assert check_lost(out, lse, ref) > 0
        limit(-1)
        err.zero_()
        out, lse = call(err)
        check_attention(out, lse, ref)
        assert int(err.item()) == 0


@pytest.mark.parametrize("h,d,dv", [(16, 128, 128), (40, 512, 512), (80, 192, 128), (24, 384, 256)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("b,per", [(1, 1), (3, 2), (2, 170)])
def test_contexts_under_short_limits(limit, h, d, dv, kind, b, per):
    # contexts of many tiles, shared out or not: waits give up anywhere, or nowhere
    import gather_radix_select_gb300 as sel
    ps = 16
    mp = 40 if per > 10 else 400
    cache, scales = make_cache(b * mp, ps, d, kind, 311)
    table = make_table(b, mp, b * mp, 312)
    q = make_q(b * per, h, d, 313)
    end = torch.tensor([mp * ps - 3 * i % 200 for i in range(b * per)], dtype=torch.int32)
    ref = attend64(q, rows64(cache, scales), table, per, end, None, dv, 1 / math.sqrt(d))
    for cycles in (0, 500, 3000, 10000, -1):
        limit(cycles)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv, return_lse=True, err_flag=err)
        torch.cuda.synchronize()
        lost = check_lost(out, lse, ref)
        assert int(err.item()) in ((0,) if cycles == -1 else (0, ETIMEOUT))
        assert lost == 0 or int(err.item()) == ETIMEOUT
