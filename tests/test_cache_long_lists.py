"""Attention at lists of millions of entries of which only the first are positions: nothing waits longer than for any
other list, and the results are those of the short list."""
import math

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_cache, make_q, make_table, rows64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("h,d", [(16, 128), (24, 512), (80, 192)])
@pytest.mark.parametrize("rows,n", [(1, 8_000_000), (3, 2_000_001)])
def test_lists_with_long_empty_ends(kind, h, d, rows, n):
    import gather_radix_select_gb300 as sel
    from gather_radix_select_gb300 import _native
    ps, mp, used = 16, 40, 300
    cache, scales = make_cache(mp, ps, d, kind, 701)
    table = make_table(1, mp, mp, 702)
    q = make_q(rows, h, d, 703)
    g = torch.Generator().manual_seed(704)
    short = torch.randint(0, mp * ps, (rows, used), generator=g, dtype=torch.int32)
    idx = torch.full((rows, n), -1, dtype=torch.int32, device="cuda")
    idx[:, :used] = short.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib = _native.load()
    try:
        lib.sel_cache_set_wait_limit(4_000_000)  # (about 2 ms instead of 2 s)
        out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx, return_lse=True, err_flag=err)
        torch.cuda.synchronize()
    finally:
        lib.sel_cache_set_wait_limit(-1)
    assert int(err.item()) == 0
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, rows, None, short, d, 1 / math.sqrt(d)))
