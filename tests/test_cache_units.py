"""Attention over the paged cache where every CTA takes several rows one after the other, each of several tiles of
128 positions: more items than twice the processors, so that nothing is shared out.  One case for each layout of
the kernel: chunks of 128 elements a row (1 to 4), 64 or 128 columns, bf16 or 8-bit rows.  Tolerances are those of
test_cache.py."""
import math

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_cache, make_q, make_table, rows64

pytestmark = pytest.mark.gpu

LAYOUTS = [(h, d, dv, kind) for h, d, dv in ((40, 128, 128), (40, 256, 200), (24, 384, 384), (24, 512, 512),
                                             (80, 128, 128), (80, 192, 192), (80, 192, 128))
           for kind in ("bf16", "fp8")]
layouts = pytest.mark.parametrize("h,d,dv,kind", LAYOUTS)


def whole_items(rows, h, d, dv, b, mp, ps, n=None):
    """Whether no row of such a call is shared out (its CTAs then take several rows each)."""
    from gather_radix_select_gb300 import _native
    return _native.load().sel_cache_attention_workspace_size(rows, h, d, dv, b, mp, ps, n is not None, n or 0) == 0


def many():
    """More rows than twice the processors: some CTAs take three."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count + 16


@layouts
def test_entries_without_a_row_in_every_tile(h, d, dv, kind):
    # lists of 6 tiles with empty entries throughout and positions on pages outside the cache, of another number in
    # every tile and row
    import gather_radix_select_gb300 as sel
    rows, n, ps, mp = many(), 700, 16, 40
    cache, scales = make_cache(mp, ps, d, kind, 201)
    table = make_table(1, mp, mp, 202)
    table[0, 7::9] = -1
    q = make_q(rows, h, d, 203)
    g = torch.Generator().manual_seed(204)
    idx = torch.randint(0, mp * ps, (rows, n), generator=g, dtype=torch.int32)
    idx[torch.rand(idx.shape, generator=g) < torch.rand((rows, 1), generator=g)] = -1
    idx[5] = -1
    idx[6, 130:] = -1
    assert whole_items(rows, h, d, dv, 1, mp, ps, n)
    out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx.cuda(), dv=dv, return_lse=True)
    check_attention(out, lse, attend64(q, rows64(cache, scales), table, rows, None, idx, dv, 1 / math.sqrt(d)))
