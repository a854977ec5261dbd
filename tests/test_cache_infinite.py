"""Attention over a paged cache that holds infinite elements: a position whose score is -inf has the weight 0, and
the others are what they would be without it."""
import math

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_q, make_table, rows64

pytestmark = pytest.mark.gpu

# (heads, d, dv): every layout that bf16 rows have.  (8-bit rows have no infinity.)
LAYOUTS = [(40, 128, 120), (40, 256, 200), (24, 384, 256), (24, 512, 504), (80, 128, 64), (80, 192, 128)]


def low_scores(rows, h, d, mp, ps, seed, low):
    """Queries of positive last elements and a cache whose scores are all near `low` (at a scale of 1)."""
    q = make_q(rows, h, d, seed) / 16
    q[:, :, d - 1] = q[:, :, d - 1].abs() + 1
    q[:, :, 0] = 1
    g = torch.Generator().manual_seed(seed + 1)
    cache = torch.randn((mp, ps, d), generator=g)
    cache[:, :, 0] = low
    return q.to(torch.bfloat16), cache.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("low", [-100.0, -400.0, 300.0])
@pytest.mark.parametrize("h,d,dv", LAYOUTS)
def test_a_tile_of_minus_infinity_before_low_scores(h, d, dv, low):
    # the first tiles hold nothing but a position that scores -inf for every head; the scores after it are so low
    # that 2^score is 0.  Listed positions, several rows a CTA and few enough to be shared out.
    import gather_radix_select_gb300 as sel
    ps, mp = 16, 30
    for rows in (2, 2 * torch.cuda.get_device_properties(0).multi_processor_count + 16):
        q, cache = low_scores(rows, h, d, mp, ps, 501, low)
        table = make_table(1, mp, mp, 503)
        at = 77
        cache[int(table[0, at // ps]), at % ps, d - 1] = -math.inf
        g = torch.Generator().manual_seed(504)
        idx = torch.randint(78, mp * ps, (rows, 400), generator=g)
        idx[:, :256] = -1
        idx[:, 3] = at
        idx[1, :] = -1
        idx[1, [5, 399]] = at  # nothing but the position that weighs nothing
        out, lse = sel.cache_attention(q, cache, table, idx=idx.cuda(), dv=dv, scale=1.0, return_lse=True)
        idx[idx == at] = -1
        finite = rows64(cache, None)
        finite[int(table[0, at // ps]), at % ps] = 0
        check_attention(out, lse, attend64(q, finite, table, rows, None, idx, dv, 1.0))


@pytest.mark.parametrize("per,context", [(0, 500), (5, 700), (1, 60000)])
@pytest.mark.parametrize("h,d,dv", LAYOUTS)
def test_first_positions_of_minus_infinity(h, d, dv, per, context):
    # every position of the first tile scores -inf, over contexts: whole rows, parts of a tile, parts of several tiles
    import gather_radix_select_gb300 as sel
    ps = 32
    per = per or 2 * torch.cuda.get_device_properties(0).multi_processor_count + 16
    mp = -(-context // ps)
    q, cache = low_scores(per, h, d, mp, ps, 511, -300.0)
    table = make_table(1, mp, mp, 512)
    finite = rows64(cache, None)
    skip = 131
    for p in range(skip):
        cache[int(table[0, p // ps]), p % ps, d - 1] = -math.inf
    end = torch.tensor([context - per + 1 + i for i in range(per)], dtype=torch.int32)
    out, lse = sel.cache_attention(q, cache, table, end=end.cuda(), dv=dv, scale=1.0, return_lse=True)
    idx = torch.arange(skip, context).expand(per, -1)
    check_attention(out, lse, attend64(q, finite, table, per, end, idx, dv, 1.0))
