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


# rows of one sequence that share a CTA's columns: two of 24 heads in 64, three of 40 in 128
SHARED = [(24, 2, d, dv, kind) for d, dv in ((128, 96), (192, 192), (256, 136), (320, 320), (512, 512))
          for kind in ("bf16", "fp8")]
SHARED += [(40, 3, d, dv, kind) for d, dv in ((128, 128), (96, 40), (192, 192), (192, 128), (144, 64))
           for kind in ("bf16", "fp8")]
shared = pytest.mark.parametrize("h,per,d,dv,kind", SHARED)
PS, MP = 16, 52  # contexts of up to 832 positions: 7 tiles


def sequences(h, per, d, dv, kind, seed):
    """A cache whose pages all sequences share, more sequences than twice the processors, rows that end at 700, 745 and
    790: the tile from 640 on has the first row's end in it, the last tile only the last row's."""
    b = many()
    cache, scales = make_cache(MP + 1, PS, d, kind, seed)
    g = torch.Generator().manual_seed(seed + 1)
    table = torch.stack([torch.randperm(MP, generator=g) for _ in range(b)]).to(torch.int32).cuda()
    q = make_q(b * per, h, d, seed + 2)
    end = torch.tensor([700 + 45 * i for i in range(per)] * b, dtype=torch.int32)
    assert whole_items(b * per, h, d, dv, b, MP, PS)
    return b, cache, scales, table, q, end


def some(b, per):
    """Sequences whose rows are compared (the lowest are the last units of their CTAs), and those rows."""
    seqs = list(range(20)) + list(range(20, b, 23)) + [b - 1]
    return seqs, torch.tensor([s * per + i for s in seqs for i in range(per)])


@shared
def test_scores_that_climb_within_a_unit(h, per, d, dv, kind):
    # the scores rise by about 30 bits a tile: references move, sums and accumulators are rescaled, in every tile
    import gather_radix_select_gb300 as sel
    b, cache, scales, table, q, end = sequences(h, per, d, dv, kind, 221)
    table[:] = torch.arange(MP, dtype=torch.int32, device="cuda")
    rise = torch.linspace(0, 35, MP * PS).view(MP, PS)
    dtype, x = cache.dtype, rows64(cache, scales).float()
    x[:MP, :, 0] = rise
    if scales is not None:
        scales[:, :, 0] = 0.125  # (codes of up to 280)
        x[:, :, : 128] /= 0.125
        if d > 128:
            x[:, :, 128:] /= scales.cpu()[:, :, 1:].repeat_interleave(128, dim=-1)[..., : d - 128]
    cache = x.to(dtype).cuda()
    q[:, :, 0] = 4.0
    out, lse = sel.cache_attention(q, cache, table, scales=scales, end=end.cuda(), dv=dv, return_lse=True, scale=1.0)
    seqs, rows = some(b, per)
    check_attention(out[rows], lse[rows], attend64(q[rows], rows64(cache, scales), table[seqs], per, end[rows], None, dv,
                                                   1.0))
    # the same positions as lists, in the order in which they climb, are taken a row a unit
    idx = torch.arange(MP * PS, dtype=torch.int32).expand(b * per, -1).contiguous()
    idx = torch.where(idx < end[:, None], idx, -1)
    if whole_items(b * per, h, d, dv, b, MP, PS, MP * PS):
        listed, lse2 = sel.cache_attention(q, cache, table, scales=scales, idx=idx.cuda(), dv=dv, return_lse=True, scale=1.0)
        check_attention(listed[rows], lse2[rows], attend64(q[rows], rows64(cache, scales), table[seqs], per, None, idx[rows],
                                                           dv, 1.0))


@shared
def test_a_row_that_is_not_finite_in_a_late_tile_of_a_late_unit(h, per, d, dv, kind):
    # position 710 of every seventh sequence is NaN: its first row, which ends at 700, does not notice
    import gather_radix_select_gb300 as sel
    b, cache, scales, table, q, end = sequences(h, per, d, dv, kind, 231)
    at = 710
    seqs, rows = some(b, per)
    was = int(table[0, at // PS])  # a copy of this page has the NaN, at 710's place in every seventh sequence
    other = table.clone()
    for s in range(0, b, 7):
        where = int((table[s] == was).nonzero())
        other[s, where], other[s, at // PS] = int(table[s, at // PS]), MP
    if scales is not None:
        scales[MP] = scales[was]
    cache = cache.float()
    cache[MP] = cache[was]
    clean = attend64(q[rows], rows64(cache.to(q.dtype if scales is None else torch.float8_e4m3fn), scales), other[seqs],
                     per, end[rows], None, dv, 1 / 16)
    seen = torch.tensor([s % 7 == 0 and i > 0 for s in seqs for i in range(per)])
    for first in (0, dv - 8, d - 1):
        poisoned = cache.clone()
        poisoned[MP, at % PS, first:] = math.nan
        poisoned = poisoned.to(torch.bfloat16 if scales is None else torch.float8_e4m3fn)
        out, lse = sel.cache_attention(q, poisoned, other, scales=scales, end=end.cuda(), dv=dv, scale=1 / 16,
                                       return_lse=True)
        out, lse = out[rows], lse[rows]
        check_attention(out[~seen], lse[~seen], tuple(t[~seen] for t in clean))
        assert bool(torch.isnan(out[seen].float()).all()) and bool(torch.isnan(lse[seen]).all())
