"""Appends of many rows, where a group of lanes takes several runs of 128 elements of a row (4 of bf16 rows, 2 of fp32):
more than 64 runs a processor.  Rows whose runs a group's share divides and others, rotated runs that cross them, padding
tokens; bits as in tests/test_cache_append.py."""
import numpy as np
import pytest
import torch

from tests.test_cache import GROUP, quantise64
from tests.test_cache_append import rotation

BF16, F32 = torch.bfloat16, torch.float32


def turned_rows(x, at, table, first, interleaved):
    """Rows x [tokens, d] rotated in 32 bits, each product and sum rounded once; at: positions, negative for those that
    stay."""
    half = table.shape[1] // 2
    j = np.arange(half)
    u_at, v_at = (first + 2 * j, first + 2 * j + 1) if interleaved else (first + j, first + half + j)
    live = np.flatnonzero(at >= 0)
    c, s = table[at[live], :half], table[at[live], half:]
    u, v = x[live][:, u_at], x[live][:, v_at]
    out = x.copy()
    out[live[:, None], u_at] = u * c - v * s
    out[live[:, None], v_at] = v * c + u * s
    return out


# d, rotated elements, the first of them: 1 to 8 runs a row; a rotated run within one run of 128, across two lanes' runs,
# across the runs of two groups, the whole row
SHAPES = [(64, 32, 32), (128, 128, 0), (144, 48, 88), (192, 192, 0), (272, 160, 64), (384, 256, 64), (512, 64, 448), (512, 512, 0),
          (576, 64, 512), (640, 320, 320), (1024, 800, 112)]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("xt", [BF16, F32], ids=["from-bf16", "from-f32"])
@pytest.mark.parametrize("d,rot,first", SHAPES)
def test_many_rows(d, rot, first, xt, kind, interleaved):
    import gather_radix_select_gb300 as sel
    runs, b, ps = -(-d // GROUP), 3, 24
    lanes = torch.cuda.get_device_properties(0).multi_processor_count * 64
    per = lanes // runs // b + 5
    tokens = b * per
    assert tokens * runs > lanes
    g = torch.Generator().manual_seed(d + rot)
    known = per + 40
    mp = -(-known // ps)
    pages = b * mp + 1
    table = torch.randperm(pages, generator=g)[: b * mp].to(torch.int32).view(b, mp)
    at = torch.stack([torch.randperm(known, generator=g)[:per] for _ in range(b)])
    at[:, 3::7] = -1
    at = at.flatten()
    x = (torch.randn((tokens, d), generator=g) * torch.exp(2 * torch.randn((tokens, 1), generator=g))).to(xt)
    angles = rotation(known, rot)
    before = torch.randint(0, 120, (pages, ps, d), generator=g, dtype=torch.uint8)
    cache = before.to(BF16).cuda() if kind == "bf16" else before.cuda().view(torch.float8_e4m3fn)
    scales = None if kind == "bf16" else torch.full((pages, ps, runs), 3.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert sel.cache_append(x.cuda(), cache, table.cuda(), at.cuda(), torch.from_numpy(angles).cuda(), scales=scales,
                            first=first, interleaved=interleaved, err_flag=err) is None
    assert int(err.item()) == 0
    rows = turned_rows(x.float().numpy(), at.numpy(), angles, first, interleaved)
    live = torch.nonzero(at >= 0).flatten()
    to = table[live // per, at[live] // ps].long() * ps + at[live] % ps
    if kind == "bf16":
        want = before.to(BF16).view(-1, d)
        want[to] = torch.from_numpy(rows[live.numpy()]).to(BF16)
        assert torch.equal(cache.cpu().view(-1, d).view(torch.int16), want.view(torch.int16))
    else:
        held, s = quantise64(rows[live.numpy()].astype(np.float64))
        want = before.view(torch.float8_e4m3fn).double().view(-1, d)
        want[to] = torch.from_numpy(held)
        want_s = torch.full((pages * ps, runs), 3.0, dtype=torch.float64)
        want_s[to] = torch.from_numpy(s)
        assert torch.equal(cache.cpu().double().view(-1, d), want)
        assert torch.equal(scales.cpu().double().view(-1, runs), want_s)
