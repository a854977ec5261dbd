"""Attention over page tables that share pages without the call saying so: the bits of a call whose sequences have copies
of those pages for themselves (what is fetched ahead goes by what neighbouring sequences share; results do not)."""
import pytest
import torch

from tests.test_cache import make_cache, make_q
from tests.test_cache_ranges import shared_tables

# (b, h, d, page size, pages, pages in common): rows of up to 512 elements, units of few tiles and of many, one sequence
CASES = [
    (3, 64, 512, 16, 130, 100),
    (5, 64, 512, 7, 400, 399),
    (2, 40, 384, 16, 100, 100),
    (1, 64, 512, 16, 90, 50),
    (4, 64, 512, 16, 50, 0),
    (200, 64, 512, 16, 60, 30),
    (160, 16, 256, 24, 80, 70),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_shared_pages_and_copies_of_them(case, kind):
    import gather_radix_select_gb300 as sel
    b, h, d, ps, mp, common = case
    cache, scales = make_cache(common + b * (mp - common), ps, d, kind, 11)
    wide = torch.zeros((b, mp + 3), dtype=torch.int32, device="cuda")
    table = wide[:, :mp]  # (rows of the page table are strided)
    table.copy_(shared_tables(b, mp, common, cache.shape[0], 12))
    whole = cache.view(torch.int16 if kind == "bf16" else torch.uint8)[table.flatten().long()].view(cache.dtype)
    own = torch.arange(b * mp, dtype=torch.int32, device="cuda").view(b, mp)
    s_own = None if scales is None else scales[table.flatten().long()]
    q = make_q(b, h, d, 13)
    end = torch.tensor([mp * ps - 3 * i if i % 7 != 6 else 0 for i in range(b)], dtype=torch.int32).clamp(min=0).cuda()
    for form in ({}, {"window": mp * ps // 2, "sinks": 5}):
        want, l1 = sel.cache_attention(q, whole, own, scales=s_own, end=end, return_lse=True, **form)
        got, l2 = sel.cache_attention(q, cache, table, scales=scales, end=end, return_lse=True, **form)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(l1, l2)
    shared, l3 = sel.cache_attention(q, cache, table, scales=scales, end=end, return_lse=True, shared=common * ps)
    plain, _ = sel.cache_attention(q, cache, table, scales=scales, end=end)
    assert bool((shared.double() - plain.double()).abs().max() <= 2.0 ** -6 * plain.double().abs().max())
    assert torch.equal(torch.isinf(l3), end[:, None].expand(-1, h) == 0)
