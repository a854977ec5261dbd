"""Windows whose positions lie just below 2^31: numbers, pages and tile counts in 32 bits.  (One cache page of 2^24 rows that
the page table names again and again; only what the rows see is compared.)"""
import math

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_q


@pytest.mark.gpu
@pytest.mark.parametrize("h,d", [(16, 16), (96, 32)])
def test_windows_far_behind(h, d):
    import gather_radix_select_gb300 as sel
    ps, mp = 1 << 24, 127
    cap = ps * mp
    g = torch.Generator(device="cuda").manual_seed(31)
    cache = torch.randn((2, ps, d), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    table = torch.zeros((1, mp), dtype=torch.int32, device="cuda")
    table[0, 1::2] = 1
    for ends, window, sinks in (([cap], 300, 5), ([cap - 1, cap], 129, 0), ([cap - 2 * ps + 1, cap - 2 * ps + 2, cap - 2 * ps + 9], 7, 200),
                                ([cap + 9], 4096, 4096)):
        q = make_q(len(ends), h, d, 32)
        end = torch.tensor(ends, dtype=torch.int32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, end=end.cuda(), return_lse=True, window=window, sinks=sinks, err_flag=err)
        seen = [torch.cat((torch.arange(sinks), torch.arange(min(e, cap) - window, min(e, cap)))) for e in ends]
        # the seen rows alone, a page a row
        flat = [(int(table[0, p // ps]), int(p % ps)) for s in seen for p in s.tolist()]
        rows = cache[torch.tensor([a for a, _ in flat]).cuda(), torch.tensor([b for _, b in flat]).cuda()].cpu().double()[:, None]
        first = [sum(len(s) for s in seen[:r]) for r in range(len(seen))]
        own = [torch.arange(first[r], first[r] + len(seen[r])) for r in range(len(seen))]
        here = torch.arange(len(flat), dtype=torch.int32)[None]
        check_attention(out, lse, attend64(q, rows, here, len(ends), None, own, d, 1 / math.sqrt(d)))
        assert int(err.item()) == 0
