"""Page table entries outside the cache, whatever their value: the positions there are left out and flagged."""
import pytest
import torch

from tests.test_cache import attend64, check_attention, make_cache, make_q, rows64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("entry", [-1, -2, 4, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1])
def test_entries_outside_the_cache(kind, entry):
    import gather_radix_select_gb300 as sel
    cache, scales = make_cache(4, 8, 64, kind, 801)
    q = make_q(2, 4, 64, 802)
    table = torch.tensor([[0, entry, 2]], dtype=torch.int32, device="cuda")
    idx = torch.tensor([[3, 9, 17, -1], [23, 1, 15, 8]], device="cuda")
    for listed in (None, idx):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=listed, return_lse=True, err_flag=err)
        check_attention(out, lse, attend64(q, rows64(cache, scales), table, 2, None, listed, 64, 1 / 8))
        assert int(err.item()) == 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sel.cache_gather(cache, table, torch.tensor([[9, 17]], device="cuda"), scales=scales, err_flag=err)
    assert int(got[0, 0].view(torch.int16).abs().sum()) == 0 and int(err.item()) == 1
    assert torch.equal(got[0, 1].double().cpu(), rows64(cache, scales)[2, 1])
