"""The queries of a token that is not rotated, a padding token or one past the rotation's table, are returned as they are:
bit for bit, whatever NaN they hold."""
import pytest
import torch

from tests.test_cache_append import rotation


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("in_place", [False, True], ids=["elsewhere", "in place"])
@pytest.mark.parametrize("first,rot", [(0, 128), (64, 64), (8, 48)])
def test_queries_that_stay_keep_their_bits(first, rot, in_place, interleaved):
    import gather_radix_select_gb300 as sel
    tokens, h, d = 7, 5, 128
    # every bit pattern class of bf16: quiet and signalling NaN of both signs with payloads, infinities, subnormals
    odd = torch.tensor([0x7F81, 0x7FC1, 0xFF81 - 0x10000, 0xFFFF - 0x10000, 0x7F80, 0xFF80 - 0x10000, 1, 0x8001 - 0x10000],
                       dtype=torch.int16)
    q = odd.repeat(tokens * h * d // 8).view(tokens, h, d).cuda()
    q[0] = 0x3F80  # (a live token, finite)
    was = q.clone()
    cache = torch.zeros((2, 8, d), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    at = torch.tensor([3, -1, -5, -1, 12, 12, -1], device="cuda")  # 12: past the rotation's table
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sel.cache_append(torch.zeros((tokens, d), device="cuda"), cache, table, at,
                           torch.from_numpy(rotation(10, rot)).cuda(), first=first, interleaved=interleaved,
                           q=q.view(torch.bfloat16), q_out=q.view(torch.bfloat16) if in_place else None, err_flag=err)
    assert int(err.item()) == 1
    assert torch.equal(got.view(torch.int16)[1:], was[1:])
