"""Attention at lists without an entry: whatever the other tensors' places, zeros and a log-sum of -inf."""
import math

import pytest
import torch


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_an_empty_list_beside_a_page_table_at_an_odd_place(kind, itype, first):
    import gather_radix_select_gb300 as sel
    from tests.test_cache import make_cache, make_q
    cache, scales = make_cache(6, 16, 64, kind, 601)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)[:, first:]
    q = make_q(4, 3, 64, 602)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.empty((4, 0), dtype=itype, device="cuda")
    out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=idx, return_lse=True, err_flag=err)
    assert out.shape == (4, 3, 64) and int(out.view(torch.int16).abs().sum()) == 0
    assert bool((lse == -math.inf).all()) and int(err.item()) == 0


def test_the_address_that_stands_for_an_empty_list_is_aligned(monkeypatch):
    # without a GPU: what the library is given
    from gather_radix_select_gb300 import _native, cache as module
    seen = []

    class Library:
        def sel_cache_attention(self, *args):
            seen.append(args[11])
            return 0

    monkeypatch.setattr(_native, "load", lambda *a, **kw: Library())
    monkeypatch.setattr(module, "_launch", lambda dev, stream, call: call(0))
    monkeypatch.setattr(module, "_scratch_bytes", lambda *a: 0)
    monkeypatch.setattr(module, "_cache_struct", lambda c, scales: _native.SelCache(
        c.data_ptr(), None, _native.SEL_BF16, *c.shape, *c.stride()[:2], 0, 0))
    q = torch.zeros((2, 2, 16), dtype=torch.bfloat16)
    cache = torch.zeros((2, 4, 16), dtype=torch.bfloat16)
    for first in range(4):
        table = torch.zeros((1, 8), dtype=torch.int32)[:, first:]
        module.cache_attention(q, cache, table, idx=torch.empty((2, 0), dtype=torch.int64))
    assert len(seen) == 4 and all(p and p % 8 == 0 for p in seen)
