"""Calls of several host threads on one stream.  A call that shares its positions out over several CTAs is two
launches, which pass data through the call's scratch; another thread's launches on the same stream may come
between them."""
import math
import threading

import pytest
import torch

from tests.test_cache import attend64, check_attention, make_cache, make_q, make_table, rows64


def test_two_calls_under_way_on_one_stream_have_scratch_of_their_own(monkeypatch):
    # without a GPU: the library is replaced by one that holds each call until the other is there too
    from gather_radix_select_gb300 import _native, cache as module
    need, both, seen = 4096, threading.Barrier(2), []

    class Library:
        def sel_cache_attention(self, *args):
            both.wait(timeout=30)
            seen.append((args[-4], args[-3]))  # the scratch and its size
            both.wait(timeout=30)
            return 0

    library = Library()
    monkeypatch.setattr(_native, "load", lambda *a, **kw: library)
    monkeypatch.setattr(module, "_launch", lambda dev, stream, call: call(7))  # one raw stream for both
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(module, "_scratch_bytes", lambda *a: need)
    monkeypatch.setattr(module, "_cache_struct", lambda c, scales: _native.SelCache(
        c.data_ptr(), None, _native.SEL_BF16, *c.shape, *c.stride()[:2], 0, 0))
    cache = torch.zeros((2, 4, 16), dtype=torch.bfloat16)
    q = torch.zeros((1, 2, 16), dtype=torch.bfloat16)
    table = torch.zeros((1, 2), dtype=torch.int32)
    threads = [threading.Thread(target=module.cache_attention, args=(q, cache, table)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a, size_a), (b, size_b) = seen
    assert size_a == size_b == need and a and b
    assert abs(a - b) >= need


@pytest.mark.gpu
def test_two_threads_on_one_stream_get_the_bits_of_one():
    import gather_radix_select_gb300 as sel
    ps, calls = 16, 300
    jobs = []
    for i, (rows, h, d, mp, kind) in enumerate([(1, 16, 128, 150, "bf16"), (3, 40, 512, 130, "fp8")]):
        cache, scales = make_cache(rows * mp, ps, d, kind, 400 + i)
        table = make_table(rows, mp, rows * mp, 410 + i)
        q = [make_q(rows, h, d, 420 + 10 * i + j) for j in range(3)]
        from gather_radix_select_gb300 import _native
        assert _native.load().sel_cache_attention_workspace_size(rows, h, d, d, rows, mp, ps, 0, 0) > 0  # (two launches)

        def run(x, cache=cache, scales=scales, table=table):
            return sel.cache_attention(x, cache, table, scales=scales, return_lse=True)

        want = [run(x) for x in q]
        for x, (out, lse) in zip(q, want):
            check_attention(out, lse, attend64(x, rows64(cache, scales), table, 1, None, None, d, 1 / math.sqrt(d)))
        jobs.append((q, run, want))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(len(jobs)), []

    def work(q, run, want):
        try:
            start.wait(timeout=60)
            got = [run(q[i % len(q)]) for i in range(calls)]
            torch.cuda.synchronize()
            for i, (out, lse) in enumerate(got):
                if not (torch.equal(out.view(torch.int16), want[i % len(q)][0].view(torch.int16))
                        and torch.equal(lse.view(torch.int32), want[i % len(q)][1].view(torch.int32))):
                    wrong.append(i)
        except Exception as e:  # (an exception in a thread does not fail the test by itself)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
