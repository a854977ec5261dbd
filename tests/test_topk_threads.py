"""Selections by several host threads on one stream: a row that is split over several CTAs takes two operations on the
stream, the reset of the scratch's counters and the kernel, and another thread's may come between them."""
import contextlib
import threading
import types

import numpy as np
import pytest
import torch


def test_calls_under_way_at_once_have_scratch_of_their_own(monkeypatch):
    # without a GPU: what two calls on one raw stream are given, both still held
    import gather_radix_select_gb300 as sel
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    stream = types.SimpleNamespace(cuda_stream=7)
    a, n = sel._workspace(4096, torch.device("cpu"), stream)
    b, _ = sel._workspace(4096, torch.device("cpu"), stream)
    assert a.numel() >= n >= 4096
    assert abs(a.data_ptr() - b.data_ptr()) >= 4096
    assert sel._workspace(0, torch.device("cpu"), stream) == (None, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("own_stream", [False, True])
def test_two_threads_on_one_stream_get_the_oracles_positions(own_stream):
    import gather_radix_select_gb300 as sel
    import oracle
    calls, jobs = 200, []
    side = torch.cuda.Stream() if own_stream else None
    for rows, cols, k in ((4, 204800, 1024), (2, 150000, 512)):
        assert sel.workspace_size(torch.bfloat16, rows, cols, k) > 0
        rng = np.random.default_rng(rows)
        x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(torch.bfloat16)
        want, _, _ = oracle.topk(x.view(torch.int16).numpy().view(np.uint16), "bf16", k, sorted_index=True)
        jobs.append((x.cuda(), k, torch.from_numpy(np.asarray(want).astype(np.int32)).cuda()))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(len(jobs)), []

    def work(x, k, want):
        try:
            start.wait(timeout=60)
            got = [sel.topk(x, k, sorted_index=True, return_value=False, stream=side)[1] for _ in range(calls)]
            torch.cuda.synchronize()
            wrong.extend(i for i, idx in enumerate(got) if not torch.equal(idx, want))
        except Exception as e:  # (an exception in a thread does not fail the test by itself)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
