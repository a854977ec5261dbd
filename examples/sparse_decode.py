"""Decoding with a paged key cache and selected positions: per step and sequence one new token's row is written
(8 bits, a power-of-two scale for each 128 elements), the positions with the best index scores are
selected among those so far, and the heads attend to them.  The step is captured once and replayed.

    python examples/sparse_decode.py [--sequences 16] [--context 8192] [--select 512] [--steps 8]

The indexer here is one bf16 vector per position with a plain matrix product for the scores; queries, rows
and index vectors are random.  Prints the time of a step and the largest difference from plain 64-bit
arithmetic over the rows read back.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gather_radix_select_gb300 as sel  # noqa: E402

PAGE, HEADS, D, DV, INDEX_D = 64, 64, 512, 512, 128


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--sequences", type=int, default=16)
    p.add_argument("--context", type=int, default=8192)
    p.add_argument("--select", type=int, default=512)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    b, pages = a.sequences, -(-(a.context + a.steps) // PAGE)
    cap = pages * PAGE

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    cache = torch.zeros((b * pages, PAGE, D), device="cuda").to(torch.float8_e4m3fn)
    scales = torch.zeros((b * pages, PAGE, -(-D // 128)), device="cuda")
    table = torch.randperm(b * pages, generator=g, device="cuda").to(torch.int32).view(b, pages)
    index = torch.zeros((b, cap, INDEX_D), dtype=torch.bfloat16, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")

    # the prompt: every sequence's rows at once
    at = torch.arange(a.context, device="cuda")
    sel.cache_write(rand(b * a.context, D), cache, (table[:, at // PAGE].long() * PAGE + at % PAGE).flatten(), scales=scales,
                    err_flag=bad)
    index[:, : a.context] = rand(b, a.context, INDEX_D)

    # a step's inputs: the position, the new rows and index vectors, the queries of the heads and of the indexer
    pos = torch.full((1,), a.context, device="cuda")
    row, key, q, q_index = rand(b, D), rand(b, 1, INDEX_D), rand(b, HEADS, D), rand(b, INDEX_D, 1)

    def step():
        slot = table.gather(1, (pos // PAGE).expand(b, 1)).long() * PAGE + pos % PAGE
        sel.cache_write(row, cache, slot.flatten(), scales=scales, err_flag=bad)
        index.index_copy_(1, pos, key)
        end = (pos + 1).to(torch.int32).repeat(b)
        _, best = sel.topk((index @ q_index).squeeze(2), a.select, end=end, return_value=False)
        out, lse = sel.cache_attention(q, cache, table, scales=scales, idx=best, end=end, dv=DV, return_lse=True,
                                       err_flag=bad)
        return best, out, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (once before the capture: libraries and attributes are set up)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        best, out, lse = step()

    begin, done = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for n in range(a.steps):
        for buffer, shape in ((row, (b, D)), (key, (b, 1, INDEX_D)), (q, (b, HEADS, D)), (q_index, (b, INDEX_D, 1))):
            buffer.copy_(rand(*shape))
        pos.fill_(a.context + n)
        begin.record()
        graph.replay()
        done.record()
        done.synchronize()
        rows = sel.cache_gather(cache, table, best, scales=scales).double()
        z = q.double() @ rows.transpose(1, 2) / math.sqrt(D)
        off = (out.double() - torch.softmax(z, -1) @ rows[..., :DV]).abs().max().item()
        off_lse = (lse.double() - torch.logsumexp(z, -1)).abs().max().item()
        print(f"position {a.context + n}: {begin.elapsed_time(done) * 1e3:.0f} us, output within {off:.1e}, "
              f"log-sum within {off_lse:.1e}")
    assert int(bad.item()) == 0


if __name__ == "__main__":
    main()
