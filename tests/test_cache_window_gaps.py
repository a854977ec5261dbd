"""Pages between the windows of a tile's rows: no row sees their positions, so they may be anything (a sequence's pages
are freed when its rows' windows have moved on) and are no finding; one that some row does see is."""
import pytest
import torch

from tests.test_cache_ranges import check_window, seen_by_window

# (b, rows a sequence, h, d, dv, page size, pages): every layout of the kernel, several heads of a row and several rows of
# a sequence in a tile, a tile of one row by itself
CASES = [
    (1, 2, 16, 128, 128, 16, 60),
    (1, 3, 40, 128, 96, 7, 140),
    (2, 4, 24, 192, 128, 16, 60),
    (3, 6, 8, 256, 256, 16, 60),
    (2, 5, 12, 320, 320, 24, 40),
    (1, 8, 8, 512, 512, 16, 60),
    (1, 3, 64, 512, 512, 16, 60),
]


def far_ends(case):
    """Ends of a sequence's rows over all of its page table, far from one another; the last one sees nothing."""
    b, per, *_, ps, mp = case
    step = ps * mp // per
    ends = torch.tensor([[40 + i * step - 3 * s for i in range(per)] for s in range(b)], dtype=torch.int32)
    if per > 2:
        ends[:, -1] = 0
    return ends.flatten()


def pages_of(case, ends, window, sinks):
    """The pages of each sequence that some row of it sees."""
    b, per, *_, ps, mp = case
    seen = seen_by_window(ends, ps * mp, window, sinks)
    return [set(int(p) // ps for r in range(s * per, (s + 1) * per) for p in seen[r]) for s in range(b)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_pages_between_windows_are_no_finding(case, kind):
    b, _, *_, mp = case
    ends = far_ends(case)
    for window, sinks in ((20, 3), (1, 0), (33, 40)):
        seen = pages_of(case, ends, window, sinks)

        def freed(cache, table):
            for s in range(b):
                for i, page in enumerate(sorted(set(range(mp)) - seen[s])):
                    table[s, page] = (-1, 1 << 30, -(1 << 31), cache.shape[0])[i % 4]

        assert check_window(case, kind, window, sinks, ends=ends, edit=freed) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_a_page_that_one_of_the_rows_sees_is_reported(case, kind):
    # each page in turn that some row sees: the first tokens', and those of each row's window
    b, per, *_, ps, mp = case
    ends, window, sinks = far_ends(case), 20, 3
    for s in range(b):
        for page in sorted(pages_of(case, ends, window, sinks)[s]):
            def lose(cache, table):
                table[s, page] = -1

            assert check_window(case, kind, window, sinks, ends=ends, edit=lose) == 1
