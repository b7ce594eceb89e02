"""GPU checks of the pasts that kv_attend_shared reads: which row's table stands for a prefix.

The check and its tolerance are those of test_gpu_drafts.py.
"""
import numpy as np
import pytest
import torch

from test_gpu_drafts import Shared, ints, nbw  # noqa: F401

pytestmark = pytest.mark.gpu


def put_table(s):
    s.cache.table.copy_(torch.from_numpy(s.table_np))


def shorten(s, row, length, past):
    """A row of that length; past it the table holds what `past` says, as a row does whose pages have gone to others."""
    s.lens[row] = length
    at = -(-length // s.page)
    s.table_np[row, at:] = np.resize(past, s.table_np.shape[1] - at)


def others(s, row):
    """Pages of another row's own slots."""
    first = s.prefix[s.group[row]] // s.page
    return s.table_np[row, first:-(-s.lens[row] // s.page)].copy()


@pytest.mark.parametrize("new", [0, 2])
@pytest.mark.parametrize("past", ["none", "others"])
@pytest.mark.parametrize("length", [0, 2, 40, 99])
@pytest.mark.parametrize("page", [16, 4])
def test_a_prefix_behind_a_first_row_that_is_shorter(nbw, length, past, new, page):  # noqa: F811
    s = Shared(nbw, [(100, [(9, new), (30, 2), (4, 1), (60, 3)]), (37, [(1, new), (8, 1)])], 8, 2, 128, page, seed=length)
    shorten(s, 0, length, others(s, 3) if past == "others" else [-1])
    shorten(s, 4, min(length, 36), others(s, 3) if past == "others" else [-1])
    put_table(s)
    s.check(s.call())


@pytest.mark.parametrize("long", [1, 2, 3, 4, 5, 6])
def test_a_prefix_that_one_row_alone_has(nbw, long):  # noqa: F811
    """Rows before and behind it are shorter, each by another length, and name others' pages past it."""
    s = Shared(nbw, [(200, [(20, 1)] * 7)], 4, 2, 64, 8, seed=long)
    past = others(s, long)
    for row in range(7):
        if row != long:
            shorten(s, row, 31 * row, past)
    put_table(s)
    s.check(s.call())


def test_a_prefix_that_no_row_has(nbw):  # noqa: F811
    s = Shared(nbw, [(200, [(20, 2)] * 5), (64, [(3, 1)] * 2)], 4, 2, 64, 8, seed=3)
    for row, n in enumerate((3, 50, 170, 169, 0, 0, 63)):
        shorten(s, row, n, [-1])
    put_table(s)
    s.check(s.call())


@pytest.mark.parametrize("long", [3, 4, 63, 68, 700, 999, None])
def test_a_prefix_of_a_thousand_rows(nbw, long):  # noqa: F811
    """The row that is as long as the prefix is anywhere among them, or there is none."""
    s = Shared(nbw, [(24, [(2, 1)] * 3), (50, [(1, 1)] * 1000), (24, [(2, 1)] * 3)], 2, 1, 64, 4, seed=4)
    for row in range(3, 1003):
        if row != (3 + long if long is not None else None):
            shorten(s, row, row % 49, [-1])
    put_table(s)
    s.check(s.call())


def test_more_groups_than_threads_behind_rows_that_have_ended(nbw):  # noqa: F811
    groups = [((0, 11, 30)[i % 3], [(5, 1)] * (2 + i % 9)) for i in range(400)]
    s = Shared(nbw, groups, 2, 1, 64, 4, seed=5)
    for g in range(400):
        for row in range(s.bounds[g], s.bounds[g + 1] - 1 - g % 2):
            shorten(s, row, (0, 7)[row % 2], [-1])
    put_table(s)
    s.check(s.call())


def test_a_first_row_that_ends_between_replays(nbw):  # noqa: F811
    s = Shared(nbw, [(120, [(9, 1), (30, 2), (60, 3)])], 8, 2, 128, 16, seed=6)
    lens, cu, groups, prefix = ints(s.lens), ints(s.cu), ints(s.bounds), ints(s.prefix)
    out = torch.zeros_like(s.q)
    workspace = torch.empty(s.cache.attend_shared_workspace_bytes(8, s.cu[-1], 1), dtype=torch.uint8, device="cuda")

    def call():
        nbw.kv_attend_shared(s.cache, s.q, lens, cu=cu, groups=groups, prefix=prefix, out=out, workspace=workspace)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for length in (129, 60, 0):
        shorten(s, 0, length, [-1])
        put_table(s)
        lens.copy_(ints(s.lens))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(out)
        assert torch.equal(out, s.call())
