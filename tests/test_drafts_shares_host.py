"""Host-side check of drafts_shares: what it is meant to find it finds, wherever it lies.  No GPU."""
import numpy as np
import pytest

import drafts_shares as ds
from oracle import kv as okv


def test_the_oracle_passes():
    rng = np.random.default_rng(0)
    k, v = np.zeros((2, 4, 1, 8, 8))
    table = np.array([[2, 0, 3]])
    dims = rng.integers(-1, 8, 24)
    for j, d in enumerate(dims):
        if d >= 0:
            v[table[0, j // 8], 0, j % 8, d] = 1
    for n in (1, 7, 17, 24):
        out = okv.attend(rng.standard_normal((1, 2, 8)), k, v, table, [n], 1.0)[0][0]
        for head in out:
            assert not len(ds.wrong(head, ds.wanted(dims, 8, n), n))


@pytest.mark.parametrize("sees", [128, 60000, 59051])
def test_a_run_left_out_or_counted_twice_is_found_wherever_it_is(sees):
    length, dim = 128, 64
    for first in range(0, -(-sees // length), dim):
        dims = ds.runs(sees, length, dim, first)
        counts = np.bincount(dims[dims >= 0], minlength=dim).astype(float)
        want = ds.wanted(dims, dim, sees)
        assert not len(ds.wrong(counts / sees, want, sees))
        for d in np.flatnonzero(counts):
            for times in (0, 2):
                mistaken = counts.copy()
                mistaken[d] *= times
                total = sees + (times - 1) * counts[d]
                assert total == 0 or d in ds.wrong(mistaken / total, want, sees) or sees == length


@pytest.mark.parametrize("sees", [40, 1500, 60000])
def test_a_slot_left_out_or_counted_twice_is_found(sees):
    dim = 64
    for first in (0, sees - 40):
        dims = ds.runs(sees, 1, dim, first)
        want = ds.wanted(dims, dim, sees)
        for slot in np.flatnonzero(dims >= 0)[::7]:
            for times in (0, 2):
                got = want * sees
                got[dims[slot]] += times - 1
                assert dims[slot] in ds.wrong(got / (sees + times - 1), want, sees)
