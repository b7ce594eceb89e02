"""GPU checks that kv_attend_shared counts every slot, and once: at every boundary of tiles, pieces, shares and sides.

The check is that of drafts_shares.py.
"""
import numpy as np
import pytest
import torch

import drafts_shares as ds
from test_gpu_drafts import BF16, FP8, Shared, f64, nbw  # noqa: F401

pytestmark = pytest.mark.gpu


class Shares(Shared):
    """Equal keys; values as the rows' slots have their dims."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        live = ~self.k.float().isnan()
        self.k.copy_(torch.where(live, 0.0, self.k.float()).to(self.k.dtype))
        for by in self.scales:
            if by is not None:
                by.fill_(1.0)
        # where each row's slots are
        self.at = []
        for row, n in enumerate(self.lens):
            slot = np.arange(n)
            pages = torch.from_numpy(self.table_np[row][slot // self.page].astype(np.int64)).cuda()
            self.at.append((pages, torch.from_numpy(slot % self.page).cuda()))

    def look(self, length, first, **kw):
        """Runs of `length` slots, number `first` on, one for each dim."""
        dim = self.dim
        for row, n in enumerate(self.lens):
            d = ds.runs(n, length, dim, first)
            value = torch.zeros((n, dim), device="cuda")
            on = np.flatnonzero(d >= 0)
            value[on, d[on]] = 1.0
            pages, places = self.at[row]
            self.v.view(torch.uint8)[pages, :, places] = value.to(self.v.dtype).view(torch.uint8)[:, None, :]
        out = f64(self.call(**kw))
        for row, n in enumerate(self.lens):
            d = ds.runs(n, length, dim, first)
            for t in range(self.cu[row], self.cu[row + 1]):
                sees = n - self.cu[row + 1] + 1 + t
                want = ds.wanted(d, dim, sees)
                for head in (range(out.shape[1]) if t in (self.cu[row], self.cu[row + 1] - 1) else [t % out.shape[1]]):
                    bad = ds.wrong(out[t, head], want, sees)
                    assert not len(bad), (row, t, head, first, bad[:4].tolist(), out[t, head, bad[:4]].tolist(), want[bad[:4]].tolist())

    def look_everywhere(self, length=1, **kw):
        for first in range(0, -(-max(self.lens) // length), self.dim):
            self.look(length, first, **kw)


SHAPES = {
    "one row": [(0, [(1300, 1)])],
    "drafts": [(0, [(700, 5), (650, 3), (9, 9)])],
    "a prefix": [(1290, [(40, 1), (1, 1), (300, 1)])],
    "a prefix and drafts": [(517, [(40, 5), (7, 7), (400, 2), (130, 0)]), (300, [(30, 1), (64, 4)])],
    "prompts": [(0, [(300, 300), (170, 129)])],
    "prompts behind a prefix": [(390, [(150, 150), (90, 70), (40, 1)])],
}


@pytest.mark.parametrize("bits", [False, True])
@pytest.mark.parametrize("which", list(SHAPES))
@pytest.mark.parametrize("q_heads,kv,dim,page,dtype", [(8, 2, 128, 16, BF16), (4, 4, 64, 8, BF16), (6, 1, 256, 64, BF16),
                                                        (8, 2, 128, 32, FP8), (4, 1, 64, 1, FP8), (4, 2, 256, 16, FP8)])
def test_every_slot_counts_once(nbw, which, q_heads, kv, dim, page, dtype, bits):  # noqa: F811
    print(which, q_heads, kv, dim, page, dtype, flush=True)
    Shares(nbw, SHAPES[which], q_heads, kv, dim, page, dtype, seed=dim).look_everywhere(all_bits=bits)


@pytest.mark.parametrize("groups", [[(0, [(60000, 1)])], [(50001, [(1, 1), (9000, 2)])], [(41000, [(300, 3), (20000, 2)])],
                                    [(0, [(58000, 2), (45001, 1)])]])
@pytest.mark.parametrize("heads,kv", [(2, 1), (8, 2)])
def test_every_piece_of_a_long_past_counts_once(nbw, groups, heads, kv):  # noqa: F811
    """More pieces of a line than the last launch looks at together: units of 128 slots, half ones, and single slots here and there."""
    s = Shares(nbw, groups, heads, kv, 64, 64, seed=3)
    s.look_everywhere(128)
    s.look_everywhere(64)
    longest = max(s.lens)
    for first in sorted({0, 1000, 4095 - 32, 128 * 32 - 32, 128 * 33 - 32, longest // 2, max(0, longest - 64), max(0, s.prefix[0] - 32)}):
        s.look(1, first)


@pytest.mark.parametrize("rows,new,tail,q_heads,heads,prefix", [(70, 40, 60, 8, 8, 0), (300, 1, 200, 2, 2, 20), (90, 3, 300, 24, 6, 0),
                                                                 (40, 20, 260, 16, 2, 333), (13, 200, 260, 10, 2, 0)])
def test_every_slot_of_many_short_rows_counts_once(nbw, rows, new, tail, q_heads, heads, prefix):  # noqa: F811
    r = np.random.default_rng(rows)
    sizes = [(max(n, int(r.integers(1, tail))), n) for n in r.integers(0, new + 1, rows).tolist()]
    Shares(nbw, [(prefix, sizes)], q_heads, heads, 64, 16, seed=rows).look_everywhere()
