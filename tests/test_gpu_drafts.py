"""GPU checks of a step with drafted tokens: kv_reserve, kv_attend_shared and verify_drafts against the oracle.

Whole numbers are compared for equality.  The attention's tolerance is derived beside its check.
"""
import math
import random

import numpy as np
import pytest
import torch

from oracle import drafts as odrafts
from oracle import kv as okv

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def nbw():
    import nested_bit_weight_amd as m
    if not torch.cuda.is_available():
        pytest.fail("needs a GPU")
    m.library()
    return m


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def f64(t):
    return t.detach().cpu().to(torch.float32).double().numpy()


# ---------------------------------------------------------------------------
# reserve

class Book:
    """A cache's table with rows that hold pages, a stack of free ones, and the same for the oracle."""

    def __init__(self, nbw, lens, held, width, page=8, spare=20, shared=None, seed=0, table_ld=None, free_size=None):
        g = np.random.default_rng(seed)
        rows = len(lens)
        pages = sum(held) + spare + 1
        order = g.permutation(pages).astype(np.int32)
        self.table = np.full((rows, width), -7, dtype=np.int32)
        at = 0
        for r, h in enumerate(held):
            self.table[r, :h] = order[at:at + h]
            at += h
        for r in range(1, rows if shared else 0):
            self.table[r, :shared[r]] = self.table[0, :shared[r]]
        self.free = np.full(free_size or pages, -9, dtype=np.int32)
        self.free[:spare] = order[at:at + spare]
        self.rows, self.page, self.pages, self.spare, self.shared = rows, page, pages, spare, shared
        self.lens, self.held = lens, held
        wide = torch.full((rows, table_ld or width), -7, dtype=torch.int32, device="cuda")
        wide[:, :width] = torch.from_numpy(self.table).cuda()
        self.wide, self.width = wide, width
        pool = torch.zeros((pages, 1, page, 64), dtype=BF16, device="cuda")
        self.cache = nbw.KVCache(pool, pool, wide[:, :width])
        self.free_t = torch.from_numpy(self.free).cuda()

    def check(self, nbw, want, most, seen=None, count=None):
        count = self.spare if count is None else count
        self.wide[:, :self.width] = torch.from_numpy(self.table).cuda()
        self.free_t.copy_(torch.from_numpy(self.free))
        ref = okv.reserve(self.table, self.page, self.pages, self.lens, want, self.held, self.free, count, most, self.shared, seen)
        for _ in range(2):  # the same inputs again give the same
            got = nbw.kv_reserve(self.cache, ints(self.lens), ints(want), ints(self.held), self.free_t, ints([count]), most,
                                 shared=None if self.shared is None else ints(self.shared), seen=None if seen is None else ints(seen))
            names = ("table", "free", "cu", "positions", "slots", "granted", "held", "count")
            have = (self.wide[:, :self.width], self.free_t, got.cu, got.positions, got.slots, got.granted, got.held, got.count)
            for name, x, y in zip(names, have, ref):
                assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1)), name
            assert got.slots.dtype == torch.int64
        assert bool((self.wide[:, self.width:] == -7).all())
        return got, ref


@pytest.mark.parametrize("rows", [1, 2, 63, 300, 1024, 1025, 2500, 5000])
@pytest.mark.parametrize("page", [1, 8, 256])
def test_reserve_mixed_rows(nbw, rows, page):
    """Rows that grow, stay, shrink, end and start, with spare pages for all."""
    r = random.Random(rows * 7 + page)
    lens = [r.choice([0, 0, r.randrange(0, 6 * page + 1)]) for _ in range(rows)]
    held = [min(12, -(-n // page) + r.choice([0, 0, 0, 1, 3])) for n in lens]
    want = [r.choice([0, 1, 1, 5, r.randrange(0, 2 * page + 2)]) for _ in range(rows)]
    b = Book(nbw, lens, held, 12, page, spare=rows * 12, seed=rows, table_ld=17)
    b.check(nbw, want, sum(want) + 3)
    b.check(nbw, want, sum(want), seen=[r.randrange(0, 10**9) for _ in lens])


@pytest.mark.parametrize("rows,page", [(5, 8), (700, 16), (3000, 4)])
@pytest.mark.parametrize("part", [0.0, 0.3, 0.9])
def test_reserve_where_pages_or_places_run_out(nbw, rows, page, part):
    r = random.Random(rows + page)
    lens = [r.randrange(0, 5 * page) for _ in range(rows)]
    held = [-(-n // page) + (2 if i % 5 == 0 else 0) for i, n in enumerate(lens)]
    want = [r.choice([0, 1, page, 2 * page + 1]) for _ in range(rows)]
    lacking = sum(max(0, -(-(n + t) // page) - h) for n, t, h in zip(lens, want, held))
    back = sum(max(0, h - -(-(n + t) // page)) for n, t, h in zip(lens, want, held))
    b = Book(nbw, lens, held, 9, page, spare=max(0, int(lacking * part) - back), seed=rows)
    b.check(nbw, want, sum(want))
    b = Book(nbw, lens, held, 9, page, spare=lacking, seed=rows)
    got, _ = b.check(nbw, want, int(sum(want) * part))
    assert int(got.cu[-1]) <= int(sum(want) * part)


def test_reserve_pages_behind_a_shared_prefix_stay(nbw):
    lens, held, shared = [40, 0, 33, 70, 0], [5, 5, 6, 9, 4], [0, 4, 4, 4, 4]
    b = Book(nbw, lens, held, 12, 8, shared=shared)
    got, ref = b.check(nbw, [1, 0, 0, 4, 9], 20)
    assert got.held.tolist() == [6, 4, 5, 10, 4]


def test_reserve_given_back_at_once_leaves_all_as_it_was(nbw):
    lens, held, want = [30, 5, 0, 64], [4, 1, 0, 8], [9, 20, 17, 0]
    b = Book(nbw, lens, held, 12, 8)
    before = b.free_t.clone()
    got, _ = b.check(nbw, want, 50)
    back = nbw.kv_reserve(b.cache, ints(lens), ints([0] * 4), got.held, b.free_t, got.count, 0)
    assert back.held.tolist() == held and int(back.count) == b.spare
    assert torch.equal(b.free_t[:b.spare], before[:b.spare])
    again = nbw.kv_reserve(b.cache, ints(lens), ints(want), back.held, b.free_t, back.count, 50)
    assert torch.equal(again.slots, got.slots)


def test_reserve_bounds_what_it_is_told(nbw):
    """Lengths, wishes, holdings and counts out of their ranges, and pages that are in no pool."""
    lens, held = [-3, 10**9, 2**31 - 1, 20, 95, 0], [0, 3, 0, 99, 12, -4]
    b = Book(nbw, [0, 24, 0, 20, 95, 0], [0, 3, 0, 12, 12, 0], 12, 8, spare=9)
    b.table[1, 1] = 10**6
    b.wide[1, 1] = 10**6
    b.table[3, 5], b.wide[3, 5] = -5, -5
    b.lens, b.held = lens, held
    for want in ([3, 1, 5, -2, 1, 4], [2**31 - 1, 2**31 - 1, 0, 2**31 - 1, 2, 1]):
        b.check(nbw, want, 30)
    for count in (-4, 10**9):
        c = Book(nbw, [9, 17], [2, 4], 12, 8, spare=9, free_size=9)
        c.check(nbw, [1, 2], 5, count=count)


def test_reserve_without_rows_and_without_places(nbw):
    pool = torch.zeros((2, 1, 8, 64), dtype=BF16, device="cuda")
    cache = nbw.KVCache(pool, pool, torch.zeros((0, 3), dtype=torch.int32, device="cuda"))
    none = ints([])
    got = nbw.kv_reserve(cache, none, none, none, ints([1, 0, 5]), ints([2]), 4)
    assert got.cu.tolist() == [0] and got.slots.tolist() == [-1] * 4 and got.positions.tolist() == [0] * 4 and int(got.count) == 2
    b = Book(nbw, [3], [1], 4)
    b.check(nbw, [0], 0)
    b.check(nbw, [1], 0)


def test_reserve_in_a_graph(nbw):
    """Captured once, replayed with other lengths, eager work in between."""
    rows, page, width = 40, 16, 20
    b = Book(nbw, [0] * rows, [0] * rows, width, page, spare=rows * width)
    state = dict(lens=ints([0] * rows), want=ints([1] * rows), held=ints([0] * rows), count=ints([b.spare]))
    out = dict(cu=ints([0] * (rows + 1)), positions=ints([0] * 200), slots=ints([0] * 200, torch.int64), granted=ints([0] * rows),
               held_out=ints([0] * rows), count_out=ints([0]))

    def call():
        nbw.kv_reserve(b.cache, state["lens"], state["want"], state["held"], b.free_t, state["count"], 200, **out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b.wide.copy_(torch.from_numpy(b.table))  # as it was before the first call
    r = random.Random(3)
    table, free, lens, held, count = b.table, b.free, [0] * rows, [0] * rows, b.spare
    for step in range(6):
        want = [r.randrange(0, 6) for _ in range(rows)]
        lens = [max(0, n - r.randrange(0, 4)) if r.random() < 0.9 else 0 for n in lens]
        ref = okv.reserve(table, page, b.pages, lens, want, held, free, count, 200)
        state["lens"].copy_(ints(lens))
        state["want"].copy_(ints(want))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((b.wide[:, :width], b.free_t, out["cu"], out["positions"], out["slots"], out["granted"], out["held_out"],
                         out["count_out"]), ref):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1)), step
        table, free, _, _, _, granted, held, count = ref
        lens = [n + g for n, g in zip(lens, granted)]
        state["held"].copy_(out["held_out"])
        state["count"].copy_(out["count_out"])


# ---------------------------------------------------------------------------
# attention

class Shared:
    """Rows in groups that share a prefix, each with a tail and new tokens of its own; what belongs to no
    row is NaN (the cache's slots past every length, and a page of its own)."""

    def __init__(self, nbw, groups, q_heads, kv, dim=128, page=16, dtype=BF16, seed=0, spread=False, width=0):
        """groups: [(prefix, [(tail, new), ...]), ...]; tail counts the new tokens."""
        g = torch.Generator().manual_seed(seed)
        self.prefix = [p for p, _ in groups]
        self.lens = [p + t for p, rows in groups for t, _ in rows]
        self.new = [n for _, rows in groups for _, n in rows]
        self.bounds = np.concatenate([[0], np.cumsum([len(rows) for _, rows in groups])]).tolist()
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).tolist()
        group = [i for i, (_, rows) in enumerate(groups) for _ in rows]
        need = [-(-n // page) for n in self.lens]
        whole = [p // page for p in self.prefix]
        pages = sum(whole) + sum(n - whole[i] for n, i in zip(need, group)) + 1
        order = torch.randperm(pages - 1, generator=g).to(torch.int32).tolist()
        rows = len(need)
        self.table_np = np.full((rows, max(need + [1]) + width), 2**30, dtype=np.int32)
        at = 0
        for i, w in enumerate(whole):
            for r in range(self.bounds[i], self.bounds[i + 1]):
                self.table_np[r, :w] = order[at:at + w]
            at += w
        for r in range(rows):
            w = whole[group[r]]
            self.table_np[r, w:need[r]] = order[at:at + need[r] - w]
            at += need[r] - w
        self.k, self.v = (torch.full((pages, kv, page, dim), math.nan, dtype=dtype, device="cuda") for _ in "kv")
        self.scales = [None, None]
        if dtype == FP8:
            self.scales = [(torch.rand(kv, generator=g) * 0.02 + 0.01).cuda() for _ in "kv"]
        for r in range(rows):
            n = self.lens[r]
            first = self.prefix[group[r]] if r > self.bounds[group[r]] else 0
            slot = np.arange(n)
            pg = torch.from_numpy(self.table_np[r][slot // page].astype(np.int64)).cuda()
            place = torch.from_numpy(slot % page).cuda()
            lead = self.bounds[group[r]]
            for pool, by in ((self.k, self.scales[0]), (self.v, self.scales[1])):
                x = torch.randn(n, kv, dim, generator=g).cuda()
                x = (x / by[None, :, None]).clamp(-448, 448) if by is not None else x
                x = x.to(dtype)
                if first:  # the first row's own bits
                    lp = torch.from_numpy(self.table_np[lead][slot[:first] // page].astype(np.int64)).cuda()
                    x.view(torch.uint8)[:first] = pool.view(torch.uint8)[lp, :, place[:first]]
                pool.view(torch.uint8)[pg, :, place] = x.view(torch.uint8)
        self.cache = nbw.KVCache(self.k, self.v, torch.from_numpy(self.table_np).cuda(), *self.scales)
        tokens = self.cu[-1]
        wide = torch.randn(tokens, q_heads * dim + (64 if spread else 0), generator=g).mul_(2).to(BF16).cuda()
        self.q = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim))
        self.nbw, self.group, self.page, self.dim = nbw, group, page, dim

    def call(self, **kw):
        kw.setdefault("cu", ints(self.cu))
        if any(self.prefix):
            kw.update(groups=ints(self.bounds), prefix=ints(self.prefix))
        return self.nbw.kv_attend_shared(self.cache, self.q, ints(self.lens), **kw)

    def pools(self):
        k, v = f64(self.k), f64(self.v)
        if self.scales[0] is not None:
            k, v = k * f64(self.scales[0])[None, :, None, None], v * f64(self.scales[1])[None, :, None, None]
        return k, v

    def check(self, out, scale=None, tokens=None):
        """Scores in fp32 are off by the sum of dim products, each off by 2^-24 of what is summed (16 times allowed for
        dims of 64 to 256 summed in blocks), which moves a weight by that, relatively; a weight is rounded to bf16, half a step
        of 2^-8 (2^-9), and divided by the sum of such: a change of at most 2^-8 of each weight beside the others in all;
        the result is rounded to bf16, 2^-8 of itself at most."""
        k, v = self.pools()
        q = f64(self.q)
        scale = self.dim ** -0.5 if scale is None else scale
        want = okv.attend_tokens(q, k, v, self.table_np, self.lens, self.cu, scale)
        mean = okv.attend_tokens(q, k, np.abs(v), self.table_np, self.lens, self.cu, scale)
        with np.errstate(invalid="ignore"):
            size = np.abs(q).sum(axis=2).max() * np.nanmax(np.abs(k[np.isfinite(k)])) * abs(scale)
            bound = 2.0**-8 * np.abs(want) + (2.0**-8 + 2 * 16 * 2.0**-24 * size) * mean + 1e-30
            got = f64(out)
            ok = (np.abs(got - want) <= bound) | (got == want) | (np.isnan(got) & np.isnan(want))
        assert ok.all(), (float(np.nanmax(np.abs(got - want) / bound)), np.argwhere(~ok)[:4].tolist())
        return want


ONE = [(0, [(1, 1)])]
GROUPS = {
    "one token alone": ONE,
    "one row, several tokens": [(0, [(70, 5)])],
    "only new tokens": [(0, [(7, 7), (1, 1)])],
    "a batch behind one prefix": [(100, [(1, 1), (17, 1), (40, 1)])],
    "prefix inside a page, drafts": [(37, [(6, 5), (3, 3), (33, 1), (2, 2)])],
    "two groups and a row alone": [(64, [(9, 2), (1, 1)]), (0, [(50, 4)]), (130, [(20, 1), (5, 5)])],
    "idle rows": [(48, [(12, 0), (3, 1), (0, 0)]), (16, [(4, 0)]), (33, [(1, 1)])],
    "many tokens": [(90, [(150, 130), (41, 40)])],
    "long": [(1500, [(300, 3), (700, 2), (1, 1)])],
}


@pytest.mark.parametrize("which", list(GROUPS))
@pytest.mark.parametrize("q_heads,kv,dim,page,dtype", [(8, 2, 128, 16, BF16), (3, 3, 64, 8, BF16), (12, 1, 64, 1, FP8), (10, 2, 256, 32, BF16),
                                                        (8, 1, 128, 128, FP8), (40, 2, 256, 4, FP8), (14, 2, 64, 64, FP8)])
def test_attend_shared(nbw, which, q_heads, kv, dim, page, dtype):
    print(which, q_heads, kv, dim, page, dtype, flush=True)
    s = Shared(nbw, GROUPS[which], q_heads, kv, dim, page, dtype, seed=len(which), spread=q_heads == 8)
    out = s.call()
    s.check(out)
    assert torch.equal(out, s.call())


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_attend_shared_lengths_around_every_boundary(nbw, n):
    s = Shared(nbw, [(n, [(1, 1), (n, 1)]), (0, [(n, min(n, 3))])], 8, 2, 64, 8, seed=n)
    s.check(s.call())


def test_attend_shared_one_token_a_row_without_cu(nbw):
    s = Shared(nbw, [(40, [(5, 1), (30, 1)]), (0, [(9, 1)])], 8, 2)
    assert torch.equal(s.call(cu=None), s.call())
    t = Shared(nbw, [(0, [(45, 1)]), (0, [(9, 1)])], 8, 2)
    assert torch.allclose(t.call(cu=None).float(), nbw.kv_attend(t.cache, t.q, ints(t.lens)).float(), atol=2.0**-6, rtol=2.0**-6)


@pytest.mark.parametrize("scale", [0.5, -0.125, 1e-20])
def test_attend_shared_scales(nbw, scale):
    s = Shared(nbw, [(40, [(5, 2), (300, 1)])], 8, 2)
    s.check(s.call(scale=scale), scale)


def at(s, row, slot):
    return int(s.table_np[row, slot // s.page]), slice(None), slot % s.page


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 4), (256, 64)])
def test_attend_shared_what_a_token_does_not_see_has_no_part(nbw, bad, dim, page):
    """A value that later drafts see and earlier ones do not: NaN or infinite for the ones, nothing for the others."""
    s = Shared(nbw, [(70, [(6, 5), (40, 4)]), (0, [(130, 9)])], 4, 2, dim, page)
    for row in range(3):
        n = s.lens[row]
        s.v[at(s, row, n - 1)] = bad
        s.v[at(s, row, n - 3)][..., 5] = -bad
        s.k[at(s, row, n - 2)] = math.nan
    out = f64(s.call())
    want = s.check(s.call())
    for row in range(3):
        first, end = s.cu[row], s.cu[row + 1]
        assert np.isfinite(out[first:end - 3]).all() and np.isnan(out[end - 2:end]).all()
    assert np.isfinite(want).any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attend_shared_infinite_values_that_all_see(nbw, bad):
    s = Shared(nbw, [(600, [(3, 2), (50, 1)])], 8, 2)
    s.v[at(s, 0, 300)][..., 3] = bad
    s.v[at(s, 1, s.lens[1] - 1)][..., 7] = -bad
    out = f64(s.call())
    assert np.array_equal(out[:, :, 3], np.full(out.shape[:2], bad), equal_nan=True)
    assert np.array_equal(out[2, :, 7], np.full(8, -bad), equal_nan=True) and np.isfinite(out[:2, :, 7]).all()


def test_attend_shared_heads_without_a_score_give_zeros(nbw):
    """All keys of a row's slots are -infinity for positive queries: zeros, whatever the values."""
    s = Shared(nbw, [(90, [(8, 2)]), (0, [(30, 1)])], 4, 2, 64, 8)
    s.q.copy_(s.q.abs().add(0.1))
    for j in range(s.lens[0]):
        s.k[at(s, 0, j)][..., 0] = -math.inf
        s.v[at(s, 0, j)][..., 1] = math.inf if j % 2 else math.nan
    out = s.call()
    assert bool((out[:2] == 0).all()) and bool(out[2].isfinite().all())


def test_attend_shared_equal_values_average_exactly(nbw):
    s = Shared(nbw, [(700, [(9, 3), (200, 1)])], 8, 2)
    s.v[~s.v.isnan()] = 1.3359375
    assert bool((s.call() == 1.3359375).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_shared_values_near_the_largest_finite_one(nbw, dim):
    s = Shared(nbw, [(700, [(9, 3), (200, 1)]), (0, [(1, 1)])], 8, 2, dim)
    s.v[~s.v.isnan()] = 3.3e38
    s.check(s.call())
    s.v[..., ::2] *= -1
    s.check(s.call())


def test_attend_shared_large_scores(nbw):
    """Scores of thousands, rising slot by slot, falling, and all equal."""
    s = Shared(nbw, [(500, [(9, 3), (200, 1)])], 8, 2)
    s.q.fill_(8.0)
    for row in (1, 0):
        for j in range(s.lens[row]):
            s.k[at(s, row, j)] = (j if row else -j) / 16.0
    s.check(s.call())
    s.k[~s.k.isnan()] = 7.0
    s.check(s.call())


def test_attend_shared_pages_that_are_not_there(nbw):
    s = Shared(nbw, [(64, [(40, 2), (70, 1)])], 8, 2)
    s.table_np[:, 1] = -1
    s.table_np[0, 5] = 2**30
    s.cache.table.copy_(torch.from_numpy(s.table_np))
    s.check(s.call())
    s.table_np[:] = -1
    s.cache.table.copy_(torch.from_numpy(s.table_np))
    assert bool((s.call() == 0).all())


def test_attend_shared_rows_shorter_than_the_prefix(nbw):
    """A group's row may be cut within its prefix, or hold nothing; its new tokens see what there is."""
    s = Shared(nbw, [(100, [(9, 2), (30, 2), (4, 1), (5, 3)])], 8, 2)
    s.lens[1], s.lens[2], s.lens[3] = 50, 0, 2
    out = s.call()
    s.check(out)
    assert bool((out[s.cu[2]:s.cu[3]] == 0).all()) and bool((out[s.cu[3]:s.cu[3] + 1] == 0).all())


def test_attend_shared_bounds_what_it_is_told(nbw):
    s = Shared(nbw, [(40, [(8, 2), (8, 1)])], 8, 2, page=16)
    want = s.call()
    cap = s.cache.capacity
    assert cap == 48
    for prefix in (10**9, -5):
        got = nbw.kv_attend_shared(s.cache, s.q, ints(s.lens), cu=ints(s.cu), groups=ints([0, 1, 2]), prefix=ints([prefix, prefix]))
        assert torch.allclose(got.float(), want.float(), atol=2.0**-6, rtol=2.0**-6)
    s.lens = [2**31 - 1, -4]
    out = s.call()
    assert bool((out[2] == 0).all()) and torch.allclose(out[:2].float(), want[:2].float(), atol=2.0**-6, rtol=2.0**-6)
    # a bound of the lengths cuts the rows
    s.lens = [48, 48]
    got = s.call(max_len=30)
    s.lens = [30, 30]
    s.check(got)


def test_attend_shared_leaves_tokens_of_no_row(nbw):
    s = Shared(nbw, [(40, [(8, 2), (8, 1)])], 8, 2)
    q = torch.cat([s.q, torch.full_like(s.q[:2], math.nan)])
    out = torch.full_like(q, 5.0)
    got = nbw.kv_attend_shared(s.cache, q, ints(s.lens), cu=ints(s.cu), groups=ints(s.bounds), prefix=ints(s.prefix), out=out)
    assert got is out and bool((out[3:] == 5).all()) and torch.equal(out[:3], s.call())


def test_attend_shared_rows_in_no_group(nbw):
    """Groups that end before the last row, and begin after the first."""
    s = Shared(nbw, [(0, [(30, 1)]), (40, [(8, 2), (8, 1)]), (0, [(60, 2)])], 8, 2)
    got = nbw.kv_attend_shared(s.cache, s.q, ints(s.lens), cu=ints(s.cu), groups=ints([1, 3]), prefix=ints([40]))
    s.check(got)


def test_attend_shared_nothing_to_do(nbw):
    pool = torch.zeros((2, 1, 8, 64), dtype=BF16, device="cuda")
    cache = nbw.KVCache(pool, pool, torch.zeros((0, 3), dtype=torch.int32, device="cuda"))
    assert nbw.kv_attend_shared(cache, torch.zeros((0, 4, 64), dtype=BF16, device="cuda"), ints([])).shape == (0, 4, 64)
    s = Shared(nbw, [(8, [(3, 0), (4, 0)])], 4, 1, 64, 8)
    assert s.call().shape == (0, 4, 64)


def test_attend_shared_strided_out_other_streams_and_own_workspace(nbw):
    s = Shared(nbw, [(300, [(9, 3), (200, 1)]), (0, [(50, 2)])], 8, 2)
    want = s.call()
    room = torch.full((6, 8 * 128 + 72), 3.0, dtype=BF16, device="cuda")
    assert torch.equal(s.call(out=room[:, :1024].unflatten(1, (8, 128))), want) and bool((room[:, 1024:] == 3).all())
    ws = torch.full((s.cache.attend_shared_workspace_bytes(8, 6, 2) + 512,), 255, dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(s.call(workspace=ws[:-512].contiguous() if i % 2 else "auto"))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got) and bool((ws[-512:] == 255).all())


def test_attend_shared_in_a_graph(nbw):
    """Captured once with a workspace of its own, replayed with other lengths and eager work in between."""
    s = Shared(nbw, [(200, [(90, 2), (140, 3), (60, 1)]), (0, [(100, 2)])], 8, 2)
    lens, prefix, cu, bounds = ints(s.lens), ints(s.prefix), ints(s.cu), ints(s.bounds)
    ws = torch.empty(s.cache.attend_shared_workspace_bytes(8, 8, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(s.q)

    def call():
        nbw.kv_attend_shared(s.cache, s.q, lens, cu=cu, groups=bounds, prefix=prefix, out=out, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for less in (0, 10, 33, 60, 3):
        s.lens = [n - less for n in (290, 340, 260, 100)]
        lens.copy_(ints(s.lens))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = s.call()
        assert torch.equal(out, want)
        s.check(out)


def test_attend_shared_pools_past_two_to_the_31(nbw):
    """Pages whose elements lie past 2^31."""
    page, kv, dim = 4096, 8, 128
    pages = 2**31 // (page * kv * dim) + 3
    k = torch.zeros((pages, kv, page, dim), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for pool in (k, v):
        pool[-2:] = torch.randn(pool[-2:].shape, generator=g, device="cuda").to(BF16)
    table = ints([[pages - 1, pages - 2], [pages - 1, pages - 2]])
    cache = nbw.KVCache(k, v, table)
    small = nbw.KVCache(k[-2:].clone(), v[-2:].clone(), ints([[1, 0], [1, 0]]))
    q = torch.randn((4, 8, dim), generator=g, device="cuda").to(BF16)
    kw = dict(cu=ints([0, 1, 4]), groups=ints([0, 2]), prefix=ints([5000]))
    lens = ints([6000, 5003])
    assert torch.equal(nbw.kv_attend_shared(cache, q, lens, **kw), nbw.kv_attend_shared(small, q, lens, **kw))


# ---------------------------------------------------------------------------
# verification

def probs(g, tokens, vocab, dtype, sharp=3.0):
    return torch.softmax(torch.randn(tokens, vocab, generator=g).mul_(sharp), dim=1).to(dtype)


def check_verify(nbw, target, ids, u, cu, draft=None, **kw):
    want = odrafts.verify(f64(target), ids.tolist(), f64(u), cu, None if draft is None else f64(draft))
    cuda = [x.cuda() if x is not None and not x.is_cuda else x for x in (target, ids, u, draft)]
    got = nbw.verify_drafts(cuda[0], cuda[1], cuda[2], draft=cuda[3], cu=ints(cu), **kw)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1], (got, want)
    return want


@pytest.mark.parametrize("vocab", [1, 2, 3, 17, 255, 1000, 4095, 4096, 4097, 9001])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify(nbw, vocab, dtype, sampled):
    g = torch.Generator().manual_seed(vocab)
    counts = [3, 1, 6, 0, 2, 9, 1, 4]
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    tokens = cu[-1]
    target = probs(g, tokens, vocab, dtype)
    draft = (target.float() * torch.exp(0.6 * torch.randn(tokens, vocab, generator=g))) if sampled else None
    if sampled:
        draft = (draft / draft.sum(dim=1, keepdim=True)).to(dtype)
    for seed in range(4):
        near = (target if draft is None else draft).float().argmax(dim=1)
        ids = torch.where(torch.rand(tokens, generator=g) < 0.8, near.roll(1), torch.randint(0, vocab, (tokens,), generator=g))
        check_verify(nbw, target, ids.to(torch.int32), torch.rand(tokens, generator=g), cu, draft)


def test_verify_a_long_run_of_drafts_and_one_row_after_it(nbw):
    g = torch.Generator().manual_seed(1)
    cu = [0, 200, 201, 330]
    target = probs(g, 330, 50, torch.float32)
    ids = torch.randint(0, 50, (330,), generator=g, dtype=torch.int32)
    for stop in (0, 1, 62, 63, 64, 65, 127, 128, 198, 199):
        u = torch.zeros(330)
        u[stop] = 1.0
        want = check_verify(nbw, target, ids, u, cu, target)
        assert want[0][0] == min(stop, 199)


def test_verify_the_comparison_is_exact(nbw):
    """u q against p next to it: numbers of 24 bits whose product fp32 cannot hold, equality is a refusal."""
    g = torch.Generator().manual_seed(2)
    tokens, vocab = 400, 3
    u, q = torch.rand(tokens, generator=g), torch.rand(tokens, vocab, generator=g) * 0.5 + 0.01
    p = (u[:, None].double() * q.double()).float()  # within half a step of the product
    p[::5] = q[::5]
    u[::5] = 1.0
    cu = list(range(0, tokens + 1, 2))
    ids = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    want = check_verify(nbw, p, ids, u, cu, q)
    assert 20 < sum(want[0]) < 180


@pytest.mark.parametrize("u", [0.0, 2.0**-24, 0.25, 0.5, 1 - 2.0**-24, 1.0, 2.0, -1.0, math.nan, math.inf])
def test_verify_numbers_at_and_out_of_their_ends(nbw, u):
    """Equal weights of a power of two: the running sums are exact and meet u times the whole."""
    target = torch.zeros(2, 1 << 13)
    target[:, 100:100 + 4096] = 2.0**-12
    check_verify(nbw, target, ints([0, 0]).cpu(), torch.tensor([u, u]), [0, 1, 2])
    check_verify(nbw, target, ints([0, 200]).cpu(), torch.tensor([u, u]), [0, 2])


def test_verify_weights_that_are_none(nbw):
    """Equal distributions that refuse, lines of zeros, negative, infinite and NaN numbers, tokens out of the vocabulary."""
    g = torch.Generator().manual_seed(4)
    vocab = 70
    target = probs(g, 14, vocab, torch.float32)
    draft = target.clone()
    target[2], draft[2] = 0.0, 0.0
    target[4, ::3], draft[4, 1::3] = math.nan, math.inf
    target[6, 5], target[6, 6], draft[6, 7] = math.inf, -2.0, math.nan
    target[8] = -target[8]
    target[10], draft[10] = math.nan, math.nan
    ids = torch.tensor([0, 5, 0, 6, 0, 9, 0, 7, 0, 9, 0, 3, 0, 10**6], dtype=torch.int32)
    u = torch.full((14,), 0.999)
    u[0::2] = 1.0
    u[8] = -0.5
    cu = list(range(0, 15, 2))
    for d in (draft, None):
        want = check_verify(nbw, target, ids, u, cu, d)
        assert want[1][1] == -1 and want[1][5] == -1
    ids[13] = -1
    check_verify(nbw, target, ids, u, cu, None)
    check_verify(nbw, target, ids, torch.full((14,), math.nan), cu, draft)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_verify_strided_lines_at_any_address(nbw, dtype):
    g = torch.Generator().manual_seed(5)
    tokens, vocab = 9, 5003
    for off in (0, 1, 3):
        room = [torch.full((tokens, vocab + 7), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
        t, d = room[0][:, off:off + vocab], room[1][:, 2:2 + vocab]
        t.copy_(probs(g, tokens, vocab, dtype))
        d.copy_(probs(g, tokens, vocab, dtype, 2.5))
        ids = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
        check_verify(nbw, t, ids, torch.rand(tokens, generator=g), [0, 4, 5, 9], d)


def test_verify_without_cu_samples_each_line(nbw):
    g = torch.Generator().manual_seed(6)
    target = probs(g, 40, 6000, torch.float32)
    u = torch.rand(40, generator=g)
    want = odrafts.verify(f64(target), [0] * 40, f64(u), list(range(41)))
    accepted, after = nbw.verify_drafts(target.cuda(), None, u.cuda())
    assert accepted.tolist() == [0] * 40 and after.tolist() == want[1]


def test_verify_follows_the_targets_distribution(nbw):
    """Tokens from a draft's distribution, verified, are distributed as the target says: over 60000 rows the share of each
    of 5 tokens is within 5 standard deviations, sqrt(p (1 - p) / 60000), of its probability."""
    rows, p, q = 60000, torch.tensor([0.4, 0.1, 0.25, 0.05, 0.2]), torch.tensor([0.1, 0.3, 0.3, 0.2, 0.1])
    g = torch.Generator(device="cuda").manual_seed(7)
    drafted = torch.multinomial(q.cuda(), rows, replacement=True, generator=g).to(torch.int32)
    ids = torch.stack([torch.zeros_like(drafted), drafted], dim=1).reshape(-1)
    u = torch.rand(2 * rows, generator=g, device="cuda")
    accepted, after = nbw.verify_drafts(p.cuda().repeat(2 * rows, 1), ids, u, draft=q.cuda().repeat(2 * rows, 1),
                                        cu=torch.arange(0, 2 * rows + 1, 2, dtype=torch.int32, device="cuda"))
    first = torch.where(accepted == 1, drafted, after)
    share = torch.bincount(first, minlength=5).double().cpu() / rows
    assert bool(((share - p).abs() <= 5 * (p * (1 - p) / rows).sqrt()).all()), share
    assert abs(float(accepted.double().mean()) - float(torch.minimum(p, q).sum())) < 0.011


def test_verify_bounds_the_rows_it_is_told(nbw):
    g = torch.Generator().manual_seed(8)
    target = probs(g, 5, 300, torch.float32)
    ids, u = torch.zeros(5, dtype=torch.int32), torch.rand(5, generator=g)
    got = nbw.verify_drafts(target.cuda(), ids.cuda(), u.cuda(), cu=ints([-3, 2, 1, 10**9, 10**9]))
    want = odrafts.verify(f64(target), ids.tolist(), f64(u), [0, 2, 2])
    tail = odrafts.verify(f64(target), ids.tolist(), f64(u), [1, 5])
    assert got[0].tolist() == want[0] + tail[0] + [0] and got[1].tolist() == want[1] + tail[1] + [-1]


def test_verify_own_workspace_streams_and_a_graph(nbw):
    from nested_bit_weight_amd import drafts
    g = torch.Generator().manual_seed(9)
    cu, vocab = [0, 4, 5, 9], 20000
    target, draft = (probs(g, 9, vocab, torch.float32, x).cuda() for x in (3.0, 2.5))
    ids = torch.randint(0, vocab, (9,), generator=g, dtype=torch.int32).cuda()
    ids[1:] = draft.argmax(dim=1)[:-1].to(torch.int32)
    u, cut = torch.rand(9, generator=g).cuda(), ints(cu)
    ws = torch.empty(drafts.verify_workspace_bytes(3, vocab), dtype=torch.uint8, device="cuda")
    out = [ints([0] * 3), ints([0] * 3)]

    def call():
        nbw.verify_drafts(target, ids, u, draft=draft, cu=cut, accepted=out[0], next=out[1], workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        u.copy_(torch.rand(9, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        have = [x.tolist() for x in out]
        with torch.cuda.stream(side):
            eager = check_verify(nbw, target, ids.cpu(), u.cpu(), cu, draft)
        assert have == [eager[0], eager[1]]


def test_verify_large_vocabulary(nbw):
    g = torch.Generator().manual_seed(10)
    target = probs(g, 3, 160001, torch.float32)
    check_verify(nbw, target, torch.zeros(3, dtype=torch.int32), torch.rand(3, generator=g), [0, 1, 3])


# ---------------------------------------------------------------------------
# another device's tensors, and none

def test_everything_goes_with_the_tensors_device(nbw):
    if torch.cuda.device_count() < 2:
        with torch.cuda.device(0):
            s = Shared(nbw, [(8, [(3, 1)])], 4, 1, 64, 8)
            s.check(s.call())
        return
    with torch.cuda.device(1):
        s = Shared(nbw, [(8, [(3, 1)])], 4, 1, 64, 8)
    s.check(s.call())
