"""More GPU checks of a step with drafted tokens: many rows, long pasts, scratch shared in turn, large vocabularies.

The checks and their tolerances are those of test_gpu_drafts.py.
"""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

from nested_bit_weight_amd import kv
from oracle import drafts as odrafts
from test_gpu_drafts import BF16, FP8, Shared, f64, ints, nbw  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("new", [1, 3])
def test_attend_shared_thousands_of_rows_in_groups(nbw, new):  # noqa: F811
    """More rows and groups than are kept together, most of the rows idle, and long runs of such between others."""
    r = random.Random(new)
    groups = []
    for i in range(1300):
        idle = 100 < i < 420 or r.random() < 0.5
        rows = [(0 if idle else r.randrange(1, 30), 0 if idle else new) for _ in range(2)]
        groups.append((r.choice([0, 4, 11]), [(max(t, n), n) for t, n in rows]))
    s = Shared(nbw, groups, 2, 1, 64, 4, seed=new)
    s.check(s.call())


def test_attend_shared_one_token_over_a_long_past(nbw):  # noqa: F811
    """More pieces of one line than the last launch looks at together, with and without a prefix."""
    for groups in ([(0, [(60000, 1)])], [(50001, [(1, 1), (9000, 2)])]):
        s = Shared(nbw, groups, 2, 1, 64, 64, seed=3)
        s.check(s.call())


@pytest.mark.parametrize("page", [1, 2, 1024, 4096])
def test_attend_shared_small_and_large_pages(nbw, page):  # noqa: F811
    s = Shared(nbw, [(300, [(200, 2), (3, 1)]), (0, [(900, 5)])], 4, 2, 128, page, seed=page)
    s.check(s.call())


@pytest.mark.parametrize("q_heads,heads", [(256, 1), (5, 5), (96, 2)])
def test_attend_shared_head_groups(nbw, q_heads, heads):  # noqa: F811
    s = Shared(nbw, [(70, [(65, 1), (1, 1), (30, 4)])], q_heads, heads, 64, 8, seed=q_heads)
    s.check(s.call())


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, FP8), (256, BF16), (256, FP8)])
def test_attend_shared_all_tokens_of_long_rows(nbw, dim, dtype):  # noqa: F811
    s = Shared(nbw, [(0, [(400, 400)]), (190, [(333, 333), (20, 1)])], 2, 1, dim, 16, dtype, seed=dim)
    s.check(s.call())


@pytest.mark.parametrize("prefix", [0, 20])
@pytest.mark.parametrize("rows,new,tail,q_heads,heads", [(70, 40, 60, 8, 8), (300, 1, 200, 2, 2), (90, 3, 300, 24, 6)])
def test_attend_shared_more_rows_than_workgroups_take_at_once(nbw, rows, new, tail, q_heads, heads, prefix):  # noqa: F811
    """Short rows of many sizes, several of them a workgroup's."""
    r = random.Random(rows)
    sizes = [(max(n, r.randrange(1, tail)), n) for n in (r.randrange(0, new + 1) for _ in range(rows))]
    s = Shared(nbw, [(prefix, sizes)], q_heads, heads, 64, 16, seed=rows + prefix)
    s.check(s.call())


def test_attend_shared_a_table_of_which_part_is_used(nbw):  # noqa: F811
    s = Shared(nbw, [(48, [(6, 5), (33, 1)])], 4, 2, 128, 16, seed=8)
    wide = torch.full((s.table_np.shape[0], 50), -5, dtype=torch.int32, device="cuda")
    wide[:, :s.table_np.shape[1]] = s.cache.table
    s.cache = nbw.KVCache(s.k, s.v, wide[:, :s.table_np.shape[1]])
    s.check(s.call())


@pytest.mark.parametrize("scale", [1e-30, 3e-38])
def test_attend_shared_scales_that_vanish_beside_the_cache_s_own(nbw, scale):  # noqa: F811
    """scale times the keys' factor is below the smallest fp32 number: equal weights, and what is not seen has none."""
    s = Shared(nbw, [(37, [(6, 5), (33, 1)])], 4, 2, 128, 16, FP8, seed=9)
    s.scales[0].fill_(1e-20)
    s.check(s.call(scale=scale), scale)


def test_attend_shared_lengths_past_max_len_are_cut(nbw):  # noqa: F811
    s = Shared(nbw, [(0, [(300, 2), (40, 1)])], 4, 2, 64, 16, seed=10)
    out = s.call(max_len=100)
    s.lens = [min(n, 100) for n in s.lens]
    s.check(out)


def test_attend_shared_is_the_same_every_time(nbw):  # noqa: F811
    s = Shared(nbw, [(1300, [(70, 5), (3, 3), (900, 1)] * 4), (0, [(2000, 40)])], 8, 2, 128, 16, seed=11)
    first = s.call()
    for _ in range(20):
        assert torch.equal(s.call(), first)
    s.check(first)


def test_attend_shared_two_graphs_with_one_workspace_in_turn(nbw):  # noqa: F811
    cases = [Shared(nbw, [(90, [(70, 5), (3, 3)])], 8, 2, 128, 16, seed=12), Shared(nbw, [(0, [(700, 2), (1, 1)])], 8, 2, 128, 16, seed=13)]
    need = max(s.cache.attend_shared_workspace_bytes(8, s.cu[-1], len(s.prefix)) for s in cases)
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    runs = []
    for s in cases:
        out = torch.zeros_like(s.q)
        kw = dict(cu=ints(s.cu), out=out, workspace=workspace)
        if any(s.prefix):
            kw.update(groups=ints(s.bounds), prefix=ints(s.prefix))
        lens = ints(s.lens)
        nbw.kv_attend_shared(s.cache, s.q, lens, **kw)
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nbw.kv_attend_shared(s.cache, s.q, lens, **kw)
        runs.append((s, graph, out, want, kw, lens))
    for turn in range(6):
        for s, graph, out, want, _, _ in runs:
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), turn
    for s, _, _, want, _, _ in runs:
        s.check(want)


def test_the_operators_on_two_streams_at_once(nbw):  # noqa: F811
    s = Shared(nbw, [(1300, [(70, 5), (3, 3), (900, 1)])], 8, 2, 128, 16, seed=14)
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn(64, 50001, generator=g, device="cuda") * 3, dim=1)
    u = torch.rand(64, generator=g, device="cuda")
    cu, lens, groups, prefix = ints(s.cu), ints(s.lens), ints(s.bounds), ints(s.prefix)
    want, tokens = s.call(), nbw.verify_drafts(p, None, u)[1]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for _ in range(10):
        for stream in streams:
            with torch.cuda.stream(stream):
                got.append((nbw.kv_attend_shared(s.cache, s.q, lens, cu=cu, groups=groups, prefix=prefix),
                            nbw.verify_drafts(p, None, u)[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, tokens) for a, b in got)


def test_attend_shared_scratch_that_is_missing_or_short_and_pools_past_its_numbers(nbw):  # noqa: F811
    """Refused on the host; the sizes depend on the device, which is why this is no test without one."""
    fake = 0x7F0000001000  # never dereferenced

    def cache(**kw):
        return kv.KVView(**{**dict(k=fake, v=fake, pages=10, heads=2, page=16, dim=128, dtype=0, table=fake, rows=3, width=5, table_ld=0), **kw})

    def size(c, *a):
        return nbw.library().nbw_kv_attend_shared_workspace_bytes(ctypes.byref(c), *a)

    def call(c, **kw):
        a = kv.AttendSharedArgs(**{**dict(q=fake, out=fake, tokens=3, q_heads=16, lens=fake), **kw})
        return nbw.library().nbw_kv_attend_shared(ctypes.byref(c), ctypes.byref(a), None)

    einval, escratch = 1, 6
    need = size(cache(), 16, 3, 0, 0)
    assert 0 < need < size(cache(), 16, 3, 2, 0)
    assert call(cache()) == escratch and call(cache(), workspace=fake, workspace_bytes=need - 1) == escratch
    # a pool of 2^32 pieces of 8 elements: 64 GiB of bf16
    big = dict(pages=1 << 20, heads=32, page=16, dim=64)
    assert size(cache(**{**big, "pages": (1 << 20) - 1}), 32, 3, 0, 0) > 0
    assert size(cache(**big), 32, 3, 0, 0) == -1
    assert call(cache(**big), q_heads=32, workspace=fake, workspace_bytes=1 << 40) == einval
    # 2^20 rows that may each be as long as the capacity, and bounded by max_len
    many = cache(rows=1 << 20, width=1 << 16, pages=1 << 20)
    assert size(many, 2, 1 << 20, 0, 0) == -1 and size(many, 2, 1 << 20, 0, 4096) > 0


# ---------------------------------------------------------------------------
# verification

def verified(nbw, target, ids, u, cu, draft):  # noqa: F811
    got = nbw.verify_drafts(target, ints(ids), torch.tensor(u, dtype=torch.float32, device="cuda"), draft=draft, cu=ints(cu))
    ref = odrafts.verify(f64(target), ids, f64(torch.tensor(u, dtype=torch.float32)), cu, None if draft is None else f64(draft))
    assert got[0].tolist() == ref[0]
    assert got[1].tolist() == ref[1]
    return ref


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify_more_spans_than_a_wave_keeps(nbw, dtype, sampled):  # noqa: F811
    vocab, cu = 300001, [0, 1, 4, 6]
    g = torch.Generator(device="cuda").manual_seed(2)
    target, draft = (torch.softmax(torch.randn(6, vocab, generator=g, device="cuda"), dim=1).to(dtype) for _ in "pq")
    draft = draft if sampled else None
    for u in (0.0, 0.1, 0.5, 0.999):
        verified(nbw, target, [0, 1, 299999, 300000, 5, 300000], [0.5, 0.0, 0.99, u, 0.999, u], cu, draft)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_verify_no_difference_above_zero(nbw, dtype):  # noqa: F811
    """p where q is nowhere below it: the sums of p are formed in the second launch, over many spans."""
    vocab = 270000
    g = torch.Generator(device="cuda").manual_seed(3)
    target = torch.softmax(torch.randn(4, vocab, generator=g, device="cuda"), dim=1).to(dtype)
    target[:, 7] = 0
    draft = target * 2
    for u in (0.0, 0.25, 0.9999):
        ref = verified(nbw, target, [1, 7, 1, 7], [0.5, u, 0.5, u], [0, 2, 4], draft)
        assert ref[0] == [0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify_weights_that_are_none_anywhere_in_a_line(nbw, dtype, sampled):  # noqa: F811
    vocab = 5000
    g = torch.Generator(device="cuda").manual_seed(4)
    target, draft = (torch.rand(9, vocab, generator=g, device="cuda").to(dtype) for _ in "pq")
    for i, bad in enumerate([math.nan, math.inf, -math.inf, -1.0]):
        for t, x in ((target, i), (draft, i + 4)):
            t[x, [0, 17, 1023, 1024, 2500, 4999]] = bad
    u = torch.rand(9, generator=g, device="cuda").tolist()
    draft = draft if sampled else None
    verified(nbw, target, [-1] * 9, u, list(range(10)), None)        # every line sampled from
    verified(nbw, target, [0] * 9, u, [0, 2, 4, 6, 9], draft)        # drafts whose own numbers are such
    verified(nbw, target, [30] * 9, [1.0] * 8 + [0.5], [0, 2, 4, 6, 9], draft)


def test_verify_a_token_left_out_at_the_ends_of_spans(nbw):  # noqa: F811
    vocab = 3000
    target = torch.zeros(2, vocab, device="cuda")
    for x in (0, 1, 1022, 1023, 1024, 2047, 2048, 2999):
        target[:] = 0
        target[:, [x, (x + 1) % vocab]] = 0.5
        for u in (0.0, 0.7):
            assert verified(nbw, target, [0, x], [0.9, u], [0, 2], None)[1] == [(x + 1) % vocab]


def test_verify_thousands_of_rows(nbw):  # noqa: F811
    r = random.Random(5)
    new = [r.choice([0, 1, 1, 2, 5, 70]) for _ in range(2500)]
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    g = torch.Generator(device="cuda").manual_seed(5)
    target, draft = (torch.softmax(torch.randn(cu[-1], 40, generator=g, device="cuda"), dim=1) for _ in "pq")
    ids = torch.randint(0, 40, (cu[-1],), generator=g, device="cuda").tolist()
    u = torch.rand(cu[-1], generator=g, device="cuda").tolist()
    verified(nbw, target, ids, u, cu, draft)
    verified(nbw, target, ids, u, cu, None)


# ---------------------------------------------------------------------------
# reservation

def test_reserve_a_batch_that_starts_and_ends_at_once(nbw):  # noqa: F811
    """Every row takes pages, then every row gives them back."""
    rows, page = 20000, 16
    pool = torch.zeros((2 * rows, 1, page, 64), dtype=BF16, device="cuda")
    table = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    cache = nbw.KVCache(pool, pool, table)
    free = torch.randperm(2 * rows, device="cuda").to(torch.int32)
    zero, count, before = ints([0] * rows), ints([2 * rows]), free.clone()
    got = nbw.kv_reserve(cache, zero, zero + 20, zero, free, count, rows * 20)
    assert int(got.count) == 0 and bool((got.held == 2).all()) and bool((got.granted == 20).all())
    assert torch.equal(table.flatten(), before.flip(0))
    assert got.slots.unique().numel() == rows * 20 and torch.equal(got.positions, torch.arange(20, device="cuda").repeat(rows).int())
    back = nbw.kv_reserve(cache, zero, zero, got.held, free, got.count, 0)
    assert int(back.count) == 2 * rows and torch.equal(free, before)


@pytest.mark.parametrize("vocab", [33, 5000, 65536, 65537])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_verify_gives_a_row_the_same_in_any_batch(nbw, vocab, dtype):  # noqa: F811
    """Few rows of few weights take one launch, others two."""
    rows = 600 if vocab < 60000 else 5
    g = torch.Generator(device="cuda").manual_seed(vocab)
    target, draft = (torch.softmax(torch.randn(2 * rows, vocab, generator=g, device="cuda") * 2, dim=1).to(dtype) for _ in "pq")
    ids = torch.randint(0, vocab, (2 * rows,), generator=g, device="cuda").int()
    u = torch.rand(2 * rows, generator=g, device="cuda")
    cu = torch.arange(0, 2 * rows + 1, 2, device="cuda").int()
    accepted, after = nbw.verify_drafts(target, ids, u, draft=draft, cu=cu)
    some = min(rows, 60)
    for r in range(0, rows, max(1, rows // some)):
        a, x = nbw.verify_drafts(target[2 * r:2 * r + 2], ids[2 * r:2 * r + 2], u[2 * r:2 * r + 2], draft=draft[2 * r:2 * r + 2], cu=cu[:2])
        assert int(a) == int(accepted[r]) and int(x) == int(after[r])
    n = min(rows, 40)
    ref = odrafts.verify(f64(target[:2 * n]), ids[:2 * n].tolist(), f64(u[:2 * n]), cu[:n + 1].tolist(), f64(draft[:2 * n]))
    assert accepted[:n].tolist() == ref[0] and after[:n].tolist() == ref[1]
