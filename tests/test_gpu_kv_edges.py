"""GPU checks of the key-value cache's operators at the edges of what they promise: weights to their last bits, values
near the largest finite one, infinities, lengths and totals out of the ordinary, tables wider than their rows.

Tolerances are derived beside each test; what only moves is compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv

from test_gpu_kv import BF16, FP8, Setup, check_attend, f64, nbw  # noqa: F401  (nbw: the fixture)

pytestmark = pytest.mark.gpu


def to_bf16(x):
    """The nearest bf16 of fp64 numbers, as fp64."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.float32).to(BF16).double().numpy()


def cut_bf16(x):
    """x cut off to bf16's 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, 8)), e - 8)


@pytest.mark.parametrize("group,dim,page", [(1, 64, 16), (8, 128, 4), (12, 128, 16), (3, 256, 16)])
def test_attend_weights_keep_their_24_bits(nbw, group, dim, page):  # noqa: F811
    """Three slots of weights 1, 1 and p and values -c1, -c2 and 1, where c1 + c2 are p's first 16 bits: the result is
    what is left of p, (p - c1 - c2) / (2 + p).  A score here is one product and exact; times log2(e) it is off by 2 units of
    2^-24 of less than 1, which moves p by 1.4 of them; the exponential by 1 unit of p below 1; the sums of products by 8.
    That is below 2^-20, and 2^-21 after the division by 2 + p > 2."""
    rows, heads = 64, 8
    rng = np.random.default_rng(group)
    s = to_bf16(-rng.uniform(0.02, 0.69, (rows, heads)))
    p = np.exp(s)
    c1 = cut_bf16(p)
    c2 = to_bf16(p - c1)
    k, v = np.zeros((rows, heads, page, dim)), np.zeros((rows, heads, page, dim))
    k[:, :, 2, 0] = s
    v[:, :, 0], v[:, :, 1], v[:, :, 2] = -c1[..., None], -c2[..., None], 1.0
    q = np.zeros((rows, heads * group, dim))
    q[:, :, 0] = 1.0
    k, v, q = (torch.from_numpy(x).to(torch.float32).to(BF16).cuda() for x in (k, v, q))
    cache = nbw.KVCache(k, v, torch.arange(rows, dtype=torch.int32, device="cuda")[:, None])
    out = f64(nbw.kv_attend(cache, q, torch.full((rows,), 3, dtype=torch.int32, device="cuda"), scale=1.0))
    want = ((p - c1 - c2) / (2 + p)).repeat(group, axis=1)[..., None]
    assert np.abs(want).max() > 2.0**-19.5  # what two parts would lose is there to be seen
    assert np.all(np.abs(out - want) <= 2.0**-8 * 1.01 * np.abs(want) + 2.0**-21), float(np.abs(out - want).max() * 2.0**21)


def rows_cache(nbw, lens, heads, dim, page, seed, width=None):  # noqa: F811
    """A bf16 cache of rows on pages of their own: (cache, lens tensor, table as numpy)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), width or max(need)), -1, dtype=np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = np.arange(at, at + m)
        at += m
    pools = [torch.from_numpy(rng.standard_normal((at, heads, page, dim)).astype(np.float32)).to(BF16).cuda() for _ in "kv"]
    cache = nbw.KVCache(*pools, torch.from_numpy(table).cuda())
    return cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), table


@pytest.mark.parametrize("lens", [[60, 60], [500, 40], [3000, 2600]])
@pytest.mark.parametrize("group,dim,page", [(2, 128, 16), (12, 64, 4), (4, 256, 32)])
def test_attend_heads_without_a_score_give_zeros_whatever_their_values(nbw, lens, group, dim, page):  # noqa: F811
    """Row 0's scores are all -infinity: zeros and unchanged totals, also where its values are infinite or NaN."""
    cache, n, table = rows_cache(nbw, lens, 2, dim, page, 7)
    mine = torch.from_numpy(table[0][table[0] >= 0]).long().cuda()
    cache.k[mine, :, :, 0] = -math.inf
    cache.v[mine[0], :, :, 3] = math.inf
    cache.v[mine[-1], :, :, 5] = -math.inf
    cache.v[mine[-1], :, 0, 7] = math.nan
    q = torch.rand((2, 2 * group, dim), device="cuda").add_(0.01).to(BF16)
    print(f"no scores {lens} group {group} dim {dim} page {page}", flush=True)
    out = nbw.kv_attend(cache, q, n)
    assert bool((out[0] == 0).all()) and bool(out[1].isfinite().all())
    acc = torch.rand((2, 2, cache.capacity), device="cuda")
    acc_out = torch.zeros_like(acc)
    assert torch.equal(nbw.kv_attend(cache, q, n, acc=acc, acc_out=acc_out), out)
    assert torch.equal(acc_out[0, :, :lens[0]], acc[0, :, :lens[0]])


@pytest.mark.parametrize("lens", [[200, 64], [3000, 900]])
@pytest.mark.parametrize("group", [2, 12])
def test_attend_weights_of_zero_add_nothing_however_large_the_value(nbw, lens, group):  # noqa: F811
    """Values of 3e38 in slots whose weight is below any number (scores 300 below the others) or 0 (scores of -infinity)."""
    s = Setup(nbw, lens, heads=2, page=16, seed=group)
    q = s.normal(2, 2 * group, 128).abs() + 0.25
    for r, j, key in ((0, 3, -30.0), (0, lens[0] - 1, -math.inf), (1, 40, -30.0), (1, 41, -30.0)):
        at = s.table_np[r, j // 16], slice(None), j % 16
        s.k[at] = key
        s.v[at] = 3e38
    out = nbw.kv_attend(s.cache, q, s.lens)
    assert bool((out.abs() < 8).all())
    check_attend(s, q, out, 128 ** -0.5)


@pytest.mark.parametrize("lens", [[200, 1], [3000, 900]])
@pytest.mark.parametrize("group,dim", [(2, 128), (12, 64), (3, 256)])
def test_attend_values_near_the_largest_finite_one(nbw, lens, group, dim):  # noqa: F811
    """All values 3.3e38, and with either sign: their mean is finite, their sum is not."""
    s = Setup(nbw, lens, heads=2, page=16, dim=dim, seed=group)
    q = s.normal(2, 2 * group, dim)
    s.v[~s.v.isnan()] = 3.3e38
    out = nbw.kv_attend(s.cache, q, s.lens)
    check_attend(s, q, out, dim ** -0.5)
    s.v[..., ::2] *= -1
    check_attend(s, q, nbw.kv_attend(s.cache, q, s.lens), dim ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("many", [False, True])
def test_append_bounds_the_lengths(nbw, dtype, many):  # noqa: F811
    """A length below 0 counts as 0, one above the capacity as the capacity, in the slots and in the lengths that come back."""
    s = Setup(nbw, [48, 48, 48, 20], page=16, dtype=dtype)
    old = [-5, 1 << 30, -2**31, 20]
    added = [7, 2, 1, 3] if many else [1] * 4
    tokens = sum(added)
    k, v = s.normal(tokens, 2, 128), s.normal(tokens, 2, 128)
    positions = np.arange(100, 100 + tokens, dtype=np.int32)
    cu = np.concatenate([[0], np.cumsum(added)]).astype(np.int32)
    pos, acc = torch.full((4, 2, 48), -4, dtype=torch.int32, device="cuda"), torch.ones((4, 2, 48), device="cuda")
    bits = torch.uint8 if dtype == FP8 else torch.int16
    kept = [x.clone() for x in (s.k, s.v)]
    _, lens = nbw.kv_append(s.cache, k, v, torch.tensor(old, dtype=torch.int32, device="cuda"), torch.from_numpy(positions).cuda(),
                            cu=torch.from_numpy(cu).cuda() if many else None, pos=pos, acc=acc)
    # the oracle moves numbers: which token is in a slot (0: what was there)
    which = np.arange(1, tokens + 1)[:, None, None] * np.ones((tokens, 2, 128))
    blank = np.zeros(s.k.shape)
    at, _, _, wpos, wacc, wlens = okv.append(blank, blank, s.table_np, old, cu, positions, which, which, pos=f64(pos) * 0 - 4,
                                             acc=f64(acc) * 0 + 1)
    assert lens.tolist() == wlens.tolist() == [added[0], 48 + added[1], added[2], 20 + added[3]]
    assert np.array_equal(f64(pos), wpos) and np.array_equal(f64(acc), wacc)
    for new, pool, was, scale in ((k, s.k, kept[0], s.scales[0]), (v, s.v, kept[1], s.scales[1])):
        x = new.float() if scale is None else (new.float() / scale[None, :, None]).clamp(-448, 448)
        x = x.to(dtype)
        want = was.clone()
        for t in range(tokens):
            page, place = np.argwhere(at[:, 0, :, 0] == t + 1).reshape(-1, 2).T
            if len(page):
                want[int(page[0]), :, int(place[0])] = x[t]
        assert torch.equal(pool.view(bits), want.view(bits))


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([70, 66], 64, 3, 5), ([66, 64], 64, 2, 62), ([700, 300], 200, 4, 100), ([3000, 900], 800, 0, 800), ([20000, 30000], 9000, 16, 3000),
    ([18000], 12000, 0, 12000),
])
def test_evict_protected_slots_stay_beside_infinite_totals(nbw, lens, budget, sink, recent):  # noqa: F811
    """More totals of +infinity than the budget has room for, in lower slots than the protected ones."""
    s = Setup(nbw, lens, heads=2, page=32, dim=64, seed=budget)
    shape = (len(lens), 2, s.cap)
    acc = s.rng.uniform(0, 1, shape).astype(np.float32)
    acc[s.rng.random(shape) < 0.9] = np.inf
    pos = np.stack([[s.rng.permutation(n) if h else np.arange(n) for h in range(2)] for n in [s.cap] * len(lens)]).astype(np.int32)
    for r, n in enumerate(lens):  # head 0: the newest lie last and have nothing
        acc[r, 0, n - recent:n] = -np.inf
    acc_t, pos_t = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    acc_out, pos_out = torch.zeros_like(acc_t), torch.full_like(pos_t, -7)
    k0, v0 = (x.view(torch.int16).cpu().numpy() for x in (s.k, s.v))
    want = okv.evict(k0, v0, s.table_np, lens, acc, pos, budget, sink, recent, acc_out.cpu().numpy(), pos_out.cpu().numpy())
    nbw.kv_evict(s.cache, acc_t, pos_t, s.lens, budget, sink=sink, recent=recent, acc_out=acc_out, pos_out=pos_out)
    for r, n in enumerate(lens):
        if n > budget:
            held = set(range(sink)) | set(range(n - recent, n))
            assert held <= set(pos_out[r, 0, :budget].tolist())
    assert np.array_equal(pos_out.cpu().numpy(), want[3]) and np.array_equal(acc_out.cpu().numpy(), want[2].astype(np.float32))
    assert np.array_equal(s.k.view(torch.int16).cpu().numpy(), want[0]) and np.array_equal(s.v.view(torch.int16).cpu().numpy(), want[1])


def test_attend_refuses_more_than_a_launch_takes(nbw):  # noqa: F811
    import ctypes

    from nested_bit_weight_amd import kv
    # one workgroup for each (row, head); then divided, the second launch with one for each query head
    for rows, heads, width, q_heads, totals, fits in ((1 << 19, 16, 1, 16, 0, True), (1 << 19, 32, 1, 32, 0, False),
                                                      (1 << 15, 8, 512, 256, 1, True), (1 << 15, 8, 512, 512, 1, False)):
        view = kv.KVView(1 << 20, 1 << 20, 10, heads, 16, 64, 0, None, None, 1 << 20, rows, width, 0)
        need = nbw.library().nbw_kv_attend_workspace_bytes(ctypes.byref(view), q_heads, 0, totals)
        assert (need >= 0) == fits, (rows, heads, width, q_heads, need)


def moves(acc, pos, n, budget, sink, recent):
    """The places below the budget that go and the slots past it that stay, of one head's first n slots (numpy, no NaN)."""
    a, p = acc[:n].astype(np.float64), pos[:n].astype(np.int64)
    held = (p < sink) | (p > p.max() - recent)
    first = np.lexsort((np.arange(n), -a, ~held))[:budget]
    stays = np.zeros(n, dtype=bool)
    stays[first] = True
    return np.flatnonzero(~stays[:budget]), budget + np.flatnonzero(stays[budget:])


def check_evict(nbw, cache, lens, table, acc, pos, budget, sink, recent, **kw):  # noqa: F811
    """One eviction on the GPU against `moves`, bit for bit."""
    rows, heads = acc.shape[:2]
    acc_out, pos_out = torch.full_like(acc, -7.0), torch.full_like(pos, -7)
    bits = [x.view(torch.uint8 if x.element_size() == 1 else torch.int16) for x in (cache.k, cache.v)]
    was = [x.clone() for x in bits]
    lens_out = nbw.kv_evict(cache, acc, pos, lens, budget, sink=sink, recent=recent, acc_out=acc_out, pos_out=pos_out, **kw)
    assert lens_out.tolist() == [min(n, budget) for n in lens.tolist()]
    total = 0
    for r, n in enumerate(lens.tolist()):
        for h in range(heads if n else 0):
            m = min(n, budget)
            a, p = acc[r, h, :n].cpu().numpy(), pos[r, h, :n].cpu().numpy()
            a2, p2 = a.copy(), p.copy()
            if n > budget:
                to, of = moves(a, p, n, budget, sink, recent)
                a2[to], p2[to] = a[of], p[of]
                total += len(to)
                at = [(torch.from_numpy(table[r, j // cache.page].astype(np.int64)).cuda(), torch.from_numpy(j % cache.page).cuda())
                      for j in (to, of)]
                for x in was:
                    x[at[0][0], h, at[0][1]] = x[at[1][0], h, at[1][1]]
            assert np.array_equal(acc_out[r, h, :m].cpu().numpy(), a2[:m]) and np.array_equal(pos_out[r, h, :m].cpu().numpy(), p2[:m])
            assert bool((acc_out[r, h, m:] == -7).all()) and bool((pos_out[r, h, m:] == -7).all())
    assert torch.equal(bits[0], was[0]) and torch.equal(bits[1], was[1])
    return total


def test_evict_more_moves_than_a_launch_has_workgroups(nbw):  # noqa: F811
    """512 rows of 8 heads in a table of 131072 slots, one of them full, brought down to half: 2^24 times 16 places for moves."""
    lens = [131072] + [0] * 511
    cache, n, table = rows_cache(nbw, lens, 8, 64, 256, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    acc = torch.empty((512, 8, cache.capacity), device="cuda")
    pos = torch.empty((512, 8, cache.capacity), dtype=torch.int32, device="cuda")
    # the upper half has the larger totals in three slots of four: 49152 moves; all of them for the last head
    acc[0] = torch.rand((8, cache.capacity), generator=g, device="cuda")
    acc[0, :, 65536:] += (torch.arange(65536, device="cuda") % 4 > 0).float()
    acc[0, 7, 65536:] += 2.0
    pos[0] = torch.arange(cache.capacity, dtype=torch.int32, device="cuda")
    assert check_evict(nbw, cache, n, table, acc, pos, 65536, 0, 100) > 7 * 45000 + 65535


def test_attend_scales_that_fp32_does_not_hold_are_refused(nbw):  # noqa: F811
    s = Setup(nbw, [40, 7], page=16)
    q = s.normal(2, 4, 128)
    for scale in (1e-46, -1e-46, 0.0, 1e39, -1e300, math.inf, math.nan):
        with pytest.raises(ValueError):
            nbw.kv_attend(s.cache, q, s.lens, scale=scale)
    for scale in (1e-30, -0.25, 1e-40):  # what it holds, subnormal numbers among it
        check_attend(s, q, nbw.kv_attend(s.cache, q, s.lens, scale=scale), float(np.float32(scale)))


def test_calls_go_to_the_tensors_gpu(nbw, monkeypatch):  # noqa: F811
    """With another GPU the current one (as far as the binding can tell), every call makes the tensors' its own for as long
    as it takes, and its results are the same."""
    from nested_bit_weight_amd import kv
    s = Setup(nbw, [3000, 40], page=16, room=2)
    q, k = s.normal(2, 4, 128), s.normal(2, 2, 128)
    acc, pos = s.totals(), torch.arange(s.cap, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    positions = torch.tensor([3000, 40], dtype=torch.int32, device="cuda")
    start = s.k.clone(), s.v.clone()

    def step():
        s.k.copy_(start[0]), s.v.copy_(start[1])
        _, lens = nbw.kv_append(s.cache, k, k, s.lens, positions)
        total, acc2, pos2 = acc.clone(), torch.zeros_like(acc), torch.zeros_like(pos)
        out = nbw.kv_attend(s.cache, q, lens, acc=total)
        left = nbw.kv_evict(s.cache, total, pos, lens, 1000, acc_out=acc2, pos_out=pos2)
        return [x.clone() for x in (lens, out, total, acc2, pos2, left, s.k.view(torch.int16), s.v.view(torch.int16))]

    want = step()
    current, entered = [1], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)
            self.was, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.was

    monkeypatch.setattr(kv, "_current_device", lambda: current[0])
    monkeypatch.setattr(kv.torch.cuda, "device", Device)
    got = step()
    assert entered == [0, 0, 0] and current == [1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_batch_without_rows(nbw):  # noqa: F811
    """Every sequence has ended: the calls take empty tensors and give empty ones."""
    pool = torch.zeros((4, 2, 16, 128), dtype=BF16, device="cuda")
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    heads = lambda h: torch.zeros((0, h, 128), dtype=BF16, device="cuda")  # noqa: E731
    cache = nbw.KVCache(pool, pool.clone(), ints(0, 3))
    acc, pos = torch.zeros((0, 2, 48), device="cuda"), ints(0, 2, 48)
    assert cache.attend_workspace_bytes(8, weights=True) == 0 and cache.evict_workspace_bytes(10) == 0
    q_out, lens = nbw.kv_append(cache, heads(2), heads(2), ints(0), ints(0), q=heads(8), pos=pos, acc=acc)
    assert q_out.shape == (0, 8, 128) and lens.shape == (0,)
    assert nbw.kv_attend(cache, heads(8), ints(0), acc=acc).shape == (0, 8, 128)
    assert nbw.kv_evict(cache, acc, pos, ints(0), 10, acc_out=acc.clone(), pos_out=pos.clone()).shape == (0,)
    # rows without a new token, and with none at all
    s = Setup(nbw, [5, 0], page=16, room=2)
    _, lens = nbw.kv_append(s.cache, heads(2), heads(2), s.lens, ints(0), cu=ints(3))
    assert lens.tolist() == [5, 0]


# ---------------------------------------------------------------------------
# tables wider than their rows: the launches, and whether loads stream, go by the capacity

def widen(nbw, s, width):  # noqa: F811
    """The cache of a Setup with a table of `width` pages a row, junk past each row's."""
    table = s.rng.choice([-1, 10**9, 0, s.cache.pages - 1], size=(len(s.lens_l), width)).astype(np.int32)
    table[:, :s.table_np.shape[1]] = s.table_np
    return nbw.KVCache(s.k, s.v, torch.from_numpy(table).cuda(), *s.scales)


@pytest.mark.parametrize("group", [4, 11])
@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_in_a_wide_table(nbw, dim, dtype, page, group):  # noqa: F811
    """Rows of a few hundred slots that may become so long that their keys and values are 256 MB and more."""
    lens = [700, 0, 333, 64, 1]
    s = Setup(nbw, lens, heads=2, page=page, dim=dim, dtype=dtype, seed=dim + group)
    slots = (256 << 20) // (len(lens) * 2 * dim * (2 if dtype == FP8 else 4)) + page
    cache = widen(nbw, s, -(-slots // page))
    print(f"wide attend dim {dim} {dtype} page {page} group {group} capacity {cache.capacity}", flush=True)
    assert len(lens) * 2 * cache.capacity * dim * (2 if dtype == FP8 else 4) > 256 << 20
    q = s.normal(len(lens), 2 * group, dim, by=1.5)
    check_attend(s, q, nbw.kv_attend(cache, q, s.lens), dim ** -0.5)
    acc = torch.rand((len(lens), 2, cache.capacity), device="cuda")
    acc_out = torch.full_like(acc, -3.0)
    out = nbw.kv_attend(cache, q, s.lens, acc=acc, acc_out=acc_out, decay=0.75)
    check_attend(s, q, out, dim ** -0.5, acc, acc_out, 0.75, before=torch.full_like(acc, -3.0))


@pytest.mark.parametrize("lens,budget,width", [([2049, 2048, 0, 2050], 2048, 4096), ([1500, 900, 3000], 700, 2048), ([30, 64], 64, 3000)])
def test_evict_in_a_wide_table(nbw, lens, budget, width):  # noqa: F811
    """Short rows whose table is longer than one workgroup ranks."""
    cache, n, table = rows_cache(nbw, lens, 3, 64, 16, 5, width=width)
    assert cache.capacity > 16384
    g = torch.Generator(device="cuda").manual_seed(6)
    acc = torch.randn((len(lens), 3, cache.capacity), generator=g, device="cuda").exp()
    pos = torch.rand((len(lens), 3, cache.capacity), generator=g, device="cuda").argsort(dim=2).int()
    total = check_evict(nbw, cache, n, table, acc, pos, budget, 4, budget // 8)
    assert (total > 0) == (max(lens) > budget)


@pytest.mark.parametrize("dim,dtype", [(64, FP8), (64, BF16), (128, BF16), (256, BF16)])
def test_evict_with_streaming_moves(nbw, dim, dtype):  # noqa: F811
    """Moves that may come to more than 64 MB, 64, 128, 256 and 512 bytes a row."""
    row = dim * (1 if dtype == FP8 else 2)
    budget = (64 << 20) // (4 * 2 * row) + 100
    lens = [budget + 700, budget + 3]
    cache, n, table = rows_cache(nbw, lens, 2, dim, 64, dim, width=-(-2 * budget // 64))
    if dtype == FP8:
        scale = torch.ones(2, device="cuda")
        cache = nbw.KVCache(cache.k.to(FP8), cache.v.to(FP8), cache.table, scale, scale)
    print(f"streaming moves of {row} bytes, budget {budget}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    acc = torch.rand((2, 2, cache.capacity), generator=g, device="cuda")
    acc[:, :, budget:] += 0.5
    pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    assert check_evict(nbw, cache, n, table, acc, pos, budget, 4, 300) > 600


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,heads,budget,streams", [
    ([3000, 0, 700, 129], 2, 300, False),    # divided attention with totals and its join; lists of moves in the workspace
    ([20000, 17000, 0, 40], 2, 9000, True),  # rows that several workgroups rank
    ([2600, 40] * 35, 4, 1000, False),       # more rows than a wave has lanes
])
def test_other_streams_and_replays_of_calls_with_a_workspace(nbw, lens, heads, budget, streams):  # noqa: F811
    """A step of append, attend and evict on another stream, and captured in a graph and replayed with longer and shorter rows
    than it was captured with, against the same step run eagerly on the same inputs."""
    rows = len(lens)
    s = Setup(nbw, lens, heads=heads, page=16, room=40, seed=8)
    if streams:
        s.cache = widen(nbw, s, s.table_np.shape[1] + 700)
    cap = s.cache.capacity
    q, k, v = s.normal(rows, heads * 4, 128), s.normal(rows, heads, 128), s.normal(rows, heads, 128)
    positions = s.lens.clone()
    sizes = s.cache.attend_workspace_bytes(heads * 4, weights=True), s.cache.evict_workspace_bytes(budget)
    assert min(sizes) > 0
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    acc0 = torch.rand((rows, heads, cap), device="cuda")
    pos0 = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(rows, heads, 1)
    b = dict(lens=s.lens.clone(), acc=acc0.clone(), pos=pos0.clone(), out=torch.empty_like(q), lens1=torch.empty_like(s.lens),
             lens2=torch.empty_like(s.lens), acc2=torch.zeros_like(acc0), pos2=torch.zeros_like(pos0))
    k0, v0 = s.k.clone(), s.v.clone()

    def step():
        nbw.kv_append(s.cache, k, v, b["lens"], positions, pos=b["pos"], acc=b["acc"], lens_out=b["lens1"])
        nbw.kv_attend(s.cache, q, b["lens1"], out=b["out"], acc=b["acc"], decay=0.5, workspace=ws)
        nbw.kv_evict(s.cache, b["acc"], b["pos"], b["lens1"], budget, recent=10, acc_out=b["acc2"], pos_out=b["pos2"],
                     lens_out=b["lens2"], workspace=ws)

    def reset(extra):
        b["lens"].copy_(torch.clamp(s.lens + extra, min=0))
        b["acc"].copy_(acc0), b["pos"].copy_(pos0), s.k.copy_(k0), s.v.copy_(v0)
        for n in ("out", "lens1", "lens2", "acc2", "pos2"):
            b[n].zero_()
        ws.fill_(0xA5)

    def results():
        torch.cuda.synchronize()
        return [x.clone().view(torch.uint8) for x in (b["out"], b["acc"], b["pos"], b["lens1"], b["lens2"], b["acc2"], b["pos2"], s.k, s.v)]

    # pages past a row's length hold NaN, which longer rows would read: give them numbers
    k0.nan_to_num_(0.25), v0.nan_to_num_(0.5)
    want = {}
    for extra in (0, 17, -350, 35):
        reset(extra)
        step()
        want[extra] = results()
    reset(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(results(), want[0]))
    g = torch.cuda.CUDAGraph()
    reset(0)
    with torch.cuda.graph(g):
        step()
    for extra in (0, 17, 35, -350, 0, 17):
        reset(extra)
        nbw.kv_attend(s.cache, q, s.lens, acc=acc0.clone())  # other eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(results(), want[extra])), extra


def test_append_limits_keys_and_values_to_the_largest_8_bit_number(nbw):  # noqa: F811
    s = Setup(nbw, [0, 0], heads=1, dim=64, dtype=FP8, room=4)
    x = s.normal(2, 1, 64)
    special = torch.tensor([1e4, -1e4, math.inf, -math.inf, math.nan, 0.0], dtype=BF16)
    x[0, 0, :6] = special
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    nbw.kv_append(s.cache, x, x, s.lens, zero)
    for pool, scale in ((s.k, s.scales[0]), (s.v, s.scales[1])):
        got = pool[s.table_np[0, 0], 0, 0].float().cpu()
        assert got[:4].tolist() == [448, -448, 448, -448] and bool(got[4].isnan()) and got[5].item() == 0
        plain = (x[1, 0].float() / scale).clamp(-448, 448).to(FP8)
        assert torch.equal(pool[s.table_np[1, 0], 0, 0].view(torch.uint8), plain.view(torch.uint8))
    # a pair within the limit whose rotation by 45 degrees is past it: 5 and 5 at a factor of 0.0125 are 400 each, and 566 together
    s.scales[0].fill_(0.0125)
    y = torch.zeros((2, 1, 64), dtype=BF16, device="cuda")
    y[:, 0, 7], y[:, 0, 32 + 7] = 5.0, 5.0
    rope = torch.full((1, 64), math.sqrt(0.5), device="cuda")
    nbw.kv_append(s.cache, y, y, zero, zero, rope=rope)
    got = s.k[s.table_np[0, 0], 0, 0].float().cpu()
    assert got[7].item() == 0 and got[32 + 7].item() == 448 and got.abs().sum().item() == 448
