"""GPU checks of the key-value cache's operators against the fp64 oracle (oracle/kv.py).

Tolerances.  bf16 results are one rounding (8 significant bits: relative 2^-8 at the most) of an fp32 result whose own
error is bounded from the operation: a score is a sum of dim products (each exact in
fp32), so its error is at most dim * 2^-24 of the sum of their magnitudes S; a softmax
weight's relative error is twice that, plus the sum's (its terms are added in pieces of
n/8 at the most) and the exponential's, so DELTA = 2^-23 * (dim * S + n / 8 + 32), plus
2^-16 where the weights are held as two bf16 parts (2^-8 of 2^-8) for the products with
the values;
a result's is DELTA * sum p |v|.  What only moves, or is rounded from an exact value, is
compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def nbw():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nested_bit_weight_amd as m
    m.library()
    return m


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float32).double().numpy()


class Setup:
    """A cache with rows of the given lengths on pages in random order.  Slots that belong to
    no row hold NaN, table entries that no length reaches hold junk."""

    def __init__(self, nbw, lens, *, heads=2, page=16, dim=128, dtype=BF16, room=0, seed=0, spare=0):
        self.rng = rng = np.random.default_rng(seed)
        self.lens_l, self.heads, self.page, self.dim, self.dtype = list(lens), heads, page, dim, dtype
        rows = len(lens)
        need = [-(-(n + room) // page) for n in lens]
        width = max(max(need, default=0), 1)
        pages = sum(need) + 2
        order = rng.permutation(pages)
        table = rng.choice([-1, -77, pages, 2**31 - 1, -2**31], size=(rows, width + spare)).astype(np.int32)
        at = 0
        for r, m in enumerate(need):
            table[r, :m] = order[at:at + m]
            at += m
        self.table_np = table[:, :width]
        self.table = torch.from_numpy(table).cuda()[:, :width]
        self.scales = [None, None]
        if dtype == FP8:
            self.scales = [torch.from_numpy(rng.uniform(0.01, 0.02, heads).astype(np.float32)).cuda() for _ in "kv"]
        pools = []
        for s in self.scales:
            x = rng.standard_normal((pages, heads, page, dim)).astype(np.float32)
            if s is not None:
                x = np.clip(x / s.cpu().numpy()[None, :, None, None], -448, 448)
            x = torch.from_numpy(x).to(dtype)
            owned = np.zeros((pages, page), dtype=bool)
            for r, n in enumerate(lens):
                j = np.arange(n)
                owned[table[r, j // page], j % page] = True
            x.view(torch.uint8 if dtype == FP8 else torch.int16).permute(0, 2, 1, 3)[torch.from_numpy(~owned)] = \
                0x7F if dtype == FP8 else 0x7FC0
            pools.append(x.cuda())
        self.k, self.v = pools
        self.lens = torch.tensor(self.lens_l, dtype=torch.int32).cuda()
        self.cap = width * page
        self.cache = nbw.KVCache(self.k, self.v, self.table, *self.scales)

    def pools64(self):
        got = []
        for x, s in ((self.k, self.scales[0]), (self.v, self.scales[1])):
            x = f64(x)
            got.append(x if s is None else x * f64(s)[None, :, None, None])
        return got

    def normal(self, *shape, by=1.0):
        x = torch.from_numpy((self.rng.standard_normal(shape) * by).astype(np.float32))
        return x.to(BF16).cuda()

    def totals(self):
        shape = (len(self.lens_l), self.heads, self.cap)
        return torch.from_numpy(self.rng.uniform(0, 2, shape).astype(np.float32)).cuda()


def check_attend(s, q, out, scale, acc=None, acc_out=None, decay=1.0, before=None):
    k, v = s.pools64()
    q64 = f64(q)
    want, total = okv.attend(q64, k, v, s.table_np, s.lens_l, scale, f64(acc), decay)
    weight = okv.attend(q64, k, np.abs(v), s.table_np, s.lens_l, scale)[0]  # sum p |v|
    size = np.zeros(q64.shape[:2])
    group = q64.shape[1] // s.heads
    for r, n in enumerate(s.lens_l):
        for g in range(q64.shape[1] if n else 0):
            kk, there = okv.gather(k, s.table_np[r], g // group, n)
            size[r, g] = np.nan_to_num((np.abs(kk[there]) * np.abs(q64[r, g])).sum(axis=1), posinf=0).max(initial=0)
    n = np.asarray(s.lens_l, dtype=np.float64)[:, None]
    delta = 2.0**-23 * (s.dim * size * abs(scale) + n / 8 + 32)
    got = f64(out)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    bound = 2.0**-8 * 1.01 * np.abs(want) + (delta[:, :, None] + 2.0**-16) * weight + 1e-30
    off = np.abs(got - want)
    assert np.all(off[~nan] <= bound[~nan]), float((off / bound)[~nan].max())
    if acc is not None:
        a = f64(acc_out)
        nan = np.isnan(total)
        assert np.array_equal(np.isnan(a), nan)
        worst = delta.reshape(len(n), s.heads, group).max(axis=2)[:, :, None]
        bound = 2.0**-22 * np.abs(total) + worst * np.abs(total - decay * f64(acc)) + 1e-30
        off = np.abs(a - total)
        for r, m in enumerate(s.lens_l):
            assert np.all(off[r, :, :m][~nan[r, :, :m]] <= bound[r, :, :m][~nan[r, :, :m]])
            if before is not None:  # what lies past the length is not written
                assert np.array_equal(a[r, :, m:], f64(before)[r, :, m:])


ATTEND = [
    # lens, heads, group, page, dim, dtype
    ([1], 1, 1, 1, 64, BF16), ([0, 1, 2, 3], 2, 1, 16, 128, BF16), ([31, 32, 33, 0, 127, 128, 129], 2, 4, 16, 128, BF16),
    ([500, 7, 255, 256, 257], 8, 4, 64, 128, BF16), ([1000], 8, 8, 32, 128, BF16), ([61, 700], 1, 16, 4, 128, BF16),
    ([300, 45], 2, 24, 16, 128, BF16), ([90, 301], 3, 5, 2, 64, BF16), ([77, 1030, 0], 12, 1, 16, 64, BF16),
    ([513, 3], 2, 7, 256, 64, BF16), ([130, 400], 2, 3, 8, 256, BF16), ([640], 1, 64, 64, 256, BF16),
    ([1, 0, 33, 200], 2, 4, 16, 128, FP8), ([999, 64], 8, 8, 64, 128, FP8), ([300, 129], 2, 12, 32, 64, FP8),
    ([257, 31], 2, 2, 8, 256, FP8), ([222], 1, 17, 1, 128, FP8), ([4000, 5, 2500], 2, 8, 128, 128, BF16),
    ([64] * 70, 1, 2, 16, 64, BF16), ([150, 0] * 150, 1, 1, 32, 128, BF16),
    # every (row, head) a workgroup's, with and without its totals; more rows than a wave has lanes, divided
    ([700, 20, 300] * 33, 8, 2, 16, 64, BF16), ([900] * 30, 20, 1, 64, 64, FP8), ([1500, 70] * 5, 2, 16, 64, 64, BF16),
    ([3000] + [10] * 69, 2, 3, 32, 64, BF16), ([2000, 0, 900], 1, 40, 128, 64, BF16),
    # shares that run from one (row, head) into the next; more rows than a workgroup has threads
    ([3000, 17, 900, 1400, 0, 2222, 128, 640] * 5, 16, 2, 64, 64, BF16), ([2900, 400, 1100] * 15, 12, 3, 16, 64, FP8),
    ([2500, 300] * 20, 16, 9, 32, 64, BF16), ([1200, 0] + [5] * 299, 1, 2, 16, 64, BF16),
]


@pytest.mark.parametrize("lens,heads,group,page,dim,dtype", ATTEND)
def test_attend_matches_the_oracle(nbw, lens, heads, group, page, dim, dtype):
    s = Setup(nbw, lens, heads=heads, page=page, dim=dim, dtype=dtype, seed=len(lens) * dim + group, spare=2)
    q = s.normal(len(lens), heads * group, dim, by=1.5)
    print(f"attend {lens[:8]} x{len(lens)} heads {heads} group {group} page {page} dim {dim} {dtype}", flush=True)
    out = torch.full_like(q, float("nan"))
    got = nbw.kv_attend(s.cache, q, s.lens, out=out)
    assert got is out
    check_attend(s, q, out, dim ** -0.5)
    acc = s.totals()
    acc_out = torch.full_like(acc, -3.0)
    out2 = nbw.kv_attend(s.cache, q, s.lens, acc=acc, acc_out=acc_out, decay=0.9, scale=0.3)
    check_attend(s, q, out2, float(np.float32(0.3)), acc, acc_out, float(np.float32(0.9)),
                 before=torch.full_like(acc, -3.0))


def test_attend_in_place_totals_strided_queries_bound_and_repeats(nbw):
    s = Setup(nbw, [200, 65, 0, 391], heads=2, seed=5)
    wide = s.normal(4, (8 + 2 * 2) * 128 + 8)
    q = wide[:, :8 * 128].view(4, 8, 128) if wide.stride(0) == 8 * 128 else wide[:, :8 * 128].unflatten(1, (8, 128))
    big = torch.full((4, 3000), 7.0, dtype=BF16, device="cuda")
    out = big[:, 8:8 + 1024].unflatten(1, (8, 128))
    acc = s.totals()
    first = acc.clone()
    nbw.kv_attend(s.cache, q, s.lens, out=out, acc=acc, max_len=400)
    check_attend(s, q, out, 128 ** -0.5, first, acc, before=first)
    assert bool((big[:, :8] == 7).all()) and bool((big[:, 8 + 1024:] == 7).all())
    for _ in range(3):  # the same bits every time
        acc2 = first.clone()
        out2 = nbw.kv_attend(s.cache, q, s.lens, acc=acc2, max_len=400)
        assert torch.equal(out2, out) and torch.equal(acc2, acc)
    # a bound below a row's length cuts the row
    s.lens_l = [min(n, 100) for n in s.lens_l]
    cut = nbw.kv_attend(s.cache, q, s.lens, max_len=100)
    check_attend(s, q, cut, 128 ** -0.5)


def test_totals_at_any_address(nbw):
    """Totals that are not 16-byte aligned, in a workgroup's hands and in the second launch's."""
    for lens, room in (([100, 70], 0), ([3000, 70], 0)):
        s = Setup(nbw, lens, page=16, seed=2)
        q = s.normal(2, 4, 128)
        first = s.totals()
        odd = torch.empty(first.numel() + 1, device="cuda")[1:].view(first.shape)
        odd.copy_(first)
        out = nbw.kv_attend(s.cache, q, s.lens, acc=odd, decay=0.5)
        check_attend(s, q, out, 128 ** -0.5, first, odd, 0.5, before=first)
    pos = torch.arange(s.cap, dtype=torch.int32, device="cuda").repeat(2, 2, 1)
    want = [torch.zeros_like(first), torch.zeros_like(pos)]
    nbw.kv_evict(s.cache, first, pos, s.lens, 900, recent=9, acc_out=want[0], pos_out=want[1])
    odd.copy_(first)
    odd_pos = torch.empty(pos.numel() + 3, dtype=torch.int32, device="cuda")[3:].view(pos.shape)
    odd_pos.copy_(pos)
    got = [torch.zeros(first.numel() + 1, device="cuda")[1:].view(first.shape), torch.zeros_like(pos)]
    nbw.kv_evict(s.cache, odd, odd_pos, s.lens, 900, recent=9, acc_out=got[0], pos_out=got[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_lengths_outside_the_table_are_bounded(nbw):
    s = Setup(nbw, [48, 48, 20], page=16)
    lens = torch.tensor([1 << 30, -5, 20], dtype=torch.int32, device="cuda")
    s.lens_l = [48, 0, 20]
    q = s.normal(3, 4, 128)
    check_attend(s, q, nbw.kv_attend(s.cache, q, lens), 128 ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_attend_leaves_out_pages_that_are_not_there(nbw, dtype):
    s = Setup(nbw, [100, 40, 70], page=16, dtype=dtype, seed=9)
    for r, i, x in ((0, 0, -1), (0, 3, 10**6), (1, 0, -9), (1, 1, -9), (1, 2, -9), (2, 4, s.cache.pages)):
        s.table_np[r, i] = x
        s.table[r, i] = x
    q = s.normal(3, 8, 128)
    acc = s.totals()
    acc_out = acc.clone()
    out = nbw.kv_attend(s.cache, q, s.lens, acc=acc, acc_out=acc_out, decay=0.5)
    check_attend(s, q, out, 128 ** -0.5, acc, acc_out, 0.5)
    assert bool((out[1] == 0).all())


def test_attend_infinities_and_nan_in_the_cache(nbw):
    s = Setup(nbw, [60, 60, 60, 60, 60], heads=1, page=16, seed=3)
    q = s.normal(5, 2, 128).abs() + 0.01

    def at(r, j):
        return s.table_np[r, j // 16], 0, j % 16

    s.k[at(0, 33)][5] = -math.inf                       # this slot weighs nothing
    for j in range(60):
        s.k[at(1, j)][0] = -math.inf                    # nothing is left: zeros
    s.k[at(2, 7)][1] = math.inf                         # a score of +inf: NaN
    s.v[at(3, 59)][17] = math.nan                       # NaN in one column
    s.k[at(4, 0)][9] = math.nan                         # NaN in a score
    acc = s.totals()
    acc_out = acc.clone()
    out = nbw.kv_attend(s.cache, q, s.lens, acc=acc, acc_out=acc_out)
    check_attend(s, q, out, 128 ** -0.5, acc, acc_out)
    assert bool((out[1] == 0).all()) and bool(out[2].isnan().all()) and bool(out[4].isnan().all())
    assert out[3].isnan().sum().item() == 2
    s.v[at(0, 33)][4] = math.inf                        # 0 * inf is NaN by the formula, in that column
    s.k[at(0, 33)][5] = 0.0
    out = nbw.kv_attend(s.cache, q, s.lens)
    assert bool((out[0, :, 4] == math.inf).all()) and out[0].isfinite().sum().item() == 2 * 127


def test_attend_large_scores_and_far_maximum(nbw):
    # the largest score comes last, far above the others: what was added before has to fade
    s = Setup(nbw, [700, 290], heads=2, page=32, seed=11)
    q = s.normal(2, 6, 128, by=6.0)
    for r, j in ((0, 699), (0, 350), (1, 289)):
        for h in range(2):
            s.k[s.table_np[r, j // 32], h, j % 32] = (q[r, 3 * h].float() * 0.7).to(BF16)
    check_attend(s, q, nbw.kv_attend(s.cache, q, s.lens), 128 ** -0.5)


def test_attend_shared_pages_and_cache_beyond_2_31_elements(nbw):
    pages, heads, page, dim = 33000, 8, 64, 128   # 2.16e9 elements a pool
    k = torch.empty((pages, heads, page, dim), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    rng = np.random.default_rng(0)
    used = [32999, 0, 32950, 16500, 32998]
    small_k, small_v = (torch.from_numpy(rng.standard_normal((5, heads, page, dim)).astype(np.float32)).to(BF16) for _ in "kv")
    k[torch.tensor(used).cuda()], v[torch.tensor(used).cuda()] = small_k.cuda(), small_v.cuda()
    table = torch.tensor([[0, 2, 4, 1], [0, 2, 3, 9]])
    big = torch.tensor([[used[i] if i < 5 else -1 for i in r] for r in table.tolist()], dtype=torch.int32).cuda()
    lens = torch.tensor([250, 190], dtype=torch.int32).cuda()
    q = torch.from_numpy(rng.standard_normal((2, 32, dim)).astype(np.float32)).to(BF16).cuda()
    out = nbw.kv_attend(nbw.KVCache(k, v, big), q, lens)
    small = nbw.KVCache(small_k.cuda(), small_v.cuda(), torch.where(table > 4, -1, table).int().cuda())
    assert torch.equal(out, nbw.kv_attend(small, q, lens))
    want, _ = okv.attend(f64(q), f64(small_k), f64(small_v), table.numpy(), [250, 190], dim ** -0.5)
    assert np.abs(f64(out) - want).max() <= 2.0**-8 * np.abs(want).max()
    # appending and evicting there as well
    new = torch.ones((2, heads, dim), dtype=BF16, device="cuda")
    solo = torch.tensor([[32999], [32950]], dtype=torch.int32).cuda()
    cache = nbw.KVCache(k, v, solo)
    nbw.kv_append(cache, new, -new, torch.tensor([3, 60], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda())
    assert bool((k[32999, :, 3] == 1).all()) and bool((v[32950, :, 60] == -1).all())
    acc = torch.zeros((2, heads, page), device="cuda")
    acc[:, :, 63] = 1.0
    pos = torch.arange(page, dtype=torch.int32, device="cuda").repeat(2, heads, 1)
    last = k[32999, :, 63].clone()
    nbw.kv_evict(cache, acc, pos, torch.tensor([64, 64], dtype=torch.int32).cuda(), 1, acc_out=acc.clone(), pos_out=pos.clone())
    assert torch.equal(k[32999, :, 0], last)


# ---------------------------------------------------------------------------

def rope_table(n, dim):
    angle = np.arange(n)[:, None] * (10000.0 ** (-np.arange(0, dim, 2) / dim))[None]
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)).cuda()


APPEND = [
    # old, new (None: one a row), heads, group, page, dim, dtype, norm, rope
    ([0], None, 1, 1, 1, 64, BF16, False, True), ([5, 0, 31, 16], None, 2, 4, 16, 128, BF16, True, True),
    ([5, 0, 31], [7, 0, 33], 2, 4, 16, 128, BF16, True, True), ([0, 3], [100, 1], 8, 8, 64, 128, BF16, False, True),
    ([1, 2], [9, 20], 3, 5, 4, 256, BF16, True, True), ([63, 1], [2, 66], 12, 1, 32, 64, BF16, False, False),
    ([0, 9, 4], [40, 0, 3], 2, 4, 16, 128, FP8, True, True), ([7, 250], None, 8, 8, 128, 128, FP8, False, True),
    ([3], [50], 2, 3, 8, 64, FP8, False, False), ([2, 0], [17, 5], 1, 16, 16, 256, FP8, True, True),
    (list(range(90)), None, 2, 2, 16, 64, BF16, False, True), ([1] * 80, [3, 0] * 40, 1, 2, 8, 128, BF16, True, True),
]


@pytest.mark.parametrize("old,new,heads,group,page,dim,dtype,norm,rope", APPEND)
def test_append_matches_the_oracle(nbw, old, new, heads, group, page, dim, dtype, norm, rope):
    rows = len(old)
    added = [1] * rows if new is None else new
    tokens = sum(added)
    s = Setup(nbw, old, heads=heads, page=page, dim=dim, dtype=dtype, room=max(added), seed=tokens + dim)
    print(f"append {old[:6]} + {added[:6]} x{rows} dim {dim} {dtype} norm {norm} rope {rope}", flush=True)
    wide = s.normal(tokens, (heads * (group + 2)) * dim + 16)
    q = wide[:, :heads * group * dim].unflatten(1, (heads * group, dim))
    k = wide[:, heads * group * dim:heads * (group + 1) * dim].unflatten(1, (heads, dim))
    v = wide[:, heads * (group + 1) * dim:heads * (group + 2) * dim].unflatten(1, (heads, dim))
    cu = np.concatenate([[0], np.cumsum(added)]).astype(np.int32)
    positions = s.rng.integers(0, 500, tokens).astype(np.int32)
    table = rope_table(500, dim) if rope else None
    qn, kn = (s.normal(dim, by=0.3) + 1, s.normal(dim, by=0.3) + 1) if norm else (None, None)
    pos = torch.full((rows, heads, s.cap), -4, dtype=torch.int32, device="cuda")
    acc = torch.full((rows, heads, s.cap), 2.5, device="cuda")
    k0, v0 = s.k.clone(), s.v.clone()
    q_out, lens = nbw.kv_append(s.cache, k, v, s.lens, torch.from_numpy(positions).cuda(), q=q, rope=table, q_norm=qn,
                                k_norm=kn, eps=1e-5, cu=None if new is None else torch.from_numpy(cu).cuda(), pos=pos, acc=acc)
    eps = float(np.float32(1e-5))
    zeros = np.zeros(s.k.shape)
    args = (s.table_np, old, cu, positions, f64(k), f64(v), f64(q), f64(table), f64(qn), f64(kn), eps)
    wk, wv, wq, wpos, wacc, wlens = okv.append(zeros, zeros, *args, f64(pos) * 0 - 4, f64(acc) * 0 + 2.5)
    touched = okv.append(zeros, zeros, *args[:4], np.ones(k.shape), np.ones(v.shape))[0] == 1
    assert lens.tolist() == wlens.tolist()
    assert np.array_equal(f64(pos), wpos) and np.array_equal(f64(acc), wacc)
    # one rounding, and the fp32 steps before it: sums of dim squares, two products of a pair
    delta = (dim + 16) * 2.0**-24
    pair = lambda x: np.abs(x) + np.abs(np.roll(x, dim // 2, axis=-1))  # noqa: E731
    assert np.all(np.abs(f64(q_out) - wq) <= 2.0**-8 * 1.01 * np.abs(wq) + delta * 2 * pair(wq) + 1e-30)
    got_k, got_v = f64(s.k), f64(s.v)
    if dtype == BF16:
        tol = 2.0**-8 * 1.01 * np.abs(wk) + delta * 2 * pair(wk) + 1e-30
        exact_v = wv
    else:
        f = f64(s.scales[0])[None, :, None, None]
        wk, amp = wk / f, pair(wk / f)
        assert np.abs(wk).max() < 448, "the case must not saturate"
        tol = np.maximum(2.0**-4 * np.abs(wk), 2.0**-10) * 1.001 + 2 * delta * amp
        x = torch.from_numpy(wv.astype(np.float32)) / s.scales[1].cpu()[None, :, None, None]
        exact_v = f64(x.clamp(-448, 448).to(FP8))
    assert np.all(np.abs(got_k - wk)[touched] <= tol[touched])
    assert np.array_equal(got_v[touched], exact_v[touched])
    same = torch.from_numpy(~touched).cuda()
    bits = torch.uint8 if dtype == FP8 else torch.int16
    for now, was in ((s.k, k0), (s.v, v0)):
        assert torch.equal(now.view(bits)[same], was.view(bits)[same])


def test_append_in_place_queries_without_queries_and_dropped_tokens(nbw):
    s = Setup(nbw, [30, 10], page=16, room=2)          # capacity 32 for both rows, row 1 has one page
    k, v, q = (s.normal(7, h, 128) for h in (2, 2, 4))
    cu = torch.tensor([0, 4, 7], dtype=torch.int32).cuda()
    positions = torch.arange(7, dtype=torch.int32).cuda()
    rope = rope_table(6, 128)                           # token 6 has no row: NaN
    kept = q.clone()
    lens = torch.tensor([30, 14], dtype=torch.int32).cuda()
    plain, out = nbw.kv_append(s.cache, k, v, lens, positions, cu=cu)
    assert plain is None and out.tolist() == [34, 17]
    t = s.table_np
    assert torch.equal(s.k[t[0, 1], :, 14:16].transpose(0, 1), k[:2]) and torch.equal(s.v[t[1, 0], :, 14:16].transpose(0, 1), v[4:6])
    got, _ = nbw.kv_append(s.cache, k, v, lens, positions, cu=cu, q=q, q_out=q, rope=rope)
    assert got is q and bool(q[6].isnan().all()) and torch.equal(q[0], kept[0])
    assert np.abs(f64(q[5]) - okv.turned(f64(kept[5]), 5, f64(rope), None, 0)).max() <= 2.0**-7 * 4


def test_append_saturates_and_keeps_nan_in_8_bits(nbw):
    s = Setup(nbw, [0], heads=1, dim=64, dtype=FP8, room=4)
    x = s.normal(1, 1, 64)
    x[0, 0, :6] = torch.tensor([1e4, -1e4, math.inf, -math.inf, math.nan, 0.0], dtype=BF16)
    nbw.kv_append(s.cache, x, x, s.lens, torch.zeros(1, dtype=torch.int32).cuda())
    got = s.v[s.table_np[0, 0], 0, 0].float().cpu()
    assert got[:4].tolist() == [448, -448, 448, -448] and bool(got[4].isnan()) and got[5].item() == 0
    assert torch.equal(s.k.view(torch.uint8)[s.table_np[0, 0], 0, 0], s.v.view(torch.uint8)[s.table_np[0, 0], 0, 0]) or \
        not torch.equal(s.scales[0], s.scales[1])


# ---------------------------------------------------------------------------

EVICT = [
    # lens, budget, sink, recent, heads, page, dim, dtype, kind of totals
    ([2], 1, 0, 0, 1, 1, 64, BF16, "spread"), ([33, 32, 31, 0, 1], 32, 0, 0, 2, 16, 128, BF16, "spread"),
    ([200, 100, 64], 64, 4, 16, 2, 16, 128, BF16, "spread"), ([500, 301], 100, 0, 50, 3, 32, 64, BF16, "ties"),
    ([700], 699, 4, 64, 8, 64, 128, BF16, "spread"), ([300, 257, 1000], 256, 1, 255, 1, 8, 256, BF16, "odd"),
    ([400, 90], 80, 80, 0, 2, 4, 128, BF16, "ties"), ([1030, 2000], 512, 16, 100, 2, 128, 128, FP8, "spread"),
    ([90, 64, 300], 33, 3, 5, 2, 16, 64, FP8, "odd"), ([129], 128, 0, 1, 4, 2, 256, FP8, "equal"),
    ([6000, 5000], 1500, 4, 200, 1, 64, 64, BF16, "ties"), ([70] * 40, 50, 2, 10, 2, 16, 64, BF16, "spread"),
    # a few over the budget, one more than those, all of them equal or among equals
    ([66, 67, 68, 69, 64, 65], 64, 0, 3, 2, 16, 64, BF16, "ties"), ([68, 69, 67], 65, 1, 0, 2, 16, 64, BF16, "equal"),
    ([3000, 2003, 1999], 2000, 0, 1, 1, 64, 64, BF16, "odd"), ([5] * 300, 3, 0, 0, 1, 8, 64, BF16, "ties"),
    ([2900] * 150, 2600, 4, 40, 2, 64, 64, BF16, "spread"),
    # longer than one workgroup ranks
    ([20000, 40001, 9000, 16384, 0], 12000, 4, 1000, 2, 64, 64, BF16, "spread"),
    ([70000, 30001], 30000, 16, 3000, 1, 128, 64, FP8, "ties"), ([33000, 21000], 20999, 0, 64, 1, 32, 64, BF16, "odd"),
    ([18001], 17990, 2, 0, 2, 16, 128, BF16, "equal"), ([17000, 25000], 25000, 0, 0, 1, 64, 64, BF16, "spread"),
    ([50000], 900, 4, 896, 1, 1, 64, FP8, "spread"),
]


@pytest.mark.parametrize("lens,budget,sink,recent,heads,page,dim,dtype,kind", EVICT)
def test_evict_matches_the_oracle(nbw, lens, budget, sink, recent, heads, page, dim, dtype, kind):
    s = Setup(nbw, lens, heads=heads, page=page, dim=dim, dtype=dtype, seed=budget)
    print(f"evict {lens[:6]} x{len(lens)} to {budget} sink {sink} recent {recent} dim {dim} {dtype} {kind}", flush=True)
    shape = (len(lens), heads, s.cap)
    acc = np.exp(1.5 * s.rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        acc = np.round(acc * 2) / 2
    elif kind == "equal":
        acc[:] = 0.25
    elif kind == "odd":
        acc = acc - 1.5
        acc[s.rng.random(shape) < 0.3] = 0.0
        acc[s.rng.random(shape) < 0.2] = -0.0
        acc[s.rng.random(shape) < 0.1] = np.nan
        acc[s.rng.random(shape) < 0.05] = np.inf
        acc[s.rng.random(shape) < 0.1] = -np.inf
        acc[s.rng.random(shape) < 0.05] = 1e-42
    acc = acc.astype(np.float32)
    pos = np.stack([[s.rng.permutation(s.cap) for _ in range(heads)] for _ in lens]).astype(np.int32)
    acc_t, pos_t = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    acc_out, pos_out = torch.full_like(acc_t, -7.0), torch.full_like(pos_t, -7)
    bits = torch.uint8 if dtype == FP8 else torch.int16
    k0, v0 = (x.view(bits).cpu().numpy() for x in (s.k, s.v))
    want = okv.evict(k0, v0, s.table_np, lens, acc, pos, budget, sink, recent, acc_out.cpu().numpy(), pos_out.cpu().numpy())
    for _ in range(2):  # the moves read nothing that they write: a second call gives the same
        lens_out = nbw.kv_evict(s.cache, acc_t, pos_t, s.lens, budget, sink=sink, recent=recent, acc_out=acc_out,
                                pos_out=pos_out, max_len=max(lens))
        assert np.array_equal(s.k.view(bits).cpu().numpy(), want[0]) and np.array_equal(s.v.view(bits).cpu().numpy(), want[1])
        assert np.array_equal(acc_out.cpu().numpy().view(np.int32), np.asarray(want[2], dtype=np.float32).view(np.int32))
        assert np.array_equal(pos_out.cpu().numpy(), want[3]) and lens_out.tolist() == list(want[4])
    assert np.array_equal(acc_t.cpu().numpy().view(np.int32), acc.view(np.int32)) and np.array_equal(pos_t.cpu().numpy(), pos)


def test_evict_pages_that_are_not_there_and_positions_that_repeat(nbw):
    s = Setup(nbw, [100, 90], page=16, seed=4)
    for r, i in ((0, 1), (0, 5), (1, 4)):
        s.table_np[r, i] = -1
        s.table[r, i] = -1
    acc = np.exp(s.rng.standard_normal((2, 2, s.cap))).astype(np.float32)
    pos = np.full((2, 2, s.cap), 3, dtype=np.int32)   # every one of them counts as protected
    pos[1] = s.rng.integers(0, 20, pos[1].shape)
    acc_t, pos_t = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    acc_out, pos_out = torch.zeros_like(acc_t), torch.zeros_like(pos_t)
    k0, v0 = (x.view(torch.int16).cpu().numpy() for x in (s.k, s.v))
    want = okv.evict(k0, v0, s.table_np, [100, 90], acc, pos, 40, 2, 3, acc_out.cpu().numpy(), pos_out.cpu().numpy())
    nbw.kv_evict(s.cache, acc_t, pos_t, s.lens, 40, sink=2, recent=3, acc_out=acc_out, pos_out=pos_out)
    assert np.array_equal(s.k.view(torch.int16).cpu().numpy(), want[0]) and np.array_equal(s.v.view(torch.int16).cpu().numpy(), want[1])
    assert np.array_equal(acc_out.cpu().numpy(), want[2].astype(np.float32)) and np.array_equal(pos_out.cpu().numpy(), want[3])


# ---------------------------------------------------------------------------

def test_other_streams_and_graph_replays(nbw):
    s = Setup(nbw, [300, 0, 64, 129], heads=2, page=16, room=8, seed=8)
    q, k, v = s.normal(4, 8, 128), s.normal(4, 2, 128), s.normal(4, 2, 128)
    positions = torch.tensor([300, 0, 64, 129], dtype=torch.int32).cuda()
    rope = rope_table(400, 128)
    ws = torch.empty(s.cache.attend_workspace_bytes(8, weights=True) + s.cache.evict_workspace_bytes(100), dtype=torch.uint8,
                     device="cuda")
    bufs = dict(q_out=torch.empty_like(q), lens1=torch.empty_like(s.lens), lens2=torch.empty_like(s.lens), out=torch.empty_like(q),
                acc=s.totals(), pos=torch.arange(s.cap, dtype=torch.int32).repeat(4, 2, 1).cuda())
    bufs["acc1"], bufs["acc2"], bufs["pos2"] = (torch.zeros_like(bufs[x]) for x in ("acc", "acc", "pos"))

    def step():
        nbw.kv_append(s.cache, k, v, s.lens, positions, q=q, rope=rope, q_out=bufs["q_out"], pos=bufs["pos"], acc=bufs["acc"],
                      lens_out=bufs["lens1"])
        nbw.kv_attend(s.cache, bufs["q_out"], bufs["lens1"], out=bufs["out"], acc=bufs["acc"], acc_out=bufs["acc1"], workspace=ws)
        nbw.kv_evict(s.cache, bufs["acc1"], bufs["pos"], bufs["lens1"], 100, recent=10, acc_out=bufs["acc2"],
                     pos_out=bufs["pos2"], lens_out=bufs["lens2"], workspace=ws)

    start = s.k.clone(), s.v.clone()
    step()
    torch.cuda.synchronize()
    names = ("q_out", "lens1", "out", "acc1", "acc2", "pos2", "lens2")
    want = [bufs[n].clone() for n in names] + [s.k.clone(), s.v.clone()]

    def reset():
        for n in names:
            bufs[n].zero_() if n in ("acc1", "acc2", "pos2") else bufs[n].fill_(99)
        s.k.copy_(start[0])
        s.v.copy_(start[1])

    def same():
        got = [bufs[n] for n in names] + [s.k, s.v]
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))

    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        reset()
        nbw.kv_attend(s.cache, q, s.lens, acc=s.totals())  # other eager work between the replays
        g.replay()
        torch.cuda.synchronize()
        assert same(), f"replay {rep}"


def test_refusals(nbw):
    s = Setup(nbw, [20, 30], heads=2, page=16, room=2)
    q, k = s.normal(2, 8, 128), s.normal(2, 2, 128)
    acc, pos = s.totals(), torch.zeros((2, 2, s.cap), dtype=torch.int32, device="cuda")
    positions = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        nbw.kv_attend(s.cache, q[:, :7], s.lens)
    with pytest.raises(TypeError):
        nbw.kv_attend(s.cache, q.float(), s.lens)
    with pytest.raises(TypeError):
        nbw.kv_attend(s.cache, q, s.lens.long())
    with pytest.raises(ValueError):
        nbw.kv_attend(s.cache, q, s.lens, acc=acc[:, :, 1:])
    with pytest.raises(ValueError):
        nbw.kv_attend(s.cache, q, s.lens, acc_out=acc)
    with pytest.raises(ValueError):
        nbw.kv_attend(s.cache, q.transpose(0, 1).contiguous().transpose(0, 1), s.lens)
    with pytest.raises(ValueError):
        nbw.kv_attend(s.cache, q, s.lens, scale=0.0)
    long = Setup(nbw, [3000, 30], heads=2, page=64)
    with pytest.raises(nbw.NBWError):
        nbw.kv_attend(long.cache, q, long.lens, acc=long.totals(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nbw.NBWError):
        nbw.kv_attend(long.cache, q, long.lens, workspace=None)
    with pytest.raises(ValueError):
        nbw.kv_append(s.cache, k[:1], k[:1], s.lens, positions[:1])
    with pytest.raises(ValueError):
        nbw.kv_append(s.cache, k, k, s.lens, positions, q_norm=q[0, 0])
    with pytest.raises(nbw.NBWError):
        nbw.kv_append(s.cache, k, k, s.lens, positions, lens_out=s.lens)
    with pytest.raises(ValueError):
        nbw.kv_evict(s.cache, acc, pos, s.lens, 0, acc_out=acc.clone(), pos_out=pos.clone())
    with pytest.raises(ValueError):
        nbw.kv_evict(s.cache, acc, pos, s.lens, 8, sink=4, recent=5, acc_out=acc.clone(), pos_out=pos.clone())
    with pytest.raises(nbw.NBWError):
        nbw.kv_evict(s.cache, acc, pos, s.lens, 8, acc_out=acc, pos_out=pos.clone())
    with pytest.raises(ValueError):
        nbw.KVCache(s.k, s.v, s.table, s.lens.float(), s.lens.float())
    with pytest.raises(ValueError):
        nbw.KVCache(s.k[..., :96].contiguous(), s.v[..., :96].contiguous(), s.table)
    with pytest.raises(ValueError):
        nbw.KVCache(s.k, s.v[:1], s.table)
