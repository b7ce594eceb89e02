"""Host-side checks of the key-value cache's operators: no GPU, no device work queued.

The oracle is pinned by cases whose answers follow from the definitions without it;
the entry points reject every bad argument before any HIP call.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import nested_bit_weight_amd as nbw
from nested_bit_weight_amd import kv
from oracle import kv as okv

OK, EINVAL, EALIGN, EUNSUPPORTED, ESCRATCH = 0, 1, 2, 4, 6
FAKE = 0x7F0000001000  # a 256-byte aligned address that is never dereferenced


# ---------------------------------------------------------------------------
# the oracle

def _pools(rng, pages, heads, page, dim):
    return rng.standard_normal((pages, heads, page, dim)), rng.standard_normal((pages, heads, page, dim))


def test_attend_equal_scores_average_the_values():
    rng = np.random.default_rng(0)
    k, v = _pools(rng, 4, 2, 4, 8)
    q = np.zeros((1, 4, 8))
    table = np.array([[2, 0, 3]])
    out, acc = okv.attend(q, k, v, table, [6], 1.0, acc=np.ones((1, 2, 12)), decay=0.5)
    for h in range(2):
        want = np.concatenate([v[2, h], v[0, h, :2]]).mean(axis=0)
        assert np.allclose(out[0, 2 * h], want) and np.allclose(out[0, 2 * h + 1], want)
    assert np.allclose(acc[0, :, :6], 0.5 + 2 / 6) and np.all(acc[0, :, 6:] == 1.0)


def test_attend_one_slot_empty_row_and_two_slots():
    rng = np.random.default_rng(1)
    k, v = _pools(rng, 3, 1, 2, 4)
    q = rng.standard_normal((3, 1, 4))
    out, _ = okv.attend(q, k, v, np.array([[0], [1], [2]]), [0, 1, 2], 0.7)
    assert np.all(out[0] == 0)
    assert np.allclose(out[1, 0], v[1, 0, 0])
    d = 0.7 * float(q[2, 0] @ (k[2, 0, 1] - k[2, 0, 0]))
    w = 1 / (1 + math.exp(-d))  # two scores: the logistic function of their difference
    assert np.allclose(out[2, 0], (1 - w) * v[2, 0, 0] + w * v[2, 0, 1])


def test_attend_order_of_slots_does_not_matter_and_minus_infinity_weighs_nothing():
    rng = np.random.default_rng(2)
    k, v = _pools(rng, 2, 1, 4, 4)
    q = np.abs(rng.standard_normal((1, 2, 4)))
    a, _ = okv.attend(q, k, v, np.array([[0, 1]]), [8], 0.5)
    perm = rng.permutation(8)
    k2, v2 = (x.reshape(8, 4)[perm].reshape(x.shape) for x in (k, v))
    assert np.allclose(a, okv.attend(q, k2, v2, np.array([[0, 1]]), [8], 0.5)[0])
    k[1, 0, 3, 0] = -np.inf
    assert np.allclose(okv.attend(q, k, v, np.array([[0, 1]]), [8], 0.5)[0],
                       okv.attend(q, k, v, np.array([[0, 1]]), [7], 0.5)[0])
    # a page that is not there: as if its slots were not
    assert np.allclose(okv.attend(q, k, v, np.array([[-1, 0]]), [8], 0.5)[0],
                       okv.attend(q, k, v, np.array([[0, 1]]), [4], 0.5)[0])


def test_turning_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(3)
    angle = np.arange(20)[:, None] * np.array([1.0, 0.3])[None]
    rope = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    a, b = rng.standard_normal((2, 1, 4))
    assert np.allclose(okv.turned(a, 0, rope, None, 0), a)
    t = [okv.turned(x, p, rope, None, 0) for x, p in ((a, 3), (b, 7), (a, 12), (b, 16))]
    assert np.allclose((t[0] ** 2).sum(), (a ** 2).sum())
    assert np.allclose((t[0] * t[1]).sum(), (t[2] * t[3]).sum())  # both 4 positions apart
    x = okv.turned(a, 5, None, np.full(4, 2.0), 0.0)
    assert np.allclose((x ** 2).mean(), 4.0) and np.isnan(okv.turned(a, 20, rope, None, 0)).all()


def test_append_places_tokens_and_drops_what_does_not_fit():
    k0, v0 = np.zeros((3, 1, 2, 4)), np.zeros((3, 1, 2, 4))
    new = np.arange(1, 6)[:, None, None] * np.ones((5, 1, 4))
    k, v, _, pos, acc, lens = okv.append(k0, v0, np.array([[2, 0], [1, 9]]), [1, 0], [0, 2, 5], [11, 12, 13, 14, 15],
                                         new, -new, pos=np.zeros((2, 1, 4)), acc=np.ones((2, 1, 4)))
    assert k[:, 0, :, 0].tolist() == [[2, 0], [3, 4], [0, 1]] and np.array_equal(v, -k)
    assert pos[:, 0].tolist() == [[0, 11, 12, 0], [13, 14, 0, 0]]
    assert acc[:, 0].tolist() == [[1, 0, 0, 1], [0, 0, 1, 1]] and lens.tolist() == [3, 3]


def test_append_bounds_the_lengths():
    k0 = np.zeros((3, 1, 2, 4))
    new = np.arange(1, 6)[:, None, None] * np.ones((5, 1, 4))
    k, _, _, pos, _, lens = okv.append(k0, k0, np.array([[2], [1], [0]]), [-7, 9, 1], [0, 2, 3, 5], [11, 12, 13, 14, 15], new, new,
                                       pos=np.zeros((3, 1, 2)))
    assert k[:, 0, :, 0].tolist() == [[0, 4], [0, 0], [1, 2]]  # row 0 from slot 0 on, row 1 is full, row 2's second does not fit
    assert pos[:, 0].tolist() == [[11, 12], [0, 0], [0, 14]] and lens.tolist() == [2, 3, 3]


def test_evict_worked_example():
    acc = np.array([[[5.0, 1.0, 3.0, 3.0, np.nan, 9.0, 3.0, 0.0]]])
    pos = np.arange(8).reshape(1, 1, 8)
    k = np.arange(8.0).reshape(4, 1, 2, 1)
    args = (k, -k, np.array([[0, 1, 2, 3]]), [8], acc, pos)
    blank = np.full((1, 1, 8), -1.0), np.full((1, 1, 8), -1)
    # budget 4, no one protected: 5 (9.0), 0 (5.0), then the lowest two of the equals 2, 3, 6
    k2, v2, a2, p2, lens = okv.evict(*args, 4, 0, 0, *blank)
    assert k2.ravel()[:4].tolist() == [0, 5, 2, 3] and np.array_equal(v2, -k2)
    assert a2[0, 0].tolist() == [5, 9, 3, 3, -1, -1, -1, -1] and p2[0, 0, :4].tolist() == [0, 5, 2, 3]
    assert lens.tolist() == [4]
    # the first two positions and the last one stay: 0, 1, 7 and then 5
    k2, _, a2, p2, _ = okv.evict(*args, 4, 2, 1, *blank)
    assert k2.ravel()[:4].tolist() == [0, 1, 5, 7] and p2[0, 0, :4].tolist() == [0, 1, 5, 7]
    # within the budget nothing moves
    k2, _, a2, p2, lens = okv.evict(*args, 8, 0, 0, *blank)
    assert np.array_equal(k2, k) and lens.tolist() == [8] and p2[0, 0].tolist() == list(range(8))


def test_evict_protected_slots_come_before_infinite_totals():
    inf = np.inf
    k = np.arange(6.0).reshape(3, 1, 2, 1)
    blank = np.full((1, 1, 6), -1.0), np.full((1, 1, 6), -1)
    k2, _, a2, p2, _ = okv.evict(k, -k, np.array([[0, 1, 2]]), [6], np.array([[[inf, inf, inf, 1.0, -inf, 0.0]]]),
                                 np.array([[[4, 3, 1, 2, 0, 5]]]), 3, 1, 1, *blank)
    assert k2.ravel()[:3].tolist() == [0, 4, 5] and p2[0, 0].tolist() == [4, 0, 5, -1, -1, -1]
    assert a2[0, 0].tolist() == [inf, -inf, 0, -1, -1, -1]


# ---------------------------------------------------------------------------
# refusals

@pytest.fixture(scope="module")
def lib():
    return nbw.library()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, pages=10, heads=2, page=16, dim=128, dtype=0, k_scale=None, v_scale=None, table=FAKE,
             rows=3, width=5, table_ld=0)
    return kv.KVView(**{**f, **kw})


BAD_CACHES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(table=None), EINVAL), (dict(dim=96), EUNSUPPORTED),
    (dict(dtype=2), EUNSUPPORTED), (dict(page=0), EUNSUPPORTED), (dict(page=24), EUNSUPPORTED),
    (dict(page=8192), EUNSUPPORTED), (dict(heads=0), EINVAL), (dict(heads=1025), EINVAL), (dict(pages=0), EINVAL),
    (dict(pages=1 << 31), EINVAL), (dict(rows=-1), EINVAL), (dict(width=0), EINVAL), (dict(width=1 << 27), EINVAL),
    (dict(table_ld=4), EINVAL), (dict(dtype=1), EINVAL), (dict(dtype=1, k_scale=FAKE), EINVAL),
    (dict(k_scale=FAKE, v_scale=FAKE), EINVAL), (dict(k=FAKE + 8), EALIGN), (dict(v=FAKE + 2), EALIGN),
    (dict(table=FAKE + 2), EALIGN), (dict(dtype=1, k_scale=FAKE + 1, v_scale=FAKE), EALIGN),
]


def append_args(**kw):
    f = dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, tokens=3, q_heads=4, eps=1e-6, lens=FAKE, positions=FAKE)
    return kv.AppendArgs(**{**f, **kw})


def attend_args(**kw):
    f = dict(q=FAKE, out=FAKE, q_heads=4, lens=FAKE, workspace=None, workspace_bytes=0)
    return kv.AttendArgs(**{**f, **kw})


def evict_args(**kw):
    f = dict(acc=FAKE, pos=FAKE, lens=FAKE, budget=40, sink=4, recent=8, acc_out=FAKE + 256, pos_out=FAKE + 256,
             lens_out=FAKE + 256)
    return kv.EvictArgs(**{**f, **kw})


def call(lib, name, c, a):
    return getattr(lib, name)(None if c is None else ctypes.byref(c), None if a is None else ctypes.byref(a), None)


@pytest.mark.parametrize("name,args", [("nbw_kv_append", append_args), ("nbw_kv_attend", attend_args),
                                       ("nbw_kv_evict", evict_args)])
def test_bad_caches_are_refused(lib, name, args):
    assert call(lib, name, None, args()) == EINVAL
    assert call(lib, name, cache(), None) == EINVAL
    for change, status in BAD_CACHES:
        assert call(lib, name, cache(**change), args()) == status, change


@pytest.mark.parametrize("change,status", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(positions=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(q_out=None), EINVAL), (dict(tokens=-1), EINVAL), (dict(tokens=4), EINVAL), (dict(tokens=1 << 31), EINVAL),
    (dict(q_heads=3), EINVAL), (dict(q_heads=0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
    (dict(rope=FAKE), EINVAL), (dict(k_ld=128), EINVAL), (dict(k_ld=260), EALIGN), (dict(q_ld=508), EINVAL),
    (dict(v_ld=264 + 4), EALIGN), (dict(q_out_ld=516), EALIGN), (dict(lens_out=FAKE), EINVAL),
    (dict(k=FAKE + 2), EALIGN), (dict(q=FAKE + 8), EALIGN), (dict(rope=FAKE + 4, rope_rows=9), EALIGN),
    (dict(q_norm=FAKE + 2), EALIGN), (dict(lens=FAKE + 1), EALIGN), (dict(pos=FAKE + 2), EALIGN),
])
def test_bad_append_arguments_are_refused(lib, change, status):
    assert call(lib, "nbw_kv_append", cache(), append_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(lens=None), EINVAL), (dict(q_heads=5), EINVAL),
    (dict(q_heads=0), EINVAL), (dict(q_heads=2 * 257), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(scale=math.inf), EINVAL), (dict(max_len=-1), EINVAL), (dict(acc=FAKE), EINVAL), (dict(acc_out=FAKE), EINVAL),
    (dict(acc=FAKE, acc_out=FAKE, decay=math.nan), EINVAL), (dict(q_ld=256), EINVAL), (dict(out_ld=516), EALIGN),
    (dict(q=FAKE + 2), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(lens=FAKE + 2), EALIGN),
    (dict(workspace=FAKE + 16), EALIGN), (dict(workspace_bytes=-1), EINVAL),
])
def test_bad_attend_arguments_are_refused(lib, change, status):
    assert call(lib, "nbw_kv_attend", cache(), attend_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(acc=None), EINVAL), (dict(pos=None), EINVAL), (dict(lens=None), EINVAL), (dict(acc_out=None), EINVAL),
    (dict(acc_out=FAKE), EINVAL), (dict(pos_out=FAKE), EINVAL), (dict(lens_out=FAKE), EINVAL),
    (dict(budget=0), EINVAL), (dict(budget=81), EINVAL), (dict(sink=-1), EINVAL), (dict(recent=-1), EINVAL),
    (dict(sink=33), EINVAL), (dict(recent=1 << 62), EINVAL), (dict(max_len=-5), EINVAL),
    (dict(acc=FAKE + 2), EALIGN), (dict(pos_out=FAKE + 2), EALIGN), (dict(workspace=FAKE + 4), EALIGN),
    (dict(workspace_bytes=-1), EINVAL),
])
def test_bad_evict_arguments_are_refused(lib, change, status):
    assert call(lib, "nbw_kv_evict", cache(), evict_args(**change)) == status


def test_a_missing_or_small_workspace_is_refused(lib):
    # 320 slots brought down to 100: more moves than the ranking's workgroup makes itself
    big = cache(width=20)
    assert call(lib, "nbw_kv_evict", big, evict_args(budget=100)) == ESCRATCH
    assert call(lib, "nbw_kv_evict", big, evict_args(budget=100, workspace=FAKE, workspace_bytes=8)) == ESCRATCH
    need = lib.nbw_kv_evict_workspace_bytes(ctypes.byref(big), 100, 0)
    assert call(lib, "nbw_kv_evict", big, evict_args(budget=100, workspace=FAKE, workspace_bytes=need - 1)) == ESCRATCH


def test_empty_batches_queue_nothing(lib):
    none = cache(rows=0)
    assert call(lib, "nbw_kv_append", none, append_args(tokens=0)) == OK
    assert call(lib, "nbw_kv_append", none, append_args(tokens=2)) == EINVAL
    assert call(lib, "nbw_kv_attend", none, attend_args(q=None)) == OK
    assert call(lib, "nbw_kv_evict", none, evict_args(acc=None)) == OK


def test_a_batch_without_rows_needs_no_table(lib):
    none = cache(rows=0, table=None)
    assert call(lib, "nbw_kv_append", none, append_args(tokens=0)) == OK
    assert call(lib, "nbw_kv_attend", none, attend_args(q=None, out=None, lens=None)) == OK
    assert call(lib, "nbw_kv_evict", none, evict_args(acc=None)) == OK
    assert lib.nbw_kv_evict_workspace_bytes(ctypes.byref(none), 40, 0) == 0
    assert call(lib, "nbw_kv_attend", cache(rows=-1, table=None), attend_args()) == EINVAL


def test_workspace_sizes_refuse_bad_arguments(lib):
    c = cache()
    assert lib.nbw_kv_attend_workspace_bytes(ctypes.byref(c), 5, 0, 0) == -1
    assert lib.nbw_kv_attend_workspace_bytes(ctypes.byref(c), 4, -1, 0) == -1
    assert lib.nbw_kv_attend_workspace_bytes(ctypes.byref(cache(dim=80)), 4, 0, 0) == -1
    assert lib.nbw_kv_evict_workspace_bytes(ctypes.byref(c), 0, 0) == -1
    assert lib.nbw_kv_evict_workspace_bytes(ctypes.byref(c), 81, 0) == -1
    assert lib.nbw_kv_evict_workspace_bytes(ctypes.byref(c), 40, 40) == 0
    assert lib.nbw_kv_evict_workspace_bytes(ctypes.byref(cache(width=20)), 100, 0) > 0


def test_more_than_a_launch_takes_is_refused_before_anything_is_queued(lib):
    size = lib.nbw_kv_evict_workspace_bytes
    many = dict(rows=1 << 20, width=1, page=16)
    assert size(ctypes.byref(cache(**many, heads=15)), 8, 0) == 0
    assert size(ctypes.byref(cache(**many, heads=16)), 8, 0) == -1    # 2^24 workgroups of 256 threads
    assert size(ctypes.byref(cache(rows=1 << 20, width=256, page=16, heads=8)), 8, 0) == -1   # 2^23 of 512
    assert size(ctypes.byref(cache(rows=1 << 20, width=512, page=16, heads=4)), 8, 0) == -1   # 2^22 of 1024
    assert size(ctypes.byref(cache(rows=1 << 14, width=4096, page=1024, heads=1)), 8, 0) == -1  # 1024 parts each
    assert call(lib, "nbw_kv_evict", cache(**many, heads=16), evict_args(budget=8, sink=0)) == EINVAL
    # a move launch is never more than one takes: 64 x 8 rows of 2^20 slots brought down to half
    assert size(ctypes.byref(cache(rows=64, heads=8, width=4096, page=256)), 1 << 19, 0) > 0
    for tokens in ((1 << 24) - (1 << 13) + 1, 1 << 24, (1 << 31) - (1 << 20)):
        assert call(lib, "nbw_kv_append", cache(), append_args(cu=FAKE, tokens=tokens, k=FAKE + 2)) == EINVAL
    assert call(lib, "nbw_kv_append", cache(), append_args(cu=FAKE, tokens=(1 << 24) - (1 << 13), k=FAKE + 2)) == EALIGN


def test_workspace_sizes_that_a_cache_remembers_are_few():
    c = nbw.KVCache.__new__(nbw.KVCache)
    c._sizes, c._ref, c._dev = {}, None, 0
    asked = []

    def query(ref, *sizes):
        asked.append(sizes)
        return 0

    for step in range(1, 2000):  # a bound of the lengths that grows with every token
        assert c._scratch("auto", query, (32, step, True), 0) == (None, 0)
        assert len(c._sizes) <= kv.SIZES_KEPT
    last = len(asked)
    for _ in range(3):
        c._scratch("auto", query, (32, 1999, True), 0)
    assert last == 1999 and len(asked) == last


def test_binding_refuses_cpu_tensors():
    pool = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nbw.KVCache(pool, pool.clone(), torch.zeros((1, 1), dtype=torch.int32))
    with pytest.raises(TypeError):
        nbw.KVCache(None, pool, torch.zeros((1, 1), dtype=torch.int32))
