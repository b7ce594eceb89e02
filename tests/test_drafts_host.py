"""Host-side checks of a step with drafted tokens: no GPU, no device work queued.

The oracle is pinned by cases whose answers follow from the definitions without it;
the entry points reject every bad argument before any HIP call.
"""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import nested_bit_weight_amd as nbw
from nested_bit_weight_amd import drafts, kv
from oracle import drafts as odrafts
from oracle import kv as okv

OK, EINVAL, EALIGN, EUNSUPPORTED, ESCRATCH = 0, 1, 2, 4, 6
FAKE = 0x7F0000001000  # a 256-byte aligned address that is never dereferenced
OTHER = FAKE + 4096


# ---------------------------------------------------------------------------
# the oracle

def test_reserve_worked_example():
    # pages of 4 slots; row 0 has pages 5 and 6 and needs a third, row 1 gives back 8 and 9, row 2 starts
    table = np.array([[5, 6, -1, -1], [7, 8, 9, -1], [-1, -1, -1, -1]])
    out = okv.reserve(table, 4, 10, [7, 2, 0], [3, 1, 5], [2, 3, 0], np.array([1, 2, 3, 0, 0, 0]), 3, 12)
    table2, free, cu, positions, slots, granted, held, count = out
    # the stack is 1 2 3 9 8: 8, the first one given back, on top
    assert table2.tolist() == [[5, 6, 8, -1], [7, 8, 9, -1], [9, 3, -1, -1]]
    assert granted == [3, 1, 5] and held == [3, 1, 2] and count == 2 and free.tolist() == [1, 2, 3, 0, 0, 0]
    assert cu.tolist() == [0, 3, 4, 9]
    assert positions.tolist() == [7, 8, 9, 2, 0, 1, 2, 3, 4, 0, 0, 0]
    assert slots.tolist() == [27, 32, 33, 30, 36, 37, 38, 39, 12, -1, -1, -1]


def test_reserve_serves_in_order_until_something_lacks():
    table = np.full((4, 3), -1)
    args = (table, 2, 9, [0, 0, 0, 0], [2, 5, 1, 0], [0] * 4, np.array([3, 4, 5]), 3)
    assert okv.reserve(*args, 99)[5] == [2, 0, 0, 0]      # three pages for row 1: two are left, and row 2 waits too
    assert okv.reserve(*args[:7], 4, 99)[5] == [2, 0, 0, 0]  # a count of 4 is bounded by the stack of 3
    more = (table, 2, 9, [0, 0, 0, 0], [2, 5, 1, 0], [0] * 4, np.array([3, 4, 5, 6, 7]), 5)
    assert okv.reserve(*more, 99)[5] == [2, 5, 1, 0] and okv.reserve(*more, 7)[5] == [2, 5, 0, 0]
    assert okv.reserve(*more, 6)[5] == [2, 0, 0, 0]
    assert okv.reserve(table[:1], 2, 9, [5], [2], [0], np.array([3, 4, 5]), 3, 9)[5] == [0]  # past the capacity: not asked for


def test_reserve_leaves_shared_pages_with_the_row():
    table = np.array([[1, 2, 3]])
    out = okv.reserve(table, 4, 9, [0], [0], [3], np.array([0, 0, 0]), 0, 0, shared=[2])
    assert out[6] == [2] and out[7] == 1 and out[1][0] == 3


def test_attend_tokens_sees_the_past_and_itself():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 3, 1, 4, 8))
    q = rng.standard_normal((5, 2, 8))
    table = np.array([[2, 0], [1, 1]])
    out = okv.attend_tokens(q, k, v, table, [6, 2], [0, 3, 5], 0.3)
    for t, (row, n) in enumerate([(0, 4), (0, 5), (0, 6), (1, 1), (1, 2)]):
        assert np.array_equal(out[t], okv.attend(q[t:t + 1], k, v, table[row:row + 1], [n], 0.3)[0][0])
    assert np.allclose(out[3, 0], v[1, 0, 0])  # one slot only
    flat = okv.attend_tokens(0 * q, k, v, table, [6, 2], [0, 3, 5], 0.3)
    assert np.allclose(flat[2, 1], np.concatenate([v[2, 0], v[0, 0, :2]]).mean(axis=0))
    assert np.all(okv.attend_tokens(q, k, v, table, [2, 2], [0, 3, 5], 0.3)[0] == 0)  # three tokens, two slots: the first sees none


def test_verified_tokens_are_distributed_as_the_target():
    p, q = np.array([[0.5, 0.125, 0.375]] * 2), np.array([[0.25, 0.5, 0.25]] * 2)
    odds = [Fraction(0)] * 3
    for x in range(3):
        for u in (0.0, 0.25, 0.5, 0.75):            # 4 places, of which token 1 stands in one (p / q = 1 / 4)
            for v in (0.0, 0.34, 0.67):             # p - q is 2 / 8 for token 0 and 1 / 8 for token 2
                accepted, after = odrafts.verify(p, [9, x], [u, v], [0, 2], q)
                odds[x if accepted[0] else after[0]] += Fraction(float(q[0, x])) / 12
    assert odds == [Fraction(1, 2), Fraction(1, 8), Fraction(3, 8)]


def test_verify_closed_forms():
    p = np.array([[0.25, 0.75], [0.0, 1.0], [1.0, 0.0]])
    # looked-up drafts stand if u < p; the next token is drawn from the last line
    assert odrafts.verify(p, [0, 1, 1], [0.5, 0.5, 0.5], [0, 3]) == ([2], [0])
    assert odrafts.verify(p, [0, 0, 1], [0.25, 0.5, 0.5], [0, 3]) == ([0], [1])   # 0.25 < 0.25 does not hold; 0 is left out
    assert odrafts.verify(p, [0, 0, 1], [0.2, 0.5, 0.5], [0, 3]) == ([2], [0])
    assert odrafts.verify(p, [0, 1, 0], [0.5, 0.0, 0.5], [0, 3]) == ([1], [1])    # p of token 0 is 0 there
    assert odrafts.verify(p, [0, 2, 1], [0.0, 0.0, 0.5], [0, 3]) == ([0], [1])    # outside the vocabulary
    # p = q: nothing is above 0 in their difference, so p itself
    assert odrafts.verify(p[:2], [0, 0], [1.0, 0.1], [0, 2], p[:2]) == ([0], [0])
    assert odrafts.verify(p, [0, 0, 0], [0.3, 0.2, 0.0], [0, 1, 1, 3]) == ([0, 0, 0], [1, -1, 1])
    assert odrafts.verify(0 * p, [0, 0, 0], [0.3, 0.2, 0.0], [0, 1, 2, 3]) == ([0, 0, 0], [-1, -1, -1])
    assert odrafts.verify(p[:1], [0], [1.0], [0, 1]) == ([0], [1])                # u = 1: the last that has a weight


# ---------------------------------------------------------------------------
# refusals

@pytest.fixture(scope="module")
def lib():
    return nbw.library()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, pages=10, heads=2, page=16, dim=128, dtype=0, k_scale=None, v_scale=None, table=FAKE,
             rows=3, width=5, table_ld=0)
    return kv.KVView(**{**f, **kw})


def reserve_args(**kw):
    f = dict(table=FAKE, lens=FAKE, want=FAKE, held=FAKE, free=FAKE, free_size=10, count=FAKE, max_tokens=9, cu=FAKE, positions=FAKE,
             slots=FAKE, granted=FAKE, held_out=OTHER, count_out=OTHER)
    return kv.ReserveArgs(**{**f, **kw})


def shared_args(**kw):
    f = dict(q=FAKE, out=FAKE, tokens=3, q_heads=4, lens=FAKE)
    return kv.AttendSharedArgs(**{**f, **kw})


def verify_args(**kw):
    f = dict(target=FAKE, tokens=3, vocab=100, rows=3, u=FAKE, accepted=FAKE, next=OTHER)
    return drafts.VerifyArgs(**{**f, **kw})


def call(lib, name, c, a):
    return getattr(lib, name)(None if c is None else ctypes.byref(c), None if a is None else ctypes.byref(a), None)


BAD_CACHES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(table=None), EINVAL), (dict(dim=96), EUNSUPPORTED),
    (dict(dtype=2), EUNSUPPORTED), (dict(page=24), EUNSUPPORTED), (dict(page=8192), EUNSUPPORTED), (dict(heads=0), EINVAL),
    (dict(pages=0), EINVAL), (dict(rows=-1), EINVAL), (dict(width=0), EINVAL), (dict(table_ld=4), EINVAL),
    (dict(dtype=1), EINVAL), (dict(k=FAKE + 8), EALIGN), (dict(table=FAKE + 2), EALIGN),
]


@pytest.mark.parametrize("name,args", [("nbw_kv_reserve", reserve_args), ("nbw_kv_attend_shared", shared_args)])
def test_bad_caches_are_refused(lib, name, args):
    assert call(lib, name, None, args()) == EINVAL
    assert call(lib, name, cache(), None) == EINVAL
    for change, status in BAD_CACHES:
        assert call(lib, name, cache(**change), args()) == status, change


@pytest.mark.parametrize("change,status", [
    *[({name: None}, EINVAL) for name in ("lens", "want", "held", "free", "count", "cu", "positions", "slots", "granted", "held_out",
                                          "count_out")],
    *[({name: FAKE + 2}, EALIGN) for name in ("lens", "want", "held", "shared", "seen", "free", "count", "cu", "positions", "granted",
                                              "held_out", "count_out")],
    (dict(table=None), EINVAL), (dict(table=OTHER), EINVAL), (dict(slots=FAKE + 4), EALIGN), (dict(free_size=0), EINVAL),
    (dict(free_size=(1 << 30) + 1), EINVAL), (dict(max_tokens=-1), EINVAL), (dict(max_tokens=1 << 24), EINVAL),
    (dict(held_out=FAKE), EINVAL), (dict(count_out=FAKE), EINVAL),
])
def test_bad_reserve_arguments_are_refused(lib, change, status):
    assert call(lib, "nbw_kv_reserve", cache(), reserve_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(lens=None), EINVAL), (dict(q_heads=5), EINVAL),
    (dict(q_heads=0), EINVAL), (dict(q_heads=2 * 257), EINVAL), (dict(scale=math.nan), EINVAL), (dict(scale=-math.inf), EINVAL),
    (dict(max_len=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(tokens=4), EINVAL), (dict(tokens=1 << 24, cu=FAKE), EINVAL),
    (dict(tokens=1 << 23, q_heads=256, cu=FAKE), EINVAL), (dict(groups=-1), EINVAL), (dict(groups=2), EINVAL),
    (dict(groups=2, group_rows=FAKE), EINVAL), (dict(groups=2, prefix=FAKE), EINVAL),
    (dict(groups=(1 << 20) + 1, group_rows=FAKE, prefix=FAKE), EINVAL), (dict(q_ld=256), EINVAL), (dict(out_ld=516), EALIGN),
    (dict(q_ld=516), EALIGN), (dict(q=FAKE + 2), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(lens=FAKE + 2), EALIGN),
    (dict(cu=FAKE + 1), EALIGN), (dict(groups=1, group_rows=FAKE + 2, prefix=FAKE), EALIGN),
    (dict(groups=1, group_rows=FAKE, prefix=FAKE + 2), EALIGN), (dict(workspace=FAKE + 16), EALIGN),
    (dict(workspace_bytes=-1), EINVAL),
])
def test_bad_attention_arguments_are_refused(lib, change, status):
    assert call(lib, "nbw_kv_attend_shared", cache(), shared_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(target=None), EINVAL), (dict(u=None), EINVAL), (dict(accepted=None), EINVAL), (dict(next=None), EINVAL),
    (dict(next=FAKE), EINVAL), (dict(dtype=2), EUNSUPPORTED), (dict(dtype=-1), EUNSUPPORTED), (dict(vocab=0), EINVAL),
    (dict(vocab=(1 << 30) + 1), EINVAL), (dict(rows=-1), EINVAL), (dict(rows=(1 << 20) + 1), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(tokens=4), EINVAL), (dict(tokens=1 << 24, cu=FAKE, ids=FAKE), EINVAL), (dict(rows=0), EINVAL),
    (dict(cu=FAKE), EINVAL), (dict(target_ld=99), EINVAL), (dict(draft_ld=99), EINVAL), (dict(target_ld=1 << 33), EINVAL),
    (dict(target=FAKE + 2), EALIGN), (dict(draft=FAKE + 2), EALIGN), (dict(target=FAKE + 1, dtype=1), EALIGN),
    (dict(cu=FAKE + 2, ids=FAKE), EALIGN), (dict(cu=FAKE, ids=FAKE + 2), EALIGN), (dict(u=FAKE + 2), EALIGN),
    (dict(accepted=FAKE + 2), EALIGN), (dict(next=FAKE + 2), EALIGN), (dict(workspace=FAKE + 128), EALIGN),
    (dict(workspace_bytes=-1), EINVAL), (dict(), ESCRATCH), (dict(workspace=FAKE, workspace_bytes=23), ESCRATCH),
    (dict(target=FAKE + 2, dtype=1), ESCRATCH),
])
def test_bad_verification_arguments_are_refused(lib, change, status):
    assert lib.nbw_verify_drafts(ctypes.byref(verify_args(**change)), None) == status


def test_verification_without_arguments_and_without_rows(lib):
    assert lib.nbw_verify_drafts(None, None) == EINVAL
    assert lib.nbw_verify_drafts(ctypes.byref(verify_args(rows=0, tokens=0, target=None, u=None, accepted=None, next=None)), None) == OK


def test_batches_without_rows_or_tokens_queue_nothing(lib):
    assert call(lib, "nbw_kv_attend_shared", cache(rows=0, table=None), shared_args(tokens=0, q=None, out=None, lens=None)) == OK
    assert call(lib, "nbw_kv_attend_shared", cache(), shared_args(tokens=0, cu=FAKE, q=None, out=None, lens=None)) == OK


def test_workspace_sizes(lib):
    size = lib.nbw_kv_attend_shared_workspace_bytes

    def of(c, *a):
        return size(ctypes.byref(c), *a)

    assert of(cache(rows=0), 4, 0, 0, 0) == 0 and of(cache(), 4, 0, 0, 0) == 0
    for c, a in ((cache(dim=80), (4, 3, 0, 0)), (cache(), (5, 3, 0, 0)), (cache(), (4, -1, 0, 0)), (cache(), (4, 3, -1, 0)),
                 (cache(), (4, 3, (1 << 20) + 1, 0)), (cache(), (4, 3, 0, -1)), (cache(), (4, 1 << 24, 0, 0))):
        assert of(c, *a) == -1
    assert lib.nbw_verify_drafts_workspace_bytes(3, 1024) == 24 and lib.nbw_verify_drafts_workspace_bytes(3, 1025) == 48
    for rows, vocab in ((-1, 5), (1 << 21, 5), (5, 0), (5, 1 << 31), (1 << 20, 1 << 20)):
        assert lib.nbw_verify_drafts_workspace_bytes(rows, vocab) == -1


def test_binding_refuses_what_is_no_gpu_tensor():
    p, u = torch.zeros((2, 5)), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        nbw.verify_drafts(p, None, u)
    with pytest.raises(TypeError):
        nbw.verify_drafts([[0.5]], None, u)
    with pytest.raises(ValueError):
        drafts.verify_workspace_bytes(-1, 5)
