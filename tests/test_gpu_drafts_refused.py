"""GPU check of examples/speculative_decode.py where a reservation does not serve all rows.

Rows that are granted nothing lie between others, whose tokens are packed; every call of a step is checked from
the tensors that it used, whole numbers for equality, attention within the tolerance derived in test_gpu_drafts.Shared.check.
"""
import numpy as np
import pytest
import torch

from oracle import drafts as odrafts
from oracle import kv as okv
from test_gpu_drafts_example import example, f64

pytestmark = pytest.mark.gpu
ROWS, DRAFTS, PAGE, PROMPT, VOCAB = 6, 3, 8, 48, 384


def start(ex, room=64):
    s = ex.Speculation(ROWS, DRAFTS, r_draft=4, heads=4, kv=2, dim=64, vocab=VOCAB, page=PAGE, room=room, prompt=PROMPT, seed=2)
    s.read_prompt(torch.randint(0, VOCAB, (PROMPT,), generator=s.gen, device="cuda", dtype=torch.int32))
    return s


def grow(ex, s, by):
    """Rows that hold `by` slots more (of zeros)."""
    want = torch.tensor(by, dtype=torch.int32, device="cuda")
    got = ex.nbw.kv_reserve(s.cache, s.lens, want, s.held, s.free, s.count, sum(by), shared=s.shared)
    assert torch.equal(got.granted, want)
    s.lens, s.held, s.count = s.lens + want, got.held, got.count


def slots(s, lens):
    """What each row has in the cache, bit for bit."""
    table, out = s.table.long(), []
    for r, n in enumerate(lens.tolist()):
        j = torch.arange(n, device="cuda")
        at = table[r, j // PAGE], j % PAGE
        out.append([pool.view(torch.int16)[at[0], :, at[1]].clone() for pool in (s.cache.k, s.cache.v)])
    return out


def checked_step(ex, s, monkeypatch):
    """One step, its calls checked; the granted tokens of every row."""
    before, last, held = s.lens.clone(), s.last.clone(), slots(s, s.lens)
    seen = {}
    reserve, attend, verify = ex.nbw.kv_reserve, ex.nbw.kv_attend_shared, ex.nbw.verify_drafts

    def spy_reserve(*a, **kw):
        seen["got"] = reserve(*a, **kw)
        return seen["got"]

    def spy_attend(cache, q, lens, cu=None, groups=None, prefix=None):
        out = attend(cache, q, lens, cu=cu, groups=groups, prefix=prefix)
        live = (seen["got"].granted > 0).cpu().numpy()
        tokens = np.where(live, 1 if cu is None else DRAFTS + 1, 0)
        cut = np.concatenate([[0], np.cumsum(tokens)])
        mine = np.flatnonzero(live) if cu is None else np.arange(cut[-1])
        k, v, qq, table, n = f64(cache.k), f64(cache.v), f64(q)[mine], cache.table.cpu().numpy(), lens.cpu().numpy()
        want = okv.attend_tokens(qq, k, v, table, n, cut, 0.125)
        mean = okv.attend_tokens(qq, k, np.abs(v), table, n, cut, 0.125)
        size = np.abs(qq).sum(axis=2).max(initial=0) * np.abs(k).max() * 0.125
        bound = 2.0**-8 * np.abs(want) + (2.0**-8 + 2 * 16 * 2.0**-24 * size) * mean + 1e-30
        assert np.all(np.abs(f64(out)[mine] - want) <= bound)
        return out

    def spy_verify(target, ids, u, draft=None, cu=None):
        got = verify(target, ids, u, draft=draft, cu=cu)
        if cu is not None:
            cut = cu.tolist()
            first = {r: int(ids[cut[r]]) for r in range(ROWS) if cut[r + 1] > cut[r]}
            assert first == {r: int(last[r]) for r in first}  # each row's certain token in its own place
            ref = odrafts.verify(f64(target), ids.tolist(), f64(u), cut, f64(draft))
            assert got[0].tolist() == ref[0] and got[1].tolist() == ref[1]
        return got

    with monkeypatch.context() as m:
        m.setattr(ex.nbw, "kv_reserve", spy_reserve)
        m.setattr(ex.nbw, "kv_attend_shared", spy_attend)
        m.setattr(ex.nbw, "verify_drafts", spy_verify)
        accepted, after = s.step()
    granted = seen["got"].granted
    served = granted > 0
    assert torch.equal(s.lens, torch.where(served, before + accepted + 1, before)) and bool((s.lens <= s.cache.capacity).all())
    assert bool(((after >= 0) & (after < VOCAB)).all())
    assert torch.equal(after[~served], last[~served]) and not bool(accepted[~served].any())
    # what was in the cache is as it was, whoever's it is
    for a, b in zip(held, slots(s, before)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    return granted.tolist()


def test_rows_at_their_capacity_between_others(monkeypatch):
    ex = example()
    s = start(ex)
    grow(ex, s, [0, 64, 0, 61, 50, 0])
    for step in range(12):
        granted = checked_step(ex, s, monkeypatch)
        assert granted[1] == 0 and granted[3] == 0  # full, and with no room for all its drafts
    assert granted[0] and granted[4] == 0  # 14 slots were left to row 4: it stops on the way


@pytest.mark.parametrize("left", [0, 1, 3, 5])
def test_a_pool_that_is_too_small(monkeypatch, left):
    """Pages for the first rows only; a row that is full lies among them."""
    ex = example()
    s = start(ex)
    grow(ex, s, [0, 64, 0, 0, 0, 0])
    s.count.fill_(left)
    first = checked_step(ex, s, monkeypatch)
    assert first == [4 if r < left + (left > 1) and r != 1 else 0 for r in range(ROWS)]
    for _ in range(6):
        checked_step(ex, s, monkeypatch)


def test_places_of_a_reservation_follow_from_cu():
    """Row and number of each token, as the documentation says."""
    import nested_bit_weight_amd as nbw
    pool = torch.zeros((40, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = nbw.KVCache(pool, pool, torch.full((5, 4), -1, dtype=torch.int32, device="cuda"))
    got = nbw.kv_reserve(cache, ints(0, 0, 0, 0, 0), ints(3, 17, 0, 5, 2), ints(0, 0, 0, 0, 0), torch.arange(40, dtype=torch.int32, device="cuda"),
                         ints(40), 12)
    assert got.granted.tolist() == [3, 0, 0, 5, 2]
    t = torch.arange(10, device="cuda", dtype=torch.int32)
    row = torch.searchsorted(got.cu[1:], t, right=True)
    assert row.tolist() == [0] * 3 + [3] * 5 + [4] * 2
    assert (t - got.cu[row]).tolist() == got.positions[:10].tolist() == [0, 1, 2, 0, 1, 2, 3, 4, 0, 1]
