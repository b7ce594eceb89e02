"""GPU check of examples/speculative_decode.py: products, reservation, append, attention and verification together.

Every call of a step is checked from the tensors that the step itself used, against the oracle: whole numbers for
equality, attention within its derived tolerance (see test_gpu_drafts.Shared.check).
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import drafts as odrafts
from oracle import kv as okv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().float().double().numpy()


def test_steps_of_drafts_and_their_check(monkeypatch):
    ex = example()
    rows, drafts, page, prompt = 5, 3, 8, 48
    s = ex.Speculation(rows, drafts, r_draft=4, heads=4, kv=2, dim=64, vocab=384, page=page, room=60, prompt=prompt, seed=1)
    s.read_prompt(torch.randint(0, 384, (prompt,), generator=s.gen, device="cuda", dtype=torch.int32))
    reserve, attend, verify = ex.nbw.kv_reserve, ex.nbw.kv_attend_shared, ex.nbw.verify_drafts
    seen = {"attend": 0}

    def spy_reserve(cache, lens, want, held, free, count, most, shared):
        args = [x.cpu().numpy().copy() for x in (cache.table, lens, want, held, free, shared)]
        ref = okv.reserve(args[0], page, cache.pages, args[1], args[2], args[3], args[4], int(count), most, args[5])
        got = reserve(cache, lens, want, held, free, count, most, shared=shared)
        for x, y in zip((cache.table, free, got.cu, got.positions, got.slots, got.granted, got.held, got.count), ref):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1))
        own = cache.table[:, prompt // page:]
        own = own[own >= 0]
        held_own = int(got.held.sum()) - rows * (prompt // page)
        assert held_own + int(got.count) == cache.pages - prompt // page and own.unique().numel() >= held_own
        return got

    def spy_attend(cache, q, lens, cu=None, groups=None, prefix=None):
        out = attend(cache, q, lens, cu=cu, groups=groups, prefix=prefix)
        cut = np.arange(rows + 1) if cu is None else cu.cpu().numpy()
        k, v, qq, table, n = f64(cache.k), f64(cache.v), f64(q), cache.table.cpu().numpy(), lens.cpu().numpy()
        want = okv.attend_tokens(qq, k, v, table, n, cut, 0.125)
        mean = okv.attend_tokens(qq, k, np.abs(v), table, n, cut, 0.125)
        size = np.abs(qq).sum(axis=2).max() * np.abs(k).max() * 0.125
        bound = 2.0**-8 * np.abs(want) + (2.0**-8 + 2 * 16 * 2.0**-24 * size) * mean + 1e-30
        assert np.all(np.abs(f64(out) - want) <= bound)
        seen["attend"] += 1
        return out

    def spy_verify(target, ids, u, draft=None, cu=None):
        got = verify(target, ids, u, draft=draft, cu=cu)
        cut = list(range(target.shape[0] + 1)) if cu is None else cu.tolist()
        ref = odrafts.verify(f64(target), [0] * target.shape[0] if ids is None else ids.tolist(), f64(u), cut,
                             None if draft is None else f64(draft))
        assert got[0].tolist() == ref[0] and got[1].tolist() == ref[1]
        return got

    monkeypatch.setattr(ex.nbw, "kv_reserve", spy_reserve)
    monkeypatch.setattr(ex.nbw, "kv_attend_shared", spy_attend)
    monkeypatch.setattr(ex.nbw, "verify_drafts", spy_verify)
    total = 0
    for step in range(10):
        before = s.lens.clone()
        accepted, last = s.step()
        assert bool((s.lens == before + accepted + 1).all()) and bool(((last >= 0) & (last < 384)).all())
        total += int(accepted.sum())
        # the prompt's pages are as they were read, the same for all
        assert bool((s.table[:, :prompt // page] == torch.arange(prompt // page, device="cuda")).all())
    assert seen["attend"] == 10 * (drafts + 1) and int(s.accepted) == total
    assert 0 < total < 10 * rows * drafts  # some drafts stand, some do not


def test_the_command_runs(capsys):
    assert example().main(["--rows", "2", "--steps", "5", "--drafts", "2", "--prompt", "32"]) == 0
    assert "drafts stood" in capsys.readouterr().out
